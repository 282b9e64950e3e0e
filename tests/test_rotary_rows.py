"""Rows of the rotary op's output that overlap are refused, on the host, whatever the strides."""

from invariant_vd_step_gb300 import build, vd


def layouts():
    """(T, H, token stride, head stride, whether two rows of 6 elements share one) for every small layout."""
    for T in (1, 2, 3, 5):
        for H in (1, 2, 4):
            for st in (*range(0, 40), 63):
                for sh in (0, 1, 5, 6, 7, 8, 11, 12, 13, 18, 19, 24, 25, 31, 47):
                    starts = sorted(t * st + h * sh for t in range(T) for h in range(H))
                    yield T, H, st, sh, any(b - a < 6 for a, b in zip(starts, starts[1:]))


def test_overlapping_rows_are_refused():
    build.build()
    L, r = vd.lib(), vd.Rope(6)
    n = 0
    for T, H, st, sh, overlap in layouts():
        if overlap:  # (the others would run)
            for a, b in ((1, 1), (-1, 1), (1, -1)):
                assert L.vd_op_rotary(r.h, 64, 1 << 20, T, H, 6, 6, a * st, b * sh, 0, 64, 0, None) == vd.VD_ERR_INVALID_ARG
                n += 1
    assert n > 1000
    least, most = -2 ** 63, 2 ** 63 - 1  # strides whose products need more than 64 bits
    for T, H, st, sh in ((3, 2, most // 2, most), (2, 2, least, least), (2, 3, most, most // 2 - 2), (2, 2, 0, least)):
        assert L.vd_op_rotary(r.h, 64, 1 << 20, T, H, 6, 6, st, sh, 0, 64, 0, None) == vd.VD_ERR_INVALID_ARG
