"""Refusals of the rotary op on the host: rows of the output that overlap, whatever the strides, and magnitudes that
float32 does not hold."""

import pytest

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


@pytest.mark.parametrize("attn_factor,taken", [(0.0, True), (1.25, True), (1e-30, True), (1e30, True), (1e-46, False),
                                               (1e-40, False), (1e39, False), (3e38, False), (1e300, False), (1e-300, False)])
def test_magnitudes_that_float32_holds(attn_factor, taken):
    """The op multiplies by the magnitude, or by its inverse, in float32: neither may be zero, infinite or subnormal."""
    build.build()
    scaling = {"type": "linear", "factor": 2.0, "attn_factor": attn_factor}
    if taken:
        vd.Rope(64, scaling=scaling)
        return
    with pytest.raises(vd.VDError) as e:
        vd.Rope(64, scaling=scaling)
    assert e.value.code == vd.VD_ERR_INVALID_ARG
