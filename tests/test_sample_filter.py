"""Filtered token choice on the host: argument checks and the oracle's pins."""

import numpy as np

from filter_oracle import row_choice, words
from invariant_vd_step_gb300 import build, vd
from oracle import sampler as osm


def test_oracle_words_and_unfiltered_choice_agree_with_the_sampler_oracle():
    rng = np.random.default_rng(0)
    for seed, step in ((0, 0), (2 ** 64 - 1, 2 ** 40 + 3), (123456789, 7)):
        np.testing.assert_array_equal(words(np.arange(101), seed, step), osm.philox_words(seed, step, 101))
        x = rng.standard_normal(101)
        for t in (0.0, 0.5, 1.5):
            assert row_choice(x, (seed, step, t), (0, 1.0, 0.0), 0.0)[0] == osm.sample(x, np.float64(np.float32(t)), seed, step)


def test_oracle_filters():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.25, 0.05]))
    seen = {f: {row_choice(x, (s, 0, 1.0), f, 0.0)[0] for s in range(300)} for f in
            [(2, 1.0, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.45), (4, 0.9, 0.3), (0, 0.0, 0.0)]}
    assert seen == {(2, 1.0, 0.0): {1, 3}, (0, 0.6, 0.0): {1, 3}, (0, 1.0, 0.45): {1, 2, 3}, (4, 0.9, 0.3): {1, 2, 3},
                    (0, 0.0, 0.0): {1}}


def test_arguments_are_checked_before_any_cuda_call():
    build.build()
    L = vd.lib()
    s, f = np.zeros(2, vd.SAMPLER), np.zeros(2, vd.FILTER)
    ws = L.vd_sample_workspace_bytes(2, 100)
    assert ws > 0 and L.vd_sample_workspace_bytes(-1, 100) == 0
    ok = [64, 2, 100, 100, s.ctypes.data, f.ctypes.data, 64, 64, 64, ws, None]
    for at, value, code in [(0, None, 1), (1, -1, 1), (2, 0, 1), (3, 99, 1), (4, None, 1), (6, None, 1), (8, None, 1),
                            (0, 66, 1), (6, 66, 1), (7, 66, 1), (8, 72, 1), (2, 2 ** 21 + 1, 2), (9, ws - 1, 4)]:
        a = list(ok)
        a[at] = value
        if at == 2 and code == 2:
            a[3] = value
        assert L.vd_op_sample(*a) == code, (at, value)
    for field, value in (("top_k", -1), ("top_p", 1.01), ("top_p", -0.5), ("top_p", np.nan), ("min_p", 1.5),
                         ("min_p", np.nan)):
        f["top_k"], f["top_p"], f["min_p"] = 0, 1.0, 0.0
        f[field][1] = value
        assert L.vd_op_sample(*ok) == 1, (field, value)
    a = list(ok)
    a[1] = 0
    assert L.vd_op_sample(*a) == 0  # no rows, nothing to do
    assert L.vd_sample_filtered(None, None, 1, None, None, None, None, None) == 1
