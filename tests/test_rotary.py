"""Rope configurations on the host: refusals, and the frequency scalings' definitions."""

import math

import numpy as np
import pytest

from invariant_vd_step_gb300 import build, vd

SCALINGS = {
    "linear": {"type": "linear", "factor": 4.0},
    "bands": {"type": "bands", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
              "original_max_position": 8192},
    "yarn": {"type": "yarn", "factor": 16.0, "original_max_position": 4096},
}


def frequencies(rot, theta, scaling):
    """Angle per position of each pair in float64 and the magnitude, from the published definitions."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling is None:
        return f, 1.0
    if scaling["type"] == "linear":
        return f / scaling["factor"], 1.0
    L = scaling["original_max_position"]
    out = f.copy()
    if scaling["type"] == "bands":
        lo, hi = scaling["low_freq_factor"], scaling["high_freq_factor"]
        for i, v in enumerate(f):
            wave = 2 * math.pi / v
            if wave > L / lo:
                out[i] = v / scaling["factor"]
            elif wave >= L / hi:
                k = (L / wave - lo) / (hi - lo)
                out[i] = k * v + (1 - k) * v / scaling["factor"]
        return out, 1.0
    pair = [rot * math.log(L / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
    lo, hi = max(math.floor(pair[0]), 0), min(math.ceil(pair[1]), rot - 1)
    for i, v in enumerate(f):
        r = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
        out[i] = v * (1 - r) + v / scaling["factor"] * r
    return out, 0.1 * math.log(scaling["factor"]) + 1.0


def test_rope_configurations_are_validated():
    build.build()
    vd.Rope(128, 64, "interleaved", 1e4, SCALINGS["yarn"])
    bad = [dict(head_dim=63), dict(head_dim=64, rot_dim=66), dict(head_dim=64, rot_dim=3), dict(head_dim=0),
           dict(head_dim=64, layout="quarter"), dict(head_dim=64, theta=1.0), dict(head_dim=64, theta=float("nan")),
           dict(head_dim=64, theta=float("inf")), dict(head_dim=64, scaling={"type": "cubic"}),
           dict(head_dim=64, scaling={"type": "linear", "factor": 0}),
           dict(head_dim=64, scaling={"type": "linear"}), dict(head_dim=64, scaling={"type": "linear", "facto": 2}),
           dict(head_dim=64, scaling={**SCALINGS["bands"], "high_freq_factor": 1.0}),
           dict(head_dim=64, scaling={**SCALINGS["bands"], "original_max_position": 0}),
           dict(head_dim=64, scaling={**SCALINGS["yarn"], "beta_slow": 40}),
           dict(head_dim=64, scaling={**SCALINGS["yarn"], "attn_factor": -1})]
    for kw in bad:
        with pytest.raises(vd.VDError):
            vd.Rope(**kw)
    with pytest.raises(vd.VDError) as e:
        vd.Rope(1024)
    assert e.value.code == vd.VD_ERR_UNSUPPORTED


def test_rotary_op_validates_before_any_cuda_call():
    build.build()
    L, r = vd.lib(), vd.Rope(64)
    ok = [r.h, 64, 128, 4, 2, 128, 64, 128, 64, 0, 64, 0, None]
    for at, value in [(0, None), (1, None), (2, None), (3, -1), (4, -1), (1, 65), (9, 3), (9, -1), (10, None), (10, 66),
                      (11, 2), (7, 64), (8, 32), (7, 100), (8, 0)]:
        a = list(ok)
        a[at] = value
        assert L.vd_op_rotary(*a) == vd.VD_ERR_INVALID_ARG, (at, value)
    a = list(ok)
    a[2], a[7], a[8] = 64, 512, 64   # in place with other strides
    assert L.vd_op_rotary(*a) == vd.VD_ERR_INVALID_ARG
    a = list(ok)
    a[3] = 0
    assert L.vd_op_rotary(*a) == vd.VD_OK  # nothing to do
    assert L.vd_set_rope(None, r.h, None) == vd.VD_ERR_INVALID_ARG
    assert L.vd_rope_create(None, None) == vd.VD_ERR_INVALID_ARG
