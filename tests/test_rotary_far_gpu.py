"""Rotary angles at the largest positions against a reference of sixty digits."""

import math
from decimal import Decimal as D
from decimal import getcontext

import numpy as np
import pytest
import torch

from gpu_util import ready
from invariant_vd_step_gb300 import vd

pytestmark = pytest.mark.gpu

getcontext().prec = 60
TWO_PI = D("6.283185307179586476925286766559005768394338798750211641949889184615632812572")


def frequencies(rot, theta, scaling):
    f = [D(theta) ** (D(-2 * i) / rot) for i in range(rot // 2)]
    kind, factor = scaling["type"], D(scaling["factor"])
    if kind == "linear":
        return [v / factor for v in f]
    if kind == "bands":
        lo, hi = D(scaling["low_freq_factor"]), D(scaling["high_freq_factor"])
        k = [min(max((scaling["original_max_position"] * v / TWO_PI - lo) / (hi - lo), D(0)), D(1)) for v in f]
        return [a * v + (1 - a) * v / factor for a, v in zip(k, f)]
    at = [rot * math.log(scaling["original_max_position"] / (b * 2 * math.pi)) / (2 * math.log(theta)) for b in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    r = [min(max(D(i - lo) / (hi - lo), D(0)), D(1)) for i in range(rot // 2)]
    return [(1 - a) * v + a * v / factor for a, v in zip(r, f)]


@pytest.mark.parametrize("scaling", [
    {"type": "linear", "factor": 1.0}, {"type": "linear", "factor": 2.0 ** -10},
    {"type": "bands", "factor": 0.015625, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_max_position": 8192},
    {"type": "yarn", "factor": 0.015625, "original_max_position": 4096, "attn_factor": 1.0}], ids=lambda s: f"{s['type']}-{s['factor']}")
@pytest.mark.parametrize("theta", [5e5, 1e4, 10.0])
def test_positions_near_the_ends_of_int32(scaling, theta):
    ready()
    rot, rng = 128, np.random.default_rng(int(theta))
    pos = np.concatenate([2 ** 31 - 1 - rng.integers(0, 2 ** 20, 12), -2 ** 31 + rng.integers(0, 2 ** 20, 12), [-2 ** 31, 2 ** 31 - 1]])
    x = torch.randn((len(pos), 1, rot), generator=torch.Generator().manual_seed(1))
    got = vd.Rope(rot, theta=theta, scaling=scaling).apply(x.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda())
    f = frequencies(rot, theta, scaling)
    turns = np.array([[float((int(p) * v / TWO_PI) % 1) for v in f] for p in pos])
    c, s = np.cos(2 * math.pi * turns), np.sin(2 * math.pi * turns)
    x1, x2 = x[:, 0, :rot // 2].numpy().astype(np.float64), x[:, 0, rot // 2:].numpy().astype(np.float64)
    want = np.concatenate([x1 * c - x2 * s, x2 * c + x1 * s], 1)
    # sincospi within 2 ulp (2^-22), its argument's rounding (pi/4 2^-24) and the products' and the sum's: below 2^-21 of
    # |x1| + |x2|; the reduced angle 2^-32 turns, times a frequency's excess over 1
    angle = 2 * math.pi * 2.0 ** -32 * np.maximum(1.0, np.array([float(v) for v in f]))
    e = (np.abs(x1) + np.abs(x2)) * (2.0 ** -21 + np.minimum(angle, 2 * math.pi))
    err = np.abs(got[:, 0].cpu().numpy() - want)
    assert np.all(err <= np.concatenate([e, e], 1)), f"max {(err / np.concatenate([e, e], 1)).max():.3g} of the bound"
