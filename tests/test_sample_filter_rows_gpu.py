"""Rows that the lists of the filtered token choice do not decide: what they give alone, among rows like them and beside
rows that bring the call its other kernels."""

import numpy as np
import pytest
import torch

from gpu_util import ready
from invariant_vd_step_gb300 import vd

pytestmark = pytest.mark.gpu


def choose(logits, samplers, filters):
    R = len(samplers)
    tok, lp = torch.full((R,), -9, dtype=torch.int32, device="cuda"), torch.full((R,), float("nan"), device="cuda")
    vd.sample(logits, samplers, filters, tok, lp)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy().view(np.int32)


def crowded_rows(kind, R, V, temps, rng):
    """Rows whose likeliest few hundred tokens stand side by side, so that no list holds them."""
    x = (rng.standard_normal((R, V)) * 2.0).astype(np.float32)
    if kind == "sorted":
        x.sort(axis=1)
    elif kind == "tied":  # few values, each shared by many tokens
        x = np.sort(np.round(x * 2) / 2, axis=1)
    else:  # packed: within a few hundredths of the temperature of one another
        for r in range(R):
            n, at = int(rng.integers(300, 1500)), int(rng.integers(0, V - 1500))
            x[r, at:at + n] = 12.0 - temps[r] * rng.uniform(0.01, 0.2) * rng.random(n).astype(np.float32)
    return x


@pytest.mark.parametrize("V", [8192, 33001])
@pytest.mark.parametrize("kind", ["sorted", "tied", "packed"])
def test_narrow_rows_do_not_depend_on_wide_rows(kind, V):
    """Token and log-probability, bit for bit, of rows of top_k 100 to 256: in a call without wide rows, and in one with a
    wide row at its front."""
    ready()
    rng = np.random.default_rng(V + len(kind))
    for turn in range(4):
        R = 500
        temps = rng.uniform(0.6, 1.6, R).astype(np.float32)
        x = crowded_rows(kind, R, V, temps, rng)
        s = [(int(rng.integers(0, 2 ** 62)), turn, float(t)) for t in temps]
        f = [(int(k), 1.0, float(m)) for k, m in zip(rng.integers(100, 257, R), rng.choice([0.0, 0.0, 1e-4, 0.3], R))]
        wide = (rng.standard_normal((1, V)) * 0.2).astype(np.float32)
        lg = torch.from_numpy(np.concatenate([wide, x])).cuda()
        alone = choose(lg[1:], s, f)
        beside = choose(lg, [(7, turn, 1.3)] + s, [(0, 0.95, 0.0)] + f)
        np.testing.assert_array_equal(beside[0][1:], alone[0])
        np.testing.assert_array_equal(beside[1][1:], alone[1])
        one = [choose(lg[1 + r:2 + r], s[r:r + 1], f[r:r + 1]) for r in range(0, R, 97)]
        np.testing.assert_array_equal([int(t[0]) for t, _ in one], alone[0][::97])
        np.testing.assert_array_equal([int(l[0]) for _, l in one], alone[1][::97])


@pytest.mark.parametrize("V", [1000, 40001])
def test_temperatures_whose_reciprocal_overflows(V):
    """At T = 1e-40, below float32's normal range, all mass is the largest logits': log-probability 0 for one of them,
    -log n for n that tie, and top-p keeps as many of those as it asks for."""
    ready()
    T = 1e-40
    rng = np.random.default_rng(V)
    x = -1.0 - rng.random((3, V)).astype(np.float32)
    x[0, 77], x[1, [3, 500, 999]], x[2, [5, 6]] = 2.0, 2.0, 2.0
    lg = torch.from_numpy(np.repeat(x, 4, axis=0)).cuda()
    filters = [(0, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.5), (0, 0.4, 0.0)] * 3
    tok, lp = choose(lg, [(1, k, T) for k in range(12)], filters)
    assert tok.tolist() == [77] * 4 + [3] * 4 + [5] * 4  # every score is infinite: the lowest index
    want = np.array([0.0] * 4 + [-np.log(3)] * 3 + [-np.log(2)] + [-np.log(2)] * 3 + [0.0])
    # log1p's error (2 ulp) and the rounding of a mass near 2 or 3 in float32: 2^-22 of values below 2
    assert np.all(np.abs(lp.view(np.float32) - want) <= 2.0 ** -21), lp.view(np.float32)
