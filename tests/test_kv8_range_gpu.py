"""Attention over the 8-bit cache where the V of one row's history differ by more than float32's range: every key keeps its
share of the softmax, whatever the V beside it."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from kv8_scenario import KV8Scenario, kv8_spec

pytestmark = pytest.mark.gpu


def check(sc, reqs, window=0, kernels=(1, 2)):
    """Both kernels give the same bits, within the tolerance of KV8Scenario.exact."""
    outs = [sc.attention(reqs, kernel=k) for k in kernels]
    for out in outs[1:]:
        np.testing.assert_array_equal(bits(out), bits(outs[0]))
    at = 0
    for i, c, n in reqs:
        want, tol = sc.exact(i, c, n, window)
        got = outs[0][at:at + n].double()
        err = (got - want).abs()
        assert (err <= tol).all(), (i, c, n, float((err / tol).nan_to_num(9e9).max()))
        at += n
    return outs[0]


def uniform(sc):
    """Queries of zeros: every key that a row sees weighs the same."""
    sc.q = [torch.zeros_like(q) for q in sc.q]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("e", [40, 46, 47, 60, 100, 120])
def test_zeros_beside_large_values(e, fmt):
    """V = 0 in sealed pages, own tokens, whole chunks and whole splits, beside V of 2^e, in either order."""
    ready()

    def edit(sc):
        uniform(sc)
        for r, large in enumerate([
                lambda t: t // 16 % 2 == 0,     # pages in turn
                lambda t: t // 16 % 2 == 1,
                lambda t: t % 2 == 0,           # tokens in turn: own pages with zero tokens
                lambda t: t < 16,               # one page, then zeros over two splits
                lambda t: t >= 640,             # zeros over more than a split, then large
                lambda t: t == 655]):           # the last token of the last own page
            t = torch.arange(sc.kv[r].shape[0] * 16).view(-1, 1, 16, 1)
            sc.kv[r][:, 1] = torch.where(large(t), 2.0 ** e, 0.0).bfloat16().expand(sc.kv[r][:, 1].shape)
    sc = KV8Scenario(kv8_spec(4, 2, 64), [656] * 6, fmt, seed=1, max_tokens=1400, edit=edit)
    out = check(sc, [(r, 655, 1) for r in range(6)])
    share = [21 / 41, 20 / 41, 0.5, 16 / 656, 16 / 656, 1 / 656]  # of 656 equal weights, 41 pages
    for r in range(6):
        want = share[r] * 2.0 ** e
        assert ((out[r].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want).all(), r
    check(sc, [(r, 500, 156) for r in range(6)])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("hd,Hq,Hkv,window", [(64, 4, 2, 0), (128, 8, 2, 300), (256, 4, 2, 0)])
def test_tiny_values_beside_large_ones(hd, Hq, Hkv, window, fmt):
    """Pages of V between 2^-70 and 2^110 in any order, ordinary scores: as single tokens and in chunks."""
    ready()
    g = torch.Generator().manual_seed(hd)

    def edit(sc):
        for kv in sc.kv:
            kv[:, 1] *= torch.exp2(torch.randint(-70, 111, (kv.shape[0], 1, 1, 1), generator=g).float()).bfloat16()
            kv[::5, 1] = 0
    sc = KV8Scenario(kv8_spec(Hq, Hkv, hd, window), [1100, 90, 700], fmt, seed=3, max_tokens=1400, edit=edit)
    check(sc, [(0, 1099, 1), (1, 89, 1), (2, 511, 1)], window)
    check(sc, [(0, 600, 500), (1, 0, 90), (2, 0, 700)], window)
    whole = bits(sc.attention([(0, 600, 500)]))
    for c in (600, 767, 768, 1023, 1024, 1099):
        np.testing.assert_array_equal(bits(sc.attention([(0, c, 1)]))[0], whole[c - 600], err_msg=str(c))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_blocks_that_fold_their_own_splits(fmt):
    """Zeros, large and tiny V over several splits in blocks that write the output themselves."""
    ready()

    def edit(sc):
        for v, e in ((sc.kv[0][:, 1], 90), (sc.kv[1][:, 1], -60)):
            v[:36] = 0                  # the first split and a bit
            v[36:70] *= 2.0 ** e
            v[70:72] *= 2.0 ** -e
    sc = KV8Scenario(kv8_spec(32, 8, 128), [1500, 1300], fmt, seed=8, max_tokens=2300, edit=edit)
    out = check(sc, [(0, 200, 1300), (1, 500, 800)])
    for c in (200, 511, 600, 1024, 1499):
        np.testing.assert_array_equal(bits(sc.attention([(0, c, 1)]))[0], bits(out)[c - 200], err_msg=str(c))


@pytest.mark.parametrize("kernel", [1, 2])
@pytest.mark.parametrize("e", [-60, 0, 60])
def test_one_key_wins_by_far_whatever_its_v(e, kernel):
    """Scores of 2^30 and more apart, where the V scale is lost in their last place: the row is the winner's value."""
    ready()

    def edit(sc):
        kv = sc.kv[0]
        kv[:, 0] = 0
        kv[3, 0, :, 5] = 2.0 ** 20      # a key of a sealed page, then one of its own page
        kv[12, 0, :, 4] = 2.0 ** 24
        kv[:, 1] *= 2.0 ** e
        sc.q = [torch.full_like(sc.q[0], 2.0 ** 10)]
    sc = KV8Scenario(kv8_spec(4, 2, 64), [200], "int8", seed=4, edit=edit)
    out = sc.attention([(0, 100, 100)], kernel=kernel).double()
    for p in range(100, 200):
        want = sc.exact(0, p, 1)[0][0]
        # int8 codes, and the product, off by 2^-8 together with the rounding to bf16
        assert ((out[p - 100] - want).abs() <= 2.0 ** -7 * want.abs()).all(), p
