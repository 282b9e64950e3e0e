"""Calls with more pages than one launch takes, and layers of a model of which some are local."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import vd
from kv8_scenario import KV8Scenario, kv8_spec, sealed_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [448, 449, 4000, 4001, 8100])
def test_seals_and_copies_of_many_pages(n):
    """On both sides of the sizes at which the page lists change their place, or take another launch."""
    ready()
    rng = np.random.default_rng(n)
    model = KV8Scenario(kv8_spec(2, 1, 64), [16], "int8").model
    mem = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")  # noqa: E731
    pool = vd.KVPool(model, 2 * n, memory=mem(model.pool_bytes(2 * n)))
    cache = vd.KV8Cache(model, 2 * n, "int8", memory=mem(model.kv8_bytes(2 * n)))
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(pool.view().shape, generator=g, device="cuda").bfloat16()
    pool.view().copy_(x)
    src, dst = rng.permutation(2 * n)[:n], rng.permutation(2 * n)[:n]
    cache.seal(pool, src, dst)
    pool.view().fill_(3.0)
    back = rng.permutation(2 * n)[:n]
    cache.unseal(pool, dst, back)
    want = torch.full_like(x, 3.0)
    want[:, back] = sealed_values(x[:, src], "int8").bfloat16()
    # (2^-8 of a value and 2^-22 for the scale and the product in float32, as one rounding to bf16 may go either way)
    assert ((pool.view().double() - want.double()).abs() <= (2.0 ** -8 + 2.0 ** -22) * want.double().abs()).all()
    order = rng.permutation(2 * n)
    for pages, parts in ((pool, [pool.view]), (cache, [cache.codes, cache.scales])):
        before = [p().clone() for p in parts]
        pages.copy_pages(order[:n], order[n:])
        torch.cuda.synchronize()
        for p, b in zip(parts, before):
            b[:, order[n:]] = b[:, order[:n]]
            assert torch.equal(p().view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("Hq,Hkv,hd,window", [(32, 8, 128, 300), (12, 4, 64, 700), (48, 24, 256, 100)])
def test_local_layers_beside_global_ones(Hq, Hkv, hd, window, fmt):
    """One plan for a model whose layers take turns: long chunks, most of whose blocks fold their own splits, and a single
    token, in either layer, against 64 bits, the mma.sync kernel and tokens alone."""
    ready()
    spec = kv8_spec(Hq, Hkv, hd, window, layers=2).with_(local_global_period=2)
    sc = KV8Scenario(spec, [1500, 700, 900], fmt, seed=8, max_tokens=2100)
    reqs = [(2, 899, 1), (0, 200, 1300), (1, 0, 700)]
    for layer in (0, 1):
        w = window if layer % 2 == 0 else 0  # every second layer is global
        out = sc.attention(reqs, layer=layer, kernel=2)
        got = bits(out)
        np.testing.assert_array_equal(bits(sc.attention(reqs, layer=layer, kernel=1)), got)
        for c in (200, 511, 777, 1024, 1499):
            np.testing.assert_array_equal(bits(sc.attention([(0, c, 1)], layer=layer))[0], got[1 + c - 200], err_msg=str(c))
        at = 0
        for rid, c, n in reqs:
            want, tol = sc.exact(rid, c, n, w)
            assert ((out[at:at + n].double() - want).abs() <= tol).all(), (layer, rid)
            at += n
