"""Copies of pages of the bf16 pool and of the 8-bit cache."""

import numpy as np
import pytest
import torch

from gpu_util import ready
from invariant_vd_step_gb300 import vd
from kv8_scenario import KV8Scenario, kv8_spec

pytestmark = pytest.mark.gpu


def make(kind, Hkv, hd, layers, pages):
    model = KV8Scenario(kv8_spec(2 * Hkv, Hkv, hd, layers=layers), [16], "int8").model
    g = torch.Generator(device="cuda").manual_seed(pages)
    nbytes = model.pool_bytes(pages) if kind == "bf16" else model.kv8_bytes(pages)
    mem = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    cache = vd.KVPool(model, pages, memory=mem) if kind == "bf16" else vd.KV8Cache(model, pages, kind, memory=mem)
    mem.copy_(torch.randint(0, 256, mem.shape, generator=g, device="cuda", dtype=torch.uint8))
    parts = [mem.view(layers, pages, -1)] if kind == "bf16" else \
        [cache.codes().view(layers, pages, -1), cache.scales().view(torch.uint8).view(layers, pages, -1)]
    return cache, parts


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3"])
@pytest.mark.parametrize("Hkv,hd,layers,pages,n", [(1, 128, 1, 2, 1), (2, 64, 3, 9, 4), (5, 256, 2, 40, 20),
                                                   (1, 128, 2, 2000, 1000), (24, 128, 1, 6, 2)])
def test_copies(kind, Hkv, hd, layers, pages, n):
    ready()
    cache, parts = make(kind, Hkv, hd, layers, pages)
    order = np.random.default_rng(n).permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    src[-1] = src[0]  # one page to several
    want = [p.clone() for p in parts]
    for w in want:
        w[:, dst] = w[:, src]
    cache.copy_pages(src, dst)
    torch.cuda.synchronize()
    for p, w in zip(parts, want):
        assert torch.equal(p, w)
    cache.copy_pages([], [])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_copies_in_a_captured_graph_and_on_a_stream(kind):
    ready()
    cache, parts = make(kind, 2, 64, 2, 12)
    first = [p.clone() for p in parts]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cache.copy_pages([1, 2], [3, 4], stream=s)
    torch.cuda.synchronize()
    for p, w in zip(parts, first):
        assert torch.equal(p, w)
    for _ in range(2):
        for p in parts:
            p[:, 1] += 1
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for p in parts:
            assert torch.equal(p[:, 3], p[:, 1]) and torch.equal(p[:, 4], p[:, 2])
    s.wait_stream(torch.cuda.current_stream())
    cache.copy_pages([5], [6], stream=s)
    cache.copy_pages([6], [7], stream=s)  # in the stream's order
    torch.cuda.synchronize()
    for p in parts:
        assert torch.equal(p[:, 7], p[:, 5])


@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_refusals(kind):
    ready()
    cache, parts = make(kind, 1, 128, 1, 4)
    before = [p.clone() for p in parts]
    for code, src, dst in [(3, [4], [0]), (3, [0], [4]), (3, [-1], [0]), (1, [0, 1], [2, 2]), (1, [0, 2], [2, 3]),
                           (1, [1], [1]), (1, [0, 1], [2]), (1, [0.5], [2])]:
        with pytest.raises(vd.VDError) as e:
            cache.copy_pages(src, dst)
        assert e.value.code == code, (src, dst, e.value)
    cache.close()
    with pytest.raises(vd.VDError):
        cache.copy_pages([0], [1])
    torch.cuda.synchronize()
    for p, w in zip(parts, before):
        assert torch.equal(p, w)
