"""The 8-bit cache on a GPU: sealing, attention against 64 bits, and rows that do not depend on how they are run."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import vd
from kv8_scenario import KV8Scenario, e4m3, kv8_spec, sealed_values

pytestmark = pytest.mark.gpu

FORMATS = ["int8", "e4m3"]


def _pool(model, x):
    pool = vd.KVPool(model, x.shape[1], memory=torch.zeros(x.nbytes, dtype=torch.uint8, device="cuda"))
    pool.view().copy_(x)
    return pool


def _decode(cache, fmt):
    """Codes [L][P][2][Hkv][16][hd] (64 bits) by the layout formula of vd_kv8.h, and scales."""
    raw, (L, P, H, n) = cache.codes(), cache.codes().shape
    hd = n // 32
    j, c = torch.meshgrid(torch.arange(16), torch.arange(hd), indexing="ij")
    k = (c // 32) * 512 + ((j % 8) * 4 + (c % 8) // 2) * 16 + (c // 16 % 2) * 8 + (j // 8) * 4 + (c // 8 % 2) * 2 + c % 2
    v = 16 * hd + (c // 32) * 512 + ((c % 8) * 4 + (j % 8) // 2) * 16 + (c // 8 % 4) * 4 + (j // 8) * 2 + j % 2
    at = torch.stack([k, v]).reshape(-1).cuda()
    assert len(set(at.tolist())) == n
    x = raw[..., at].view(L, P, H, 2, 16, hd).transpose(2, 3)
    return (x.double() - 128 if fmt == "int8" else x.view(torch.float8_e4m3fn).double()), cache.scales()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hd,Hkv,layers,pages", [(64, 2, 2, 5), (128, 1, 3, 449), (256, 3, 1, 7)])
def test_seal_and_unseal_are_the_definitions(fmt, hd, Hkv, layers, pages):
    ready()
    model = KV8Scenario(kv8_spec(2 * Hkv, Hkv, hd, layers=layers), [16], fmt).model
    g = torch.Generator(device="cuda").manual_seed(hd)
    x = torch.randn((layers, pages, 2, Hkv, 16, hd), generator=g, device="cuda") * \
        torch.exp2(torch.randint(-20, 20, (layers, pages, 2, Hkv, 1, 1), generator=g, device="cuda").float())
    x[:, 0] = 0                       # a block of zeros
    x[:, 1, 0] = 2.0 ** -90           # below the least scale
    x[:, 2, 1] = x[:, 2, 1].sign() * torch.randint(1, 128, x[:, 2, 1].shape, generator=g, device="cuda") / 2
    x[:, 2, 1, :, 0, 0] = 63.5        # with a = 63.5 or 127 / 2: quotients that are ties
    x[:, 3, 0, 0, 7, 11] = float("inf")
    x[:, 3, 1, -1, 15, hd - 1] = float("nan")
    x = x.bfloat16()
    mem = torch.full((model.kv8_bytes(pages + 2),), 77, dtype=torch.uint8, device="cuda")
    cache = vd.KV8Cache(model, pages + 2, fmt, memory=mem)
    assert not mem.any()
    mem.fill_(77)
    src = np.random.default_rng(1).permutation(pages)
    dst = np.random.default_rng(2).permutation(pages + 2)[:pages]
    pool = _pool(model, x)
    cache.seal(pool, src, dst)
    codes, scales = _decode(cache, fmt)
    xs, codes, scales = x[:, src].double(), codes[:, dst], scales[:, dst]
    a = xs.abs().amax((-2, -1), keepdim=True).clamp(min=2.0 ** -80)
    fin = a.isfinite()
    want = torch.round(xs * 127 / a) if fmt == "int8" else e4m3(xs * 448 / a)
    assert torch.equal(codes, torch.where(fin, want, 0.0))  # the code of the exact quotient, everywhere
    s = (a[..., 0, 0] / (127 if fmt == "int8" else 448)).float()  # float32 quotient, rounded once
    ok = fin[..., 0, 0]
    got = torch.stack([scales[..., 0], scales[..., 3]], 2)
    assert torch.equal(got.isnan(), ~ok)
    # one rounding each (2^-24), of a quotient here taken in 64 bits first
    assert ((got - s).abs()[ok] <= 2.0 ** -23 * s[ok]).all()
    kn, vn = ok[:, :, 0], ok[:, :, 1]
    assert ((scales[..., 1] * scales[..., 3] - 1).abs()[vn] <= 2.0 ** -22).all()
    assert ((scales[..., 2] - scales[..., 3].log2()).abs()[vn] <= 1e-5).all() and scales[..., 1][~vn].isnan().all()
    # pages that were not named are as they were
    rest = torch.tensor(sorted(set(range(pages + 2)) - set(dst.tolist())), device="cuda")
    assert (cache.codes()[:, rest] == 77).all() and (cache.scales()[:, rest].view(torch.uint8) == 77).all()
    back = _pool(model, torch.full_like(x, 3.0))
    cache.unseal(back, dst[:-1], src[:-1])
    want = sealed_values(x[:, src], fmt)
    got = back.view()[:, src].double()
    assert (got[:, -1] == 3).all()
    want, got = want[:, :-1], got[:, :-1]
    assert torch.equal(got.isnan(), want.isnan())
    err = (got - want).abs()
    # bf16 of code * scale: 2^-8, and 2^-23 for the scale and product in float32
    assert (err[~want.isnan()] <= (2.0 ** -8 + 2.0 ** -22) * want.abs()[~want.isnan()]).all()
    assert kn.any()


def test_seal_takes_one_layer_and_a_page_into_several():
    ready()
    model = KV8Scenario(kv8_spec(4, 2, 64, layers=3), [16], "int8").model
    x = torch.randn((3, 4, 2, 2, 16, 64), device="cuda").bfloat16()
    mem = torch.zeros(model.kv8_bytes(6), dtype=torch.uint8, device="cuda")
    cache, pool = vd.KV8Cache(model, 6, "int8", memory=mem), _pool(model, x)
    cache.seal(pool, [2, 2, 0], [5, 1, 3], layer=1)
    assert not cache.codes()[0].any() and not cache.codes()[2].any()
    assert torch.equal(cache.codes()[1, 5], cache.codes()[1, 1]) and cache.codes()[1, 5].any()
    cache.seal(pool, [2, 0], [5, 3])
    want = cache.codes()[1, [5, 3]].clone()
    cache.seal(pool, [2, 0], [0, 2], layer=1)
    assert torch.equal(cache.codes()[1, [0, 2]], want)
    cache.seal(pool, [], [])


# heads, head dim, window, requests (cached, new): single tokens, chunks, boundaries of pages, chunks of 128 and splits of 512
SHAPES = [
    (4, 2, 64, 0, [(0, 1), (15, 1), (16, 1), (31, 2), (127, 1), (128, 1), (511, 1), (512, 1), (1030, 1)]),
    (32, 8, 128, 0, [(0, 1), (1, 1), (700, 1), (1023, 2), (47, 4)]),
    (8, 8, 128, 0, [(5, 16), (500, 16), (640, 9), (15, 17)]),
    (16, 1, 128, 0, [(9, 1), (600, 1), (130, 2)]),
    (8, 4, 256, 0, [(0, 1), (300, 1), (511, 8), (1000, 3)]),
    (8, 4, 256, 64, [(0, 1), (300, 1), (511, 8), (1000, 3), (62, 70)]),
    (4, 2, 64, 1, [(0, 1), (300, 1), (15, 2)]),
    (4, 2, 64, 17, [(0, 40), (300, 1), (511, 20)]),
    (8, 2, 128, 200, [(0, 33), (511, 1), (900, 130), (190, 1)]),
    (4, 4, 64, 0, [(0, 300), (513, 77)]),
    (12, 4, 128, 0, [(0, 65), (250, 140), (1, 1)]),
    (32, 2, 64, 0, [(33, 20)]),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,hd,window,reqs", SHAPES)
def test_attention_against_64_bits(Hq, Hkv, hd, window, reqs, fmt):
    ready()
    sc = KV8Scenario(kv8_spec(Hq, Hkv, hd, window), [c + n for c, n in reqs], fmt, seed=hd + window)
    for kernel in (1, 2):
        out = sc.attention([(i, c, n) for i, (c, n) in enumerate(reqs)], kernel=kernel).double()
        at = 0
        for i, (c, n) in enumerate(reqs):
            want, tol = sc.exact(i, c, n, window)
            err = (out[at:at + n] - want).abs()
            assert (err <= tol).all(), (kernel, i, c, n, float((err / tol).max()))
            at += n


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,hd,window", [(4, 2, 64, 0), (8, 2, 128, 0), (8, 4, 256, 100), (16, 1, 128, 0), (4, 4, 64, 30),
                                              (8, 1, 256, 0)])
def test_rows_do_not_depend_on_how_they_are_run(Hq, Hkv, hd, window, fmt):
    """A prompt at once, in chunks, token by token, alone and beside others, anywhere in the cache: the same bits."""
    ready()
    n = 661
    sc = KV8Scenario(kv8_spec(Hq, Hkv, hd, window), [n, 300, 40], fmt, seed=9, max_tokens=2048)
    whole = bits(sc.attention([(0, 0, n)]))
    for kernel in (1, 2):
        np.testing.assert_array_equal(bits(sc.attention([(0, 0, n)], kernel=kernel)), whole, err_msg=str(kernel))
    for cuts in ([(0, 16), (16, 17), (33, 95), (128, 400), (528, 133)], [(0, 650), (650, 11)]):
        for c, k in cuts:
            for kernel in (0, 2):
                got = bits(sc.attention([(1, 299, 1), (0, c, k), (2, 0, 40)], kernel=kernel))
                np.testing.assert_array_equal(got[1:1 + k], whole[c:c + k], err_msg=f"{c} {k} {kernel}")
    for c in (0, 1, 15, 16, 100, 127, 128, 129, 511, 512, 640, 660):
        k = min(16 // (Hq // Hkv), n - c)
        for m in {1, max(1, min(2, k)), k}:
            got = bits(sc.attention([(0, c, m), (1, 7, 1)], scatter=c % 2 == 0))
            np.testing.assert_array_equal(got[:m], whole[c:c + m], err_msg=f"{c} {m}")


def test_many_requests_and_odd_orders():
    """More requests than one search step of the plan takes, both classes, random splits."""
    ready()
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(1, 260, 70)]
    sc = KV8Scenario(kv8_spec(8, 2, 64), lens, "int8", seed=5)
    reqs = []
    for i in rng.permutation(70):
        c = int(rng.integers(0, lens[i]))
        reqs.append((int(i), c, lens[i] - c if rng.random() < 0.5 else 1))
    for kernel in (0, 2):
        out, at = sc.attention(reqs, kernel=kernel).double(), 0
        for i, c, n in reqs:
            want, tol = sc.exact(i, c, n)
            assert ((out[at:at + n] - want).abs() <= tol).all(), (kernel, i, c, n)
            at += n


@pytest.mark.parametrize("fmt", FORMATS)
def test_scales_that_differ_by_many_orders(fmt):
    """Pages whose V are tiny, zero or huge beside the others: the V scale enters through the exponent."""
    ready()

    def edit(sc):
        kv = sc.kv[0]
        kv[3, 1] *= 2.0 ** -60
        kv[5, 1] = 0
        kv[9, 1] *= 2.0 ** 40
        kv[2, 0] = 0
        kv[11, 1] *= 2.0 ** -30
        kv[-1, 1, :, 3] *= 2.0 ** 30
        sc.kv[1][:, 1] *= 2.0 ** -70     # a whole request of tiny values
        sc.kv[2][:, 1] = 0               # and one of zeros
    sc = KV8Scenario(kv8_spec(4, 2, 128), [220, 150, 90], fmt, seed=2, edit=edit)
    reqs = [(0, 0, 220), (1, 149, 1), (2, 50, 40)]
    for kernel in (1, 2):
        out, at = sc.attention(reqs, kernel=kernel).double(), 0
        for i, c, n in reqs:
            want, tol = sc.exact(i, c, n)
            err = (out[at:at + n] - want).abs()
            assert (err <= tol).all(), (kernel, i, float((err - tol).max()))
            at += n
        assert (out[221:] == 0).all()


@pytest.mark.parametrize("q_scale", [2.0 ** -100, 30.0, 2.0 ** 60])
def test_queries_of_any_size(q_scale):
    """Uniform weights, weights on one key, and scores beyond what float32 tells apart but for the largest."""
    ready()
    sc = KV8Scenario(kv8_spec(4, 2, 64), [200], "int8", seed=4, q_scale=q_scale)
    out = sc.attention([(0, 100, 100)]).double()
    want, tol = sc.exact(0, 100, 100)
    if q_scale < 2.0 ** 50:
        assert ((out - want).abs() <= tol).all()
    else:  # the largest score wins by far more than float32's error of the others
        assert out.isfinite().all() and ((out - want).abs() <= tol).double().mean() > 0.99


@pytest.mark.parametrize("kind", ["inf", "nan"])
@pytest.mark.parametrize("which", [0, 1])
def test_values_that_are_not_finite_reach_the_rows_that_see_them_only(kind, which):
    """One K or V value of token 70 (page 4): rows of page 4 from 70 on see it in bf16, later rows see the whole page NaN;
    rows before it, and rows whose window has passed page 4, are as without it."""
    ready()
    n, window = 200, 48

    def edit(sc):
        sc.kv[0][4, which, :, 6, 5] = float(kind)
    for w in (0, window):
        spec = kv8_spec(8, 4, 64, w)
        clean = bits(KV8Scenario(spec, [n], "int8", seed=6).attention([(0, 0, n)]))
        sc = KV8Scenario(spec, [n], "int8", seed=6, edit=edit)
        for reqs in ([(0, 0, n)], [(0, 33, 90)], [(0, 69, 1)], [(0, 70, 2)], [(0, 126, 1)], [(0, 128, 2)]):
            c, k = reqs[0][1:]
            out = sc.attention(reqs, kernel=1)
            np.testing.assert_array_equal(bits(sc.attention(reqs, kernel=2)), bits(out))
            for r in range(k):
                p = c + r
                sees = 70 <= p < 80 if p // 16 == 4 else p >= 80 and (w == 0 or p - w + 1 <= 79)
                if p // 16 == 4 and w and p - w + 1 > 70:
                    sees = False
                if sees:
                    # an infinite key gives its row a weight of 0 or NaN: NaN unless every product with it is -inf
                    if not (which == 0 and kind == "inf" and p < 80):
                        assert out[r].isnan().all(), (w, p)
                else:
                    np.testing.assert_array_equal(bits(out[r]), clean[p], err_msg=f"{w} {p}")


@pytest.mark.parametrize("Hq,Hkv,hd,window", [(32, 8, 128, 0), (12, 4, 64, 700), (24, 8, 128, 0)])
def test_blocks_that_fold_their_splits_and_blocks_cut_into_runs(Hq, Hkv, hd, window):
    """More row blocks than SMs, over several splits: most fold their own splits, the last ones leave them to the merge;
    with 3 heads per KV head a token's rows may lie in two blocks.  Every row as its token alone."""
    ready()
    n = 1500
    sc = KV8Scenario(kv8_spec(Hq, Hkv, hd, window), [n, 700], "int8", seed=8, max_tokens=2300)
    reqs = [(0, 200, n - 200), (1, 0, 700)]
    got = bits(sc.attention(reqs, kernel=2))
    np.testing.assert_array_equal(bits(sc.attention(reqs, kernel=1)), got)
    for c in (200, 511, 777, 1024, n - 1):
        np.testing.assert_array_equal(bits(sc.attention([(0, c, 1)]))[0], got[c - 200], err_msg=str(c))
    want, tol = sc.exact(1, 0, 700, window)
    assert ((sc.attention(reqs, kernel=2)[n - 200:].double() - want).abs() <= tol).all()


def test_streams_and_two_plans():
    """Two plans over one cache on two streams at once, and the same on one: the same bits."""
    ready()
    sc = KV8Scenario(kv8_spec(8, 2, 128), [900, 700], "e4m3", seed=7)
    cu, cached, t8, t16, _ = sc.setup([(0, 300, 600), (1, 699, 1)])
    q = [sc.q[0][300:900], sc.q[1][699:700]]
    want = [bits(sc.attention([(0, 300, 600)])), bits(sc.attention([(1, 699, 1)]))]
    cu, cached, t8, t16, _ = sc.setup([(0, 300, 600), (1, 699, 1)])
    plans = [vd.KV8Plan(sc.model, 600), vd.KV8Plan(sc.model, 1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.full_like(x, float("nan")) for x in q]
    torch.cuda.synchronize()
    for rep in range(3):
        for i in (0, 1):
            plans[i].plan(sc.cache, sc.pool, [0, len(q[i])], cached[i:i + 1], t8[i:i + 1], t16[i:i + 1], stream=streams[i])
            plans[i].seal(sc.cache, sc.pool, 0, stream=streams[i])
            plans[i].attention(sc.cache, sc.pool, 0, q[i], outs[i], stream=streams[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            np.testing.assert_array_equal(bits(outs[i]), want[i])


def test_refusals():
    ready()
    sc = KV8Scenario(kv8_spec(4, 2, 64, layers=2), [40, 40], "int8", max_tokens=64)
    other = KV8Scenario(kv8_spec(4, 2, 64, layers=2), [40], "int8")
    cu, cached, t8, t16, _ = sc.setup([(0, 20, 13), (1, 31, 1)])
    other.setup([(0, 20, 2)])
    plan = vd.KV8Plan(sc.model, 32)
    q = torch.zeros((14, 4, 64), dtype=torch.bfloat16, device="cuda")

    def refused(code, f, *a, **k):
        with pytest.raises(vd.VDError) as e:
            f(*a, **k)
        assert e.value.code == code, (e.value, code)

    refused(1, plan.seal, sc.cache, sc.pool, 0)  # no plan
    good = dict(cu_q=cu, cached_len=cached, page_table=t8, open_table=t16)
    make = lambda **k: plan.plan(sc.cache, sc.pool, **{**good, **k})  # noqa: E731
    make()
    free8 = max(sc.cache.num_pages, 0)
    bad = t8.copy()
    bad[0, 0] = free8
    refused(3, make, page_table=bad)
    bad = t8.copy()
    bad[1, 1] = t8[0, 1]
    refused(1, make, page_table=bad)       # sealed twice
    bad = t8.copy()
    bad[1, 0] = t8[0, 1]
    refused(1, make, page_table=bad)       # sealed and seen as an earlier page
    bad = t16.copy()
    bad[0, 1] = sc.pool.num_pages
    refused(3, make, open_table=bad)
    bad = t16.copy()
    bad[0, 1] = bad[0, 0]
    refused(1, make, open_table=np.repeat(bad[:, :1], 2, 1), cu_q=[0, 31, 32], cached_len=[1, 31])  # one slot twice
    refused(3, make, open_table=t16[:, :1])
    refused(3, make, page_table=t8[:, :1])
    refused(1, make, cached_len=[-1, 31])
    refused(1, make, cu_q=[0, 0, 14])
    refused(1, make, cu_q=[1, 13, 14])
    refused(4, make, cached_len=[20, 4000])
    refused(4, plan.plan, sc.cache, sc.pool, [0, 33], [0], np.zeros((1, 2), int), np.zeros((1, 3), int))
    refused(3, make, token_ids=np.full(14, 512))
    refused(3, make, logit_rows=[14])
    refused(1, plan.plan, other.cache, sc.pool, **good)
    refused(1, plan.plan, sc.cache, other.pool, **good)
    # the plan before is still in force
    out = torch.full_like(q, float("nan"))
    plan.seal(sc.cache, sc.pool, 0)
    plan.attention(sc.cache, sc.pool, 0, q, out)
    torch.cuda.synchronize()
    assert out.isfinite().all()
    refused(3, plan.attention, sc.cache, sc.pool, 2, q, out)
    refused(3, plan.seal, sc.cache, sc.pool, -1)
    refused(1, plan.attention, sc.cache, sc.pool, 0, q[:13], out)
    refused(1, plan.attention, sc.cache, sc.pool, 0, q.float(), out)
    refused(1, plan.attention, other.cache, sc.pool, 0, q, out)
    refused(1, plan.step, sc.cache, sc.pool)  # no token ids
    cache2 = vd.KV8Cache(sc.model, sc.cache.num_pages, "int8")
    refused(1, plan.attention, cache2, sc.pool, 0, q, out)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        refused(2, plan.attention, sc.cache, sc.pool, 0, q, out, stream=s)
        refused(2, make, stream=s)
        sc.cache.copy_pages([0], [1], stream=s)  # (something to capture; page copies may be)
    # seal and unseal
    n8, n16 = sc.cache.num_pages, sc.pool.num_pages
    refused(3, sc.cache.seal, sc.pool, [n16], [0])
    refused(3, sc.cache.seal, sc.pool, [0], [n8])
    refused(3, sc.cache.seal, sc.pool, [-1], [0])
    refused(1, sc.cache.seal, sc.pool, [0, 1], [2, 2])
    refused(1, sc.cache.seal, sc.pool, [0, 1], [2])
    refused(3, sc.cache.seal, sc.pool, [0], [0], layer=2)
    refused(3, sc.cache.unseal, sc.pool, [n8], [0])
    refused(3, sc.cache.unseal, sc.pool, [0], [n16])
    refused(1, sc.cache.unseal, sc.pool, [0, 1], [1, 1])
    refused(1, sc.cache.seal, other.pool, [0], [0])
    refused(1, vd.KV8Cache, sc.model, 0)
    refused(1, vd.KV8Cache, sc.model, 4, "int4")
    refused(4, vd.KV8Cache, sc.model, 4, "int8", memory=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    refused(4, vd.KV8Plan, sc.model, 65)
    refused(1, vd.KV8Plan, sc.model, 0)
    refused(1, plan.set_prefill, 3)
    refused(1, plan.set_prefill, -1)
    # a plan without work
    plan.plan(sc.cache, sc.pool, [0], [], np.zeros((0, 0)), np.zeros((0, 0)))
    plan.seal(sc.cache, sc.pool, 0)
    plan.attention(sc.cache, sc.pool, 0, q[:0], out[:0])
    plan.step(sc.cache, sc.pool)
    plan.close()
    refused(1, plan.seal, sc.cache, sc.pool, 0)
    assert sc.model.device_status() == 0
