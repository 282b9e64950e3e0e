"""The 8-bit cache where sizes and offsets are large, calls run at once or are captured, and buffers overlap."""

import threading

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import vd
from kv8_scenario import KV8Scenario, e4m3, kv8_spec, sealed_values
from test_kv8_gpu import _decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", [1, 2])
def test_pages_behind_four_gigabytes(kernel):
    """The same rows from pages at the end of a cache and a pool of more than 2^32 bytes."""
    ready()
    Hkv, hd = 4, 128
    sc = KV8Scenario(kv8_spec(8, Hkv, hd), [700, 400], "int8", seed=3)
    reqs = [(0, 600, 60), (1, 333, 1)]
    want = bits(sc.attention(reqs, kernel=kernel))
    cu, cached, t8, t16, _ = sc.setup(reqs)
    N8, N16 = 2 ** 32 // (32 * hd * Hkv) + 100, 2 ** 32 // (64 * hd * Hkv) + 100
    cache = vd.KV8Cache(sc.model, N8, "int8", memory=torch.empty(sc.model.kv8_bytes(N8), dtype=torch.uint8, device="cuda"))
    pool = vd.KVPool(sc.model, N16, memory=torch.zeros(sc.model.pool_bytes(N16), dtype=torch.uint8, device="cuda"))
    near8, near16 = np.arange(sc.cache.num_pages), np.arange(sc.pool.num_pages)
    for (rid, c, _), row in zip(reqs, t8):
        pool.view()[:, :c // 16] = sc.kv[rid][:c // 16]
        cache.seal(pool, np.arange(c // 16), row[:c // 16])
    cache.copy_pages(near8, N8 - 1 - near8)
    cache.scales()[:, :sc.cache.num_pages] = float("nan")
    pool.view()[:, :sc.pool.num_pages] = sc.pool.view()
    pool.copy_pages(near16, N16 - 1 - near16)
    pool.view()[:, :100] = float("nan")
    plan = vd.KV8Plan(sc.model, 61)
    plan.set_prefill(kernel)
    plan.plan(cache, pool, cu, cached, N8 - 1 - np.maximum(t8, 0), N16 - 1 - np.maximum(t16, 0))
    plan.seal(cache, pool, 0)
    q = torch.cat([sc.q[0][600:660], sc.q[1][333:334]])
    out = torch.full_like(q, float("nan"))
    plan.attention(cache, pool, 0, q, out)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(out), want)
    # and back: a page that the step sealed, opened into the pool's last page
    cache.unseal(pool, [N8 - 1 - t8[0, 600 // 16]], [N16 - 1])
    torch.cuda.synchronize()
    assert torch.equal(pool.view()[0, -1], sealed_values(sc.kv[0][600 // 16], "int8").bfloat16())
    assert sc.model.device_status() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_a_long_history(fmt):
    """70000 tokens, 137 splits: a chunk on either kernel, and its last row as a single token, against 64 bits."""
    ready()
    n = 70000
    sc = KV8Scenario(kv8_spec(4, 1, 64), [n], fmt, seed=4, max_tokens=128)
    got = [sc.attention([(0, n - 100, 100)], kernel=k) for k in (1, 2)]
    np.testing.assert_array_equal(bits(got[0]), bits(got[1]))
    np.testing.assert_array_equal(bits(sc.attention([(0, n - 1, 1)])), bits(got[0])[-1:])
    want, tol = sc.exact(0, n - 100, 100)
    assert ((got[0].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("hd", [64, 128, 256])
@pytest.mark.parametrize("end", [513, 545, 640, 641, 1024, 1025, 1153])
def test_ends_behind_a_split(end, hd):
    """Chunks whose last keys begin a split: two ends of splits follow each other."""
    ready()
    sc = KV8Scenario(kv8_spec(4, 2, hd), [end], "e4m3", seed=end, max_tokens=512)
    got = [bits(sc.attention([(0, end - 150, 150)], kernel=k)) for k in (1, 2)]
    np.testing.assert_array_equal(got[0], got[1])
    # among enough blocks that most fold their splits themselves
    many = [(0, end - 150, 150)] * 3
    sc = KV8Scenario(kv8_spec(128, 64, hd), [end], "e4m3", seed=end, max_tokens=512)
    got = [bits(sc.attention(many, kernel=k)) for k in (1, 2)]
    np.testing.assert_array_equal(got[0], got[1])
    np.testing.assert_array_equal(got[0][:150], got[0][300:])


def test_overlapping_queries_and_outputs_are_refused():
    ready()
    sc = KV8Scenario(kv8_spec(4, 2, 64), [200], "int8")
    cu, cached, t8, t16, _ = sc.setup([(0, 100, 100)])
    plan = vd.KV8Plan(sc.model, 100)
    plan.plan(sc.cache, sc.pool, cu, cached, t8, t16)
    plan.seal(sc.cache, sc.pool, 0)
    room = torch.zeros((201, 4, 64), dtype=torch.bfloat16, device="cuda")
    room[:100] = sc.q[0][100:]
    for o in (0, 1, 99):
        for q, out in [(room[:100], room[o:o + 100]), (room[o:o + 100], room[:100])]:
            with pytest.raises(vd.VDError) as e:
                plan.attention(sc.cache, sc.pool, 0, q, out)
            assert e.value.code == 1
    plan.attention(sc.cache, sc.pool, 0, room[:100], room[100:200])  # neighbours
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(room[100:200]), bits(sc.attention([(0, 100, 100)])))
    assert (room[200] == 0).all()


def test_two_threads_with_plans_of_their_own():
    ready()
    sc = KV8Scenario(kv8_spec(8, 2, 128), [900, 700], "e4m3", seed=7)
    reqs = [(0, 300, 600), (1, 650, 50)]
    want = [bits(sc.attention([r])) for r in reqs]
    cu, cached, t8, t16, _ = sc.setup(reqs)
    q = [sc.q[rid][c:c + n] for rid, c, n in reqs]
    failed = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            plan = vd.KV8Plan(sc.model, len(q[i]))
            for rep in range(20):
                plan.set_prefill(rep % 3)
                plan.plan(sc.cache, sc.pool, [0, len(q[i])], cached[i:i + 1], t8[i:i + 1], t16[i:i + 1], stream=s)
                plan.seal(sc.cache, sc.pool, 0, stream=s)
                with torch.cuda.stream(s):
                    out = torch.full_like(q[i], float("nan"))
                plan.attention(sc.cache, sc.pool, 0, q[i], out, stream=s)
                s.synchronize()
                np.testing.assert_array_equal(bits(out), want[i])
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert sc.model.device_status() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_sealing_captured_and_replayed(fmt):
    """A graph holds the page ids, not the values: each replay seals what the pages hold then."""
    ready()
    sc = KV8Scenario(kv8_spec(2, 2, 64, layers=2), [16], fmt)
    pool = vd.KVPool(sc.model, 4, memory=torch.zeros(sc.model.pool_bytes(4), dtype=torch.uint8, device="cuda"))
    cache = vd.KV8Cache(sc.model, 3, fmt)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        cache.seal(pool, [0, 1], [2, 0], stream=s)
        cache.unseal(pool, [2, 0], [3, 2], layer=1, stream=s)
    for rep in range(3):
        pool.view().copy_(torch.randn(pool.view().shape, device="cuda") * 10.0 ** rep)
        before = pool.view().clone()
        g.replay()
        torch.cuda.synchronize()
        want = before.clone()
        want[1, 3], want[1, 2] = (sealed_values(before[1, i], fmt).bfloat16() for i in (0, 1))
        assert torch.equal(pool.view(), want)


def test_few_pages_of_many_are_checked():
    ready()
    sc = KV8Scenario(kv8_spec(2, 1, 64), [16], "int8")
    n = 8192
    cache = vd.KV8Cache(sc.model, n, "int8", memory=torch.empty(sc.model.kv8_bytes(n), dtype=torch.uint8, device="cuda"))
    cache.codes().copy_(torch.randint(0, 256, cache.codes().shape, device="cuda", dtype=torch.uint8))
    before = cache.codes().clone()
    for code, src, dst in [(3, [n], [0]), (3, [0], [n]), (3, [0], [-1]), (1, [0, 1, 2], [n - 1, 5, n - 1]),
                           (1, [0, 1, n - 1], [n - 1, 5, 6]), (1, [7], [7])]:
        with pytest.raises(vd.VDError) as e:
            cache.copy_pages(src, dst)
        assert e.value.code == code, (src, dst, e.value)
    torch.cuda.synchronize()
    assert torch.equal(cache.codes(), before)
    cache.copy_pages([0, 0, 1], [n - 1, 5, 6])
    before[:, [n - 1, 5, 6]] = before[:, [0, 0, 1]]
    torch.cuda.synchronize()
    assert torch.equal(cache.codes(), before)


def test_memory_that_is_not_on_the_models_device_is_refused():
    """(host memory; another GPU's takes the same check)"""
    import ctypes
    ready()
    sc = KV8Scenario(kv8_spec(2, 1, 64), [16], "int8")
    n = sc.model.kv8_bytes(4)
    host = torch.zeros(n + 256, dtype=torch.uint8).pin_memory()
    h = ctypes.c_void_p()
    at = (host.data_ptr() + 255) // 256 * 256
    assert vd.lib().vd_kv8_create(sc.model.h, 0, 4, at, n, ctypes.byref(h)) == 1 and not h.value
    with pytest.raises(vd.VDError):
        vd.KV8Cache(sc.model, 4, "int8", memory=host)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("exponent", [-78, -3, 0, 100, 127])
def test_codes_of_every_pair_of_significands(fmt, exponent):
    """Blocks whose largest magnitudes have each of bf16's 128 significands, over values that have each of them at eight
    exponents, a / 2 among them: every tie of the codes' rounding is there, and goes to the even code."""
    ready()
    sc = KV8Scenario(kv8_spec(2, 1, 64), [16], fmt)
    a = (1 + torch.arange(128, device="cuda").double() / 128)[:, None]                   # [128][1]
    x = (1 + torch.arange(128, device="cuda").double() / 128)[:, None] * 2.0 ** -torch.arange(8, device="cuda").double()
    x = x.reshape(1, -1).repeat(128, 1)                                                  # [128][1024]
    x = torch.where(x > a, a / 2, x)
    x[:, 0] = a[:, 0]
    x[:, 1::2] *= -1
    x = (x * 2.0 ** exponent).bfloat16().view(64, 2, 1, 16, 64)[None]                    # blocks: K and V of 64 pages
    pool = vd.KVPool(sc.model, 64, memory=torch.empty(x.nbytes, dtype=torch.uint8, device="cuda"))
    pool.view().copy_(x)
    cache = vd.KV8Cache(sc.model, 64, fmt, memory=torch.empty(sc.model.kv8_bytes(64), dtype=torch.uint8, device="cuda"))
    cache.seal(pool, np.arange(64), np.arange(64))
    torch.cuda.synchronize()
    codes, _ = _decode(cache, fmt)
    y = x.double()
    top = y.abs().amax((-2, -1), keepdim=True)
    assert (top.flatten() == (a * 2.0 ** exponent).flatten()).all()
    assert torch.equal(codes, torch.round(y * 127 / top) if fmt == "int8" else e4m3(y * 448 / top))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("window", [0, 1, 300])
def test_long_chunks_at_head_dimension_256(window, fmt):
    """Two CTAs share a row block there: against 64 bits, the mma.sync kernel and single tokens; with and without blocks that
    fold their own splits."""
    ready()
    for Hq, Hkv in ((8, 4), (48, 24)):
        sc = KV8Scenario(kv8_spec(Hq, Hkv, 256, window), [1100, 37], fmt, seed=6, max_tokens=900)
        reqs = [(0, 333, 767), (1, 0, 37), (1, 36, 1)]
        got = sc.attention(reqs, kernel=2)
        np.testing.assert_array_equal(bits(sc.attention(reqs, kernel=1)), bits(got))
        for c in (333, 511, 512, 800, 1099):
            np.testing.assert_array_equal(bits(sc.attention([(0, c, 1)]))[0], bits(got)[c - 333], err_msg=str(c))
        for rid, c, n, at in ((0, 333, 767, 0), (1, 0, 37, 767)):
            want, tol = sc.exact(rid, c, n, window)
            assert ((got[at:at + n].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["inf", "nan"])
@pytest.mark.parametrize("hd", [128, 256])
def test_values_that_are_not_finite_in_long_chunks(kind, hd):
    """One K value of a sealed page, then one of the chunk's own tokens: both kernels give the same bits, NaN where a row sees
    it and what they gave without it before."""
    ready()
    bad = float(kind)
    base = KV8Scenario(kv8_spec(4, 2, hd), [700], "int8", seed=9)
    clean = bits(base.attention([(0, 300, 400)], kernel=2))
    for page, token in ((10, 3), (20, 15)):  # sealed before; own and sealed by the step
        def edit(s):
            s.kv[0][page, 0, :, token, 5] = bad
        sc = KV8Scenario(kv8_spec(4, 2, hd), [700], "int8", seed=9, edit=edit)
        got = [sc.attention([(0, 300, 400)], kernel=k) for k in (1, 2)]
        assert torch.equal(got[0].isnan(), got[1].isnan())
        first = page * 16 + token  # the first position that sees it
        seen = torch.arange(300, 700, device="cuda") >= first
        assert got[1][seen].isnan().all()
        for g in got:
            np.testing.assert_array_equal(bits(g)[(~seen).cpu().numpy()], clean[(~seen).cpu().numpy()])
