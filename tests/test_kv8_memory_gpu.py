"""Device memory that plans over the 8-bit cache take, and rows that do not depend on it."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import synth, vd
from kv8_scenario import KV8Scenario, kv8_spec

pytestmark = pytest.mark.gpu

MB = 1 << 20


def taken(f):
    """Device memory that f's work takes and keeps, in bytes."""
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    f()
    torch.cuda.synchronize()
    return before - torch.cuda.mem_get_info()[0]


def test_partials_are_those_of_the_merged_tokens():
    """A single token before, behind and between long chunks, whose last blocks alone leave partials: the same bits in every
    order, and memory for few of the tokens."""
    ready()
    Hq, hd = 32, 64
    sc = KV8Scenario(kv8_spec(Hq, 8, hd), [32000, 5000, 700], "int8", seed=2, max_tokens=2500)
    long, one, mid = (0, 29952, 2048), (1, 4999, 1), (2, 300, 400)
    want = {r: bits(sc.attention([r], kernel=1)) for r in (long, one, mid)}
    for reqs in ([one, long, mid], [long, one], [one, long], [long, mid, one], [mid, one, long]):
        cu, cached, t8, t16, _ = sc.setup(reqs)
        q = torch.cat([sc.q[rid][c:c + n] for rid, c, n in reqs])
        out = torch.full_like(q, float("nan"))
        plan = vd.KV8Plan(sc.model, len(q))
        plan.set_prefill(2)
        used = taken(lambda: plan.plan(sc.cache, sc.pool, cu, cached, t8, t16))
        plan.seal(sc.cache, sc.pool, 0)
        plan.attention(sc.cache, sc.pool, 0, q, out)
        torch.cuda.synchronize()
        for i, r in enumerate(reqs):
            np.testing.assert_array_equal(bits(out[cu[i]:cu[i + 1]]), want[r], err_msg=f"{reqs} {r}")
        # Partials of all tokens are 2049 x 32 x 63 splits x 66 floats, 1040 MB; of the last partial round of row blocks,
        # at most an eighth of the chunks' 76 x 8 and less than one round of SMs, a quarter of that.  Images of the
        # histories: (32000 + 700) / 128 chunks and two more each, 8 heads, 33 KB: 69 MB.
        assert used < 400 * MB, (reqs, used / MB)
        plan.close()
    assert sc.model.device_status() == 0


def test_images_of_long_histories_are_bounded():
    """Chunks of 64 requests that share a history of 32768 tokens: its fp16 images for each, 275 MB, would be 17.6 GB.  The
    plan takes 8 GiB at most, and leaves the other requests to the kernel that needs none: the same bits."""
    ready()
    Hq, Hkv, hd, c, n, B = 128, 16, 128, 32768, 15, 64
    spec = kv8_spec(Hq, Hkv, hd)
    W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=0).items()}
    model = vd.Model(spec, W, max_tokens=B * n, max_seqs=B, max_logit_rows=1, max_context=c + n)
    g = torch.Generator(device="cuda").manual_seed(5)
    made = lambda pages: vd.KVPool(model, pages, memory=torch.zeros(model.pool_bytes(pages), dtype=torch.uint8,  # noqa: E731
                                                                    device="cuda"))
    cache, staging, pool = vd.KV8Cache(model, c // 16, "int8"), made(c // 16), made(B)
    staging.view().normal_(generator=g)
    order = np.random.default_rng(1).permutation(c // 16).astype(np.int32)
    cache.seal(staging, np.arange(c // 16), order)
    pool.view()[:] = torch.randn((1, 1, 2, Hkv, 16, hd), generator=g, device="cuda").bfloat16()
    q1 = torch.randn((n, Hq, hd), generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()

    def run(b, kernel):
        plan, q = vd.KV8Plan(model, b * n), q1.repeat(b, 1, 1)
        out = torch.full_like(q, float("nan"))
        plan.set_prefill(kernel)
        used = taken(lambda: plan.plan(cache, pool, np.arange(0, b * n + 1, n), np.full(b, c), np.tile(order, (b, 1)),
                                       np.arange(b)[:, None]))
        plan.attention(cache, pool, 0, q, out)
        torch.cuda.synchronize()
        plan.close()
        return out, used
    want, _ = run(1, 1)
    out, used = run(B, 0)
    np.testing.assert_array_equal(bits(out), np.tile(bits(want), (B, 1, 1)))
    # partials of at most all tokens: 960 x 128 x 65 splits x 130 floats, 4.2 GB
    assert 4096 * MB < used < (8192 + 4000) * MB, used / MB
    assert model.device_status() == 0


def test_a_little_more_takes_a_little_more():
    """Plans that grow by a hundredth: their memory grows by that and 64 MB at most per buffer, not by half."""
    ready()
    sc = KV8Scenario(kv8_spec(32, 8, 64), [32000], "int8", seed=2, max_tokens=1100)
    plan = vd.KV8Plan(sc.model, 1100)
    plan.set_prefill(1)
    for n, most in ((1000, 600), (1010, 80), (1011, 1)):
        cu, cached, t8, t16, _ = sc.setup([(0, 30000, n)])
        q = sc.q[0][30000:30000 + n]
        used = taken(lambda: plan.plan(sc.cache, sc.pool, cu, cached, t8, t16))
        # 1000 tokens x 32 heads x 61 splits x 66 floats: 515 MB, a hundredth of it 5
        assert used <= most * MB, (n, used / MB)
    plan.seal(sc.cache, sc.pool, 0)
    out = torch.full_like(q, float("nan"))
    plan.attention(sc.cache, sc.pool, 0, q, out)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(bits(out), bits(sc.attention([(0, 30000, 1011)])))
