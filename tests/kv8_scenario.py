"""Scenarios of the 8-bit cache: requests with seeded K/V and queries, laid out for any split into cached and new
tokens, and attention over them in 64 bits (no test functions here)."""

import numpy as np
import torch

from invariant_vd_step_gb300 import synth, vd

LEAST = 2.0 ** -80


def kv8_spec(Hq, Hkv, hd, window=0, layers=1):
    return synth.ModelSpec(f"kv8-{Hq}-{Hkv}-{hd}", layers, 256, Hq, Hkv, hd, 256, 512, sliding_window=window,
                           local_global_period=layers + 1 if window else 0)


def e4m3(y):
    """y rounded to e4m3 (64 bits; |y| <= 448): four significant bits, steps of 2^-9 below 2^-6, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def sealed_values(x, fmt):
    """What sealed blocks [...][16][hd] stand for, in 64 bits; NaN where a block holds an infinity or NaN."""
    x = x.double()
    a = x.abs().amax((-2, -1), keepdim=True).clamp(min=LEAST)
    v = torch.round(x * 127 / a) * a / 127 if fmt == "int8" else e4m3(x * 448 / a) * a / 448
    return torch.where(x.isfinite().all(-1, keepdim=True).all(-2, keepdim=True), v, float("nan"))


class KV8Scenario:
    """lens: history length of each request.  kv [rid] is bf16 [pages][2][Hkv][16][hd], q [rid] bf16 [len][Hq][hd]."""

    def __init__(self, spec, lens, fmt, seed=0, max_tokens=None, edit=None, layers=1, q_scale=1.0):
        self.spec, self.lens, self.fmt = spec, lens, fmt
        T = max_tokens or max(sum(lens), 16)
        W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=seed).items()}
        self.model = vd.Model(spec, W, max_tokens=T, max_seqs=max(len(lens), 1) * 4, max_logit_rows=8,
                              max_context=max(lens) + 16)
        g = torch.Generator().manual_seed(seed + 1)
        self.kv, self.q = [], []
        for n in lens:
            np_ = (n + 15) // 16
            kv = torch.randn((np_, 2, spec.n_kv_heads, 16, spec.head_dim), generator=g)
            kv *= torch.exp(0.5 * torch.randn((np_, 2, spec.n_kv_heads, 1, 1), generator=g))  # blocks of unequal size
            self.kv.append(kv.bfloat16())
            self.q.append((q_scale * torch.randn((n, spec.n_heads, spec.head_dim), generator=g)).bfloat16())
        if edit:
            edit(self)
        self.kv = [x.cuda() for x in self.kv]
        self.q = [x.cuda() for x in self.q]
        self.rng = np.random.default_rng(seed + 2)

    def setup(self, reqs, scatter=True):
        """reqs: list of (rid, cached, q_len).  A cache with the complete pages below `cached` sealed, a bf16 pool with the
        pages from there on, NaN behind the new tokens, and the plan's arrays.  The new tokens' complete pages are
        not sealed yet."""
        L = self.spec.n_layers
        need8 = [(c + n) // 16 for _, c, n in reqs]
        need16 = [(c + n + 15) // 16 - c // 16 for _, c, n in reqs]
        self.cache = vd.KV8Cache(self.model, sum(need8) + 3, self.fmt)
        stage = max([c // 16 for _, c, _ in reqs] + [1])
        mem = lambda n: torch.zeros(self.model.pool_bytes(n), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.pool = vd.KVPool(self.model, sum(need16) + 3, memory=mem(sum(need16) + 3))
        staging = vd.KVPool(self.model, stage, memory=mem(stage))
        self.pool.view().fill_(float("nan"))
        p8 = self.rng.permutation(sum(need8) + 3) if scatter else np.arange(sum(need8) + 3)
        p16 = self.rng.permutation(sum(need16) + 3) if scatter else np.arange(sum(need16) + 3)
        t8 = np.full((len(reqs), max(need8 + [0])), -7, np.int32)  # what no row needs is never looked at
        t16 = np.full((len(reqs), max(need16)), -7, np.int32)
        a = b = 0
        for i, (rid, c, n) in enumerate(reqs):
            t8[i, :need8[i]] = p8[a:a + need8[i]]
            t16[i, :need16[i]] = p16[b:b + need16[i]]
            a, b = a + need8[i], b + need16[i]
            done = c // 16
            if done:
                staging.view()[:, :done] = self.kv[rid][:done]
                self.cache.seal(staging, np.arange(done), t8[i, :done])
            for j in range(need16[i]):
                have = min(16, c + n - (done + j) * 16)
                self.pool.view()[:, int(t16[i, j]), :, :, :have] = self.kv[rid][done + j][:, :, :have]
        torch.cuda.synchronize()
        cu = np.concatenate([[0], np.cumsum([n for _, _, n in reqs])]).astype(np.int32)
        return cu, np.array([c for _, c, _ in reqs], np.int32), t8, t16, L

    def attention(self, reqs, layer=0, scatter=True, kernel=0):
        cu, cached, t8, t16, _ = self.setup(reqs, scatter)
        q = torch.cat([self.q[rid][c:c + n] for rid, c, n in reqs])
        out = torch.full_like(q, float("nan"))
        self.plan = vd.KV8Plan(self.model, len(q))
        self.plan.set_prefill(kernel)
        self.plan.plan(self.cache, self.pool, cu, cached, t8, t16)
        self.plan.seal(self.cache, self.pool, layer)
        self.plan.attention(self.cache, self.pool, layer, q, out)
        torch.cuda.synchronize()
        assert self.model.device_status() == 0
        return out

    def exact(self, rid, c, n, window=0):
        """(output, tolerance) of rows c .. c + n - 1 in 64 bits.

        Tolerance, with w the softmax weights and v the values: the output's rounding to bf16, 2^-8 |o|; the weights'
        to fp16, 2^-11 w each, so 2^-11 sum w |v|, or 2^-25 of a chunk's largest w * scale, whose scale is at most max
        |v| of its page / 127, times a code of at most 448: 2^-25 * 448 / 127 < 2^-23 a per key, a = max_j w_j max |v of
        j's page|; float32 of the scores: 2^-20
        of their terms' absolute sum S (sums of up to 256 exact products, the log2 of the V scale and one more sum,
        each within 2^-23), twice as it enters the weight's numerator and their sum; and 2^-16 sum w |v| for
        exponentials (2^-22) and sums of n weighted values in float32."""
        spec = self.spec
        G, hd, Hkv = spec.n_heads // spec.n_kv_heads, spec.head_dim, spec.n_kv_heads
        kv = self.kv[rid][:(c + n + 15) // 16]
        count = kv.shape[0]
        lay = lambda x: x.permute(1, 2, 0, 3, 4).reshape(2, Hkv, count * 16, hd)  # noqa: E731
        v8, v16 = lay(sealed_values(kv, self.fmt)), lay(kv.double())
        top = lay(kv.double().abs().amax((-2, -1), keepdim=True).expand(kv.shape))[1, :, :, 0]  # [Hkv][keys]
        p = torch.arange(c, c + n, device="cuda")[:, None]
        j = torch.arange(count * 16, device="cuda")[None]
        see = (j <= p) & ((j > p - window) if window else torch.ones_like(j <= p))
        mine = (j // 16) == (p // 16)
        q = self.q[rid][c:c + n].double().view(n, Hkv, G, hd).permute(1, 2, 0, 3)  # [Hkv][G][n][hd]
        k8, k16 = v8[0][:, None], v16[0][:, None]
        s = torch.where(mine, q @ k16.mT, q @ k8.mT) * hd ** -0.5
        S = (torch.where(mine, q.abs() @ k16.abs().mT, q.abs() @ k8.abs().mT) * hd ** -0.5).masked_fill(~see, 0).amax(-1)
        w = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
        pick = lambda keep, val: torch.where(keep, w, 0.0) @ torch.where(  # noqa: E731
            (see & keep).any(0)[:, None], val, 0.0)  # values that no row sees stay out
        o = pick(mine & see, v16[1][:, None]) + pick(~mine & see, v8[1][:, None])
        A = pick(mine & see, v16[1].abs()[:, None]) + pick(~mine & see, v8[1].abs()[:, None])
        a = (w * top[:, None, None]).amax(-1)
        keys = see.sum(-1)
        tol = 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -16 + 2 * 2.0 ** -20 * (S[..., None] + 160)) * A + \
            (2.0 ** -23 * keys * a)[..., None]
        fix = lambda x: x.permute(2, 0, 1, 3).reshape(n, spec.n_heads, hd)  # noqa: E731
        return fix(o), fix(tol)
