"""Workloads of the 8-bit KV cache: attention over it, sealing pages into it and
opening them again, and moving pages of either cache.

Every case runs either as elementary torch operations (``own`` false: float32,
rounded once at the end) or as the calls a program makes of this framework
(``own`` true).  ``exact`` gives the results in float64 from the definitions.

The cache.  A page holds 16 tokens.  Complete pages are held in 8 bits: per
page, K or V and KV head, a = max |x| (at least 2^-80) and the codes are
round(127 x / a) in int8 or 448 x / a in e4m3, standing for code * a / 127 or
code * a / 448.  A row at position p sees the page of its own position in bf16
and every earlier page in 8 bits.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
TOP = {"int8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -80


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One interactive request's next token (Llama-3.1-8B heads).
        {"name": "attend-one", "op": "attend", "B": 1, "n": 1, "ctx_lo": 1000, "ctx_hi": 1000, "Hq": 32, "Hkv": 8,
         "hd": 128, "window": 0, "format": "int8"},
        # The decode benchmark's batch over its contexts: the largest decode step.
        {"name": "attend-decode-256", "op": "attend", "B": 256, "n": 1, "ctx_lo": 512, "ctx_hi": 8192, "Hq": 32,
         "Hkv": 8, "hd": 128, "window": 0, "format": "int8"},
        # A quarter of it, in e4m3.
        {"name": "attend-decode-64-e4m3", "op": "attend", "B": 64, "n": 1, "ctx_lo": 512, "ctx_hi": 8192, "Hq": 32,
         "Hkv": 8, "hd": 128, "window": 0, "format": "e4m3"},
        # A local layer of the Gemma-3-4B shape (head dimension 256, window 1024): requests that verify 3 drafted
        # tokens each, odd contexts.
        {"name": "attend-local-window", "op": "attend", "B": 48, "n": 3, "ctx_lo": 100, "ctx_hi": 4001, "Hq": 8,
         "Hkv": 4, "hd": 256, "window": 1024, "format": "e4m3"},
        # A chunk of a long prompt behind what is cached of it.
        {"name": "attend-prefill-2048", "op": "attend", "B": 1, "n": 2048, "ctx_lo": 6144, "ctx_hi": 6144, "Hq": 32,
         "Hkv": 8, "hd": 128, "window": 0, "format": "int8"},
        # Odd chunks of several prompts, the tiny model's head dimension, one head each for K and V and query.
        {"name": "attend-chunks-odd", "op": "attend", "B": 9, "n": 77, "ctx_lo": 3, "ctx_hi": 2500, "Hq": 8, "Hkv": 8,
         "hd": 64, "window": 0, "format": "e4m3"},
        # Pages that a decode step of 256 requests completes, all layers, and their way back.
        {"name": "seal-step", "op": "seal", "pages": 16, "layers": 32, "Hkv": 8, "hd": 128, "format": "int8"},
        # Pages of an 8192-token prompt, all layers.
        {"name": "seal-prompt", "op": "seal", "pages": 512, "layers": 32, "Hkv": 8, "hd": 128, "format": "e4m3"},
        # One conversation forked into four: copies of the page that it is filling, in the bf16 pool.
        {"name": "copy-fork", "op": "copy", "pages": 3, "of": 64, "layers": 32, "Hkv": 8, "hd": 128, "cache": "bf16"},
        # Pages moved into the holes that finished requests have left in the 8-bit cache.
        {"name": "copy-compact-8bit", "op": "copy", "pages": 700, "of": 2000, "layers": 32, "Hkv": 8, "hd": 128,
         "cache": "int8"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "seal", "copy"])
    if op == "attend":
        Hq, Hkv, hd = rng.choice([(32, 8, 128), (8, 4, 256), (4, 2, 64), (16, 1, 128), (8, 8, 64), (12, 4, 128)])
        case = {"op": op, "Hq": Hq, "Hkv": Hkv, "hd": hd, "window": rng.choice([0, 0, 0, _log_int(rng, 1, 2048)]),
                "format": rng.choice(sorted(TOP))}
        decode = rng.random() < 0.6
        hi = _log_int(rng, 1, 8192 if decode else 6144)
        case["ctx_lo"], case["ctx_hi"] = rng.randrange(max(1, hi // 16)), hi
        if decode:
            return {**case, "B": _log_int(rng, 1, 256), "n": rng.choice([1, 1, 1, 2, 3, 4])}
        n = _log_int(rng, 5, 2048)
        return {**case, "n": n, "B": max(1, min(_log_int(rng, 1, 32), 2048 // n))}
    layers, Hkv, hd = _log_int(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    most = 32 * 8 * 128 // (layers * Hkv * hd)  # as many bytes as the listed cases at most
    if op == "seal":
        return {"op": op, "pages": _log_int(rng, 1, min(512 * max(1, most), 2000)) if most else _log_int(rng, 1, 256),
                "layers": layers, "Hkv": Hkv, "hd": hd, "format": rng.choice(sorted(TOP))}
    pages = _log_int(rng, 1, 700 if most else 300)
    return {"op": op, "pages": pages, "of": 2 * pages + rng.randrange(0, 200), "layers": layers, "Hkv": Hkv, "hd": hd,
            "cache": rng.choice(["bf16", "int8"])}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    return {"attend": _prepare_attend, "seal": _prepare_seal, "copy": _prepare_copy}[case["op"]](case, seed)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pages(g, shape):
    """bf16 pages [...][2][Hkv][16][hd]: normal values, channels of unequal size, tokens of unequal size in V."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    channel = torch.randn((2, *shape[-3:-2], 1, shape[-1]), generator=g, device="cuda").mul_(0.4).exp_()
    x.mul_(channel.bfloat16())
    token = torch.rand((16, 1), generator=g, device="cuda") + 0.5
    x[..., 1, :, :, :].mul_(token.bfloat16())
    return x


def _attend_inputs(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    B, n, Hkv, hd = case["B"], case["n"], case["Hkv"], case["hd"]
    cached = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B).astype(np.int32)
    count = (cached + n + PAGE - 1) // PAGE  # logical pages of each request
    full = (cached + n) // PAGE              # those that are complete after the step
    P, width = int(count.sum()), int(count.max())
    order, k = rng.permutation(P).astype(np.int32), 0
    table = np.zeros((B, width), np.int32)   # page of `values` that holds a request's logical page
    for b in range(B):
        table[b, :count[b]] = order[k:k + count[b]]
        k += count[b]
    first = cached // PAGE                   # the pages from here on are still in bf16
    open_width = int((count - first).max())
    open_table, at = np.zeros((B, open_width), np.int32), 0
    opened = []
    for b in range(B):
        m = count[b] - first[b]
        open_table[b, :m] = np.arange(at, at + m)
        opened.append(table[b, first[b]:count[b]])
        at += m
    values = _pages(g, (P, 2, Hkv, PAGE, hd))
    return {"case": case, "cached": cached, "full": full, "table": table, "open_table": open_table, "values": values,
            "open": values[torch.from_numpy(np.concatenate(opened)).cuda().long()],
            "q": torch.randn((B * n, case["Hq"], hd), generator=g, device="cuda").bfloat16()}


def _spec(layers, Hq, Hkv, hd, window=0):
    from invariant_vd_step_gb300 import synth
    return synth.ModelSpec("kv8", layers, 128, Hq, Hkv, hd, 128, 128, sliding_window=window,
                           local_global_period=layers + 1 if window else 0)


def _model(layers, Hq, Hkv, hd, window=0, tokens=16, seqs=1, context=16):
    from invariant_vd_step_gb300 import synth, vd
    spec = _spec(layers, Hq, Hkv, hd, window)
    return vd.Model(spec, synth.make_weights(spec, device="cuda"), max_tokens=tokens, max_seqs=seqs, max_logit_rows=1,
                    max_context=context)


def _pool(model, values):
    """The framework's bf16 pool with the pages `values` [layers][pages][2][Hkv][16][hd]."""
    from invariant_vd_step_gb300 import vd
    pool = vd.KVPool(model, values.shape[1], memory=torch.empty(values.nbytes, dtype=torch.uint8, device="cuda"))
    pool.view().copy_(values)
    return pool


def _prepare_attend(case, seed):
    st = _attend_inputs(case, seed)
    values = st.pop("values")
    B, n = case["B"], case["n"]
    if own:
        from invariant_vd_step_gb300 import vd
        context = int(st["cached"].max()) + n
        st["model"] = _model(1, case["Hq"], case["Hkv"], case["hd"], case["window"], B * n, B, context)
        source = _pool(st["model"], values[None])
        st["cache"] = vd.KV8Cache(st["model"], values.shape[0], case["format"])
        done = np.concatenate([st["table"][b, :st["full"][b]] for b in range(B)])
        st["cache"].seal(source, done, done)
        torch.cuda.synchronize()
        source.close()
        st["pool"] = _pool(st["model"], st.pop("open")[None])
        st["plan"] = vd.KV8Plan(st["model"], B * n)
        st["out"] = torch.empty_like(st["q"])
        return st
    st["codes"], st["scale"] = _quantise(values, case["format"])
    for k in ("cached", "table", "open_table"):
        st[k] = torch.from_numpy(st[k]).cuda().long()
    return st


def _quantise(x, fmt):
    """Codes and scales [...] of bf16 blocks [...][16][hd]."""
    x = x.float()
    a = x.abs().amax((-2, -1), keepdim=True).clamp(min=LEAST)
    if fmt == "int8":
        codes = ((x * 127) / a).round().to(torch.int8)
    else:
        codes = ((x * 7) / a * 64).to(torch.float8_e4m3fn)
    return codes, (a / torch.full_like(a, TOP[fmt]))[..., 0, 0]


def _prepare_seal(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    L, n, Hkv, hd = case["layers"], case["pages"], case["Hkv"], case["hd"]
    values = _pages(g, (L, n, 2, Hkv, PAGE, hd))
    st = {"case": case, "src": rng.permutation(n).astype(np.int32), "dst": rng.permutation(n).astype(np.int32)}
    if own:
        from invariant_vd_step_gb300 import vd
        st["model"] = _model(L, 2 * Hkv, Hkv, hd)
        st["pool"] = _pool(st["model"], values)
        st["back"] = _pool(st["model"], torch.zeros_like(values))
        st["cache"] = vd.KV8Cache(st["model"], n, case["format"])
        return st
    st["pool"], st["back"] = values, torch.zeros_like(values)
    st["src"], st["dst"] = (torch.from_numpy(st[k]).cuda().long() for k in ("src", "dst"))
    return st


def _prepare_copy(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    L, N, Hkv, hd = case["layers"], case["of"], case["Hkv"], case["hd"]
    order = rng.permutation(N).astype(np.int32)
    st = {"case": case, "src": order[:case["pages"]].copy(), "dst": order[case["pages"]:2 * case["pages"]].copy()}
    if case["cache"] == "bf16":
        values = _pages(g, (L, N, 2, Hkv, PAGE, hd))
        if own:
            st["model"] = _model(L, 2 * Hkv, Hkv, hd)
            st["pool"] = _pool(st["model"], values)
        else:
            st["pool"] = values
    else:
        codes = torch.randint(0, 256, (L, N, Hkv, 2 * PAGE * hd), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.rand((L, N, Hkv, 4), generator=g, device="cuda") + 0.01
        if own:
            from invariant_vd_step_gb300 import vd
            st["model"] = _model(L, 2 * Hkv, Hkv, hd)
            memory = torch.empty(st["model"].kv8_bytes(N), dtype=torch.uint8, device="cuda")
            st["cache"] = vd.KV8Cache(st["model"], N, "int8", memory=memory)
            st["cache"].codes().copy_(codes)
            st["cache"].scales().copy_(scales)
        else:
            st["codes"], st["scales"] = codes, scales
    if not own:
        st["src"], st["dst"] = (torch.from_numpy(st[k]).cuda().long() for k in ("src", "dst"))
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        if op == "attend":
            # Histories grow with every step, so a program plans each step anew: the plan is part of the pass.
            B, n = st["case"]["B"], st["case"]["n"]
            st["plan"].plan(st["cache"], st["pool"], np.arange(0, B * n + 1, n), st["cached"], st["table"],
                            st["open_table"])
            st["plan"].attention(st["cache"], st["pool"], 0, st["q"], st["out"])
            return st["out"]
        if op == "seal":
            st["cache"].seal(st["pool"], st["src"], st["dst"])
            st["cache"].unseal(st["back"], st["dst"], st["src"])
            return st["back"].view()
        if st["case"]["cache"] == "bf16":
            st["pool"].copy_pages(st["src"], st["dst"])
            return st["pool"].view()
        st["cache"].copy_pages(st["src"], st["dst"])
        return {"codes": st["cache"].codes(), "scales": st["cache"].scales()}
    return {"attend": _attend, "seal": _seal, "copy": _copy}[op](st)


def _attend(st):
    case = st["case"]
    B, n, Hq, Hkv, hd = case["B"], case["n"], case["Hq"], case["Hkv"], case["hd"]
    q = st["q"].view(B, n, Hkv, Hq // Hkv, hd).float()
    pos = st["cached"][:, None] + torch.arange(n, device="cuda")           # [B][n]
    lo = (pos - case["window"] + 1).clamp(min=0) if case["window"] else torch.zeros_like(pos)
    start = pos // PAGE * PAGE                                             # first position of the row's own page
    # the sealed pages, every row up to its own page
    table = st["table"]
    kv = st["codes"][table].float() * st["scale"][table][..., None, None]   # [B][W][2][Hkv][16][hd]
    s8 = torch.einsum("bnhgd,bwhtd->bnhgwt", q, kv[:, :, 0]).flatten(-2)
    at = torch.arange(table.shape[1] * PAGE, device="cuda")
    see8 = (at < start[..., None]) & (at >= lo[..., None])                 # [B][n][W * 16]
    # each row's own page
    page = st["open_table"].gather(1, pos // PAGE - st["cached"][:, None] // PAGE)
    mine = st["open"][page].float()                                        # [B][n][2][Hkv][16][hd]
    s16 = torch.einsum("bnhgd,bnhtd->bnhgt", q, mine[:, :, 0])
    at = start[..., None] + torch.arange(PAGE, device="cuda")
    see16 = (at <= pos[..., None]) & (at >= lo[..., None])
    s = torch.cat([s8, s16], -1) / math.sqrt(hd)
    s = s.masked_fill(~torch.cat([see8, see16], -1)[:, :, None, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True)).exp()
    p = p / p.sum(-1, keepdim=True)
    W = s8.shape[-1]
    o = torch.einsum("bnhgwt,bwhtd->bnhgd", p[..., :W].unflatten(-1, (-1, PAGE)), kv[:, :, 1]) + \
        torch.einsum("bnhgt,bnhtd->bnhgd", p[..., W:], mine[:, :, 1])
    return o.reshape(B * n, Hq, hd).bfloat16()


def _seal(st):
    codes, scale = _quantise(st["pool"][:, st["src"]], st["case"]["format"])
    st["back"][:, st["src"]] = (codes.float() * scale[..., None, None]).bfloat16()
    return st["back"]


def _copy(st):
    if st["case"]["cache"] == "bf16":
        st["pool"][:, st["dst"]] = st["pool"][:, st["src"]]
        return st["pool"]
    for x in (st["codes"], st["scales"]):
        x[:, st["dst"]] = x[:, st["src"]]
    return {"codes": st["codes"], "scales": st["scales"]}


# ---------------------------------------------------------------- work
def work(case):
    if case["op"] == "attend":
        B, n, Hq, Hkv, hd = case["B"], case["n"], case["Hq"], case["Hkv"], case["hd"]
        c = (case["ctx_lo"] + case["ctx_hi"]) / 2
        w = case["window"] or 1 << 30
        sealed = min(c + n, w + n) // PAGE  # pages that some row of a request sees in 8 bits, and in bf16
        opened = (n + PAGE - 1) // PAGE
        keys = min(c + n / 2, w)
        return {"bytes": int(B * Hkv * (sealed * (2 * PAGE * hd + 8) + opened * 4 * PAGE * hd) + 4 * B * n * Hq * hd),
                "flops": int(4 * B * n * Hq * hd * keys)}
    block = case["layers"] * case["pages"] * case["Hkv"] * 2 * PAGE * case["hd"]  # values moved
    if case["op"] == "seal":
        return {"bytes": 6 * block, "flops": 4 * block}
    return {"bytes": block * (4 if case["cache"] == "bf16" else 2), "flops": 0}


# ---------------------------------------------------------------- float64
def exact(case, seed):
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    if case["op"] == "seal":
        return _exact_seal(case, seed)
    return None  # bytes moved, nothing computed


def _exact_values(x, fmt):
    """What 8-bit blocks [...][16][hd] stand for, by the definition."""
    a = x.double().abs().flatten(-2).max(-1).values.clamp(min=LEAST)[..., None, None]
    if fmt == "int8":
        return torch.round(x.double() * 127 / a) * a / 127
    y = x.double() * 448 / a
    # e4m3: four significant bits, steps of 2^-9 below 2^-6
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step * a / 448


def _exact_attend(case, seed):
    st = _attend_inputs(case, seed)
    B, n, Hq, Hkv, hd = case["B"], case["n"], case["Hq"], case["Hkv"], case["hd"]
    G, outs = Hq // Hkv, []
    for b in range(B):
        c = int(st["cached"][b])
        count = (c + n + PAGE - 1) // PAGE
        raw = st["values"][torch.from_numpy(st["table"][b, :count]).cuda().long()]     # [W][2][Hkv][16][hd]
        lay = lambda x: x.permute(1, 2, 0, 3, 4).reshape(2, Hkv, count * PAGE, hd)      # noqa: E731
        k8, v8 = lay(_exact_values(raw, case["format"]))
        k16, v16 = lay(raw.double())
        p = torch.arange(c, c + n, device="cuda")[:, None]
        j = torch.arange(count * PAGE, device="cuda")[None]
        lo = p - case["window"] + 1 if case["window"] else torch.zeros_like(p)
        mine = (j // PAGE == p // PAGE).repeat_interleave(G, 0)                          # rows: token, head of the group
        see = ((j <= p) & (j >= lo)).repeat_interleave(G, 0)
        q = st["q"][b * n:(b + 1) * n].double().view(n, Hkv, G, hd).transpose(0, 1).reshape(Hkv, n * G, hd)
        s = torch.where(mine, q @ k16.mT, q @ k8.mT) * hd ** -0.5
        w = torch.softmax(s.masked_fill(~see, -math.inf), -1)
        del s
        o = torch.where(mine, w, 0.0) @ v16 + torch.where(mine, 0.0, w) @ v8
        outs.append(o.view(Hkv, n, G, hd).transpose(0, 1).reshape(n, Hq, hd))
    return torch.cat(outs)


def _exact_seal(case, seed):
    values = _pages(_generator(seed), (case["layers"], case["pages"], 2, case["Hkv"], PAGE, case["hd"]))
    return torch.stack([_exact_values(x, case["format"]) for x in values])
