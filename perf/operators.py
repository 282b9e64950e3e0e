"""Workloads of the speculative-decoding operators: rotary positions, attention
of a drafted token tree over the paged cache, filtered sampling and tree
acceptance.

Every case runs either as elementary torch operations (``own`` false: float32,
or float64 where float32 loses what matters, rounded once at the end) or as
the calls a program makes of this framework (``own`` true).  ``exact`` gives
the results in float64 from the definitions.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# Frequency scalings: the banded one with the published Llama-3.1 constants, YaRN and linear interpolation.
SCALINGS = {
    "none": {"type": "none"},
    "linear": {"type": "linear", "factor": 4.0},
    "bands": {"type": "bands", "factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
              "original_max_position": 8192},
    "yarn": {"type": "yarn", "factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_max_position": 4096},
}
THETA = 5e5

SAMPLER = np.dtype([("seed", "u8"), ("step", "u8"), ("temperature", "f4"), ("pad_", "f4")])
FILTER = np.dtype([("top_k", "i4"), ("top_p", "f4"), ("min_p", "f4"), ("pad_", "f4")])


# ---------------------------------------------------------------- cases
def listed():
    return [
        # Query and key heads of a 64-request decode step (Llama-3.1-8B shape), inside the fused QKV rows,
        # with the banded frequency scaling of a 131,072-token context.
        {"name": "rotary-decode-64", "op": "rotary", "T": 64, "H": 40, "row_heads": 48, "hd": 128, "rot": 128,
         "layout": "half", "scaling": "bands", "dtype": "bf16", "max_pos": 131072, "inverse": False},
        # The same for a prefill chunk of 8192 tokens.
        {"name": "rotary-prefill-8192", "op": "rotary", "T": 8192, "H": 40, "row_heads": 48, "hd": 128, "rot": 128,
         "layout": "half", "scaling": "bands", "dtype": "bf16", "max_pos": 131072, "inverse": False},
        # Undoing the rotation of a cached float32 span to re-position it: interleaved pairs over part of the
        # head, YaRN scaling, an odd number of tokens and heads.
        {"name": "rotary-part-inverse", "op": "rotary", "T": 4097, "H": 13, "row_heads": 13, "hd": 96, "rot": 64,
         "layout": "interleaved", "scaling": "yarn", "dtype": "fp32", "max_pos": 65536, "inverse": True},
        # One interactive request verifying 8 drafted tokens.
        {"name": "tree-one-request", "op": "tree", "B": 1, "N": 8, "ctx_lo": 1000, "ctx_hi": 1000, "Hq": 32,
         "Hkv": 8, "hd": 128, "window": 0},
        # A serving batch verifying 16-node trees over the contexts of the decode benchmark.
        {"name": "tree-batch-16", "op": "tree", "B": 16, "N": 16, "ctx_lo": 512, "ctx_hi": 8192, "Hq": 32, "Hkv": 8,
         "hd": 128, "window": 0},
        # Wide trees over the same contexts: the largest verification step.
        {"name": "tree-wide-64", "op": "tree", "B": 32, "N": 64, "ctx_lo": 512, "ctx_hi": 8192, "Hq": 32, "Hkv": 8,
         "hd": 128, "window": 0},
        # A local layer of the Gemma-3-4B shape (head dimension 256, window 1024), odd tree sizes and contexts.
        {"name": "tree-local-window", "op": "tree", "B": 32, "N": 13, "ctx_lo": 100, "ctx_hi": 4001, "Hq": 8,
         "Hkv": 4, "hd": 256, "window": 1024},
        # One interactive request's next token.
        {"name": "sample-one", "op": "sample", "R": 1, "V": 128256, "mix": "chat", "std": 2.0},
        # The decode benchmark's batch, each row with its own settings.
        {"name": "sample-batch-256", "op": "sample", "R": 256, "V": 128256, "mix": "mixed", "std": 2.0},
        # Wide nuclei: flat distributions at high temperature over the Gemma-3-4B shape's vocabulary.
        {"name": "sample-wide-nucleus", "op": "sample", "R": 61, "V": 262144, "mix": "wide", "std": 1.0},
        # Acceptance of one request's 8-node tree in a 32-layer cache.
        {"name": "accept-one", "op": "accept", "B": 1, "N": 8, "chain": 4, "layers": 32, "Hkv": 8, "hd": 128,
         "ctx": 520},
        # Acceptance of a batch of 32-node trees behind a shared prefix.
        {"name": "accept-batch-32", "op": "accept", "B": 32, "N": 32, "chain": 8, "layers": 32, "Hkv": 8, "hd": 128,
         "ctx": 520},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rotary", "tree", "tree", "sample", "sample", "accept"])
    if op == "rotary":
        hd = rng.choice([64, 80, 96, 128, 256])
        H = _log_int(rng, 1, 40)
        return {"op": op, "T": min(_log_int(rng, 1, 8192), 8192 * 40 * 128 * 2 // (H * hd * 4)), "H": H,
                "row_heads": H + rng.choice([0, 1, 8]), "hd": hd, "rot": rng.choice([hd, hd // 2]),
                "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(sorted(SCALINGS)),
                "dtype": rng.choice(sorted(DTYPES)), "max_pos": _log_int(rng, 8192, 1000000),
                "inverse": rng.random() < 0.3}
    if op == "tree":
        Hq, Hkv, hd = rng.choice([(32, 8, 128), (8, 4, 256), (4, 2, 64), (16, 1, 128), (8, 8, 64)])
        hi = _log_int(rng, 1, 8192)
        return {"op": op, "B": _log_int(rng, 1, 32), "N": _log_int(rng, 1, 64),
                "ctx_lo": rng.randrange(max(1, hi // 2)), "ctx_hi": hi, "Hq": Hq, "Hkv": Hkv, "hd": hd,
                "window": rng.choice([0, 0, 0, _log_int(rng, 1, 2048)])}
    if op == "sample":
        V = rng.choice([2048, 32003, 128256, 262144])
        return {"op": op, "R": min(_log_int(rng, 1, 256), 256 * 128256 // V), "V": V,
                "mix": rng.choice(["chat", "mixed", "wide"]), "std": round(rng.uniform(0.5, 4.0), 3)}
    chain = rng.randrange(1, 9)
    return {"op": op, "B": _log_int(rng, 1, 32), "N": chain + rng.randrange(0, 25), "chain": chain,
            "layers": _log_int(rng, 1, 32), "Hkv": rng.choice([1, 2, 4, 8]), "hd": rng.choice([64, 128]),
            "ctx": _log_int(rng, 16, 600)}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    return {"rotary": _prepare_rotary, "tree": _prepare_tree, "sample": _prepare_sample,
            "accept": _prepare_accept}[case["op"]](case, seed)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _frequencies(rot, scaling):
    """Angle per position of each pair (float64 numpy) and the magnitude of the rotation."""
    f = THETA ** (-2.0 * np.arange(rot // 2) / rot)
    s = SCALINGS[scaling]
    if s["type"] == "none":
        return f, 1.0
    if s["type"] == "linear":
        return f / s["factor"], 1.0
    if s["type"] == "bands":  # wavelengths short of the original context kept, long ones stretched, a ramp between
        turns = s["original_max_position"] * f / (2 * math.pi)
        keep = (turns - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
        keep = np.clip(keep, 0.0, 1.0)
        return keep * f + (1 - keep) * f / s["factor"], 1.0
    # YaRN: the ramp runs over pair indices, between the pairs that turn beta_fast and beta_slow times
    at = [rot * math.log(s["original_max_position"] / (b * 2 * math.pi)) / (2 * math.log(THETA))
          for b in (s["beta_fast"], s["beta_slow"])]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / (hi - lo if hi > lo else 0.001), 0.0, 1.0)
    return f * (1 - ramp) + f / s["factor"] * ramp, 0.1 * math.log(s["factor"]) + 1.0


def _prepare_rotary(case, seed):
    g = _generator(seed)
    T, H, hd, dt = case["T"], case["H"], case["hd"], DTYPES[case["dtype"]]
    rows = torch.randn((T, case["row_heads"], hd), generator=g, device="cuda").to(dt)
    f, mag = _frequencies(case["rot"], case["scaling"])
    st = {"case": case, "x": rows[:, :H], "y": torch.empty((T, H, hd), dtype=dt, device="cuda"), "mag": mag,
          "pos": torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda", dtype=torch.int32),
          "f": torch.from_numpy(f).cuda()}
    if own:
        from invariant_vd_step_gb300 import vd
        st["rope"] = vd.Rope(hd, rot_dim=case["rot"], layout=case["layout"], theta=THETA,
                             scaling=SCALINGS[case["scaling"]])
    return st


def _trees(rng, B, N, chain):
    """Parents [B][N] of random drafts, node 0 the root: the first `chain` nodes are the draft's best
    continuation, the others branch off earlier nodes and end no deeper than it.  And depths [B][N]."""
    parent, depth = np.full((B, N), -1, np.int32), np.zeros((B, N), np.int32)
    for b in range(B):
        for i in range(1, N):
            p = i - 1 if i < chain else int(rng.integers(0, i))
            while i >= chain and depth[b, p] >= max(chain - 1, 1):
                p = int(rng.integers(0, p + 1))
                p = 0 if chain < 2 else p
                if depth[b, p] >= max(chain - 1, 1):
                    p = max(p - 1, 0)
            parent[b, i], depth[b, i] = p, depth[b, p] + 1
    return parent, depth


def _paths(parent):
    """[B][N][N]: node j is node i or one of its ancestors."""
    B, N = parent.shape
    on = np.zeros((B, N, N), bool)
    for b in range(B):
        for i in range(N):
            if i:
                on[b, i] = on[b, parent[b, i]]
            on[b, i, i] = True
    return on


def _model(B, N, Hq, Hkv, hd, window, ctx, layers, pool):
    """The framework's model, KV pool (over the memory of `pool`, whose values it keeps) and tree handle."""
    from invariant_vd_step_gb300 import synth, vd
    spec = synth.ModelSpec("tree", layers, 128, Hq, Hkv, hd, 128, 128, rope_theta=THETA, rope_theta_local=THETA,
                           sliding_window=window, local_global_period=layers + 1 if window else 0)
    model = vd.Model(spec, synth.make_weights(spec, device="cuda"), max_tokens=B * N, max_seqs=B, max_logit_rows=1,
                     max_context=ctx + N)
    values = pool.clone()
    kv = vd.KVPool(model, pool.shape[1], memory=pool.view(torch.uint8).reshape(-1))
    pool.copy_(values)
    return model, kv, vd.Tree(model, max_nodes=B * N)


def _prepare_tree(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    B, N, Hq, Hkv, hd = case["B"], case["N"], case["Hq"], case["Hkv"], case["hd"]
    ctx = rng.integers(case["ctx_lo"], case["ctx_hi"] + 1, B).astype(np.int32)
    parent, depth = _trees(rng, B, N, max(1, N // 4))
    width = (int(ctx.max()) + N + PAGE - 1) // PAGE
    pages = [(int(c) + N + PAGE - 1) // PAGE for c in ctx]
    order, k = rng.permutation(sum(pages)), 0
    table = np.zeros((B, width), np.int32)
    for b in range(B):
        table[b, :pages[b]] = order[k:k + pages[b]]
        k += pages[b]
    pool = torch.empty((1, sum(pages), 2, Hkv, PAGE, hd), dtype=torch.bfloat16, device="cuda")
    pool.normal_(generator=g)
    st = {"case": case, "pool": pool, "q": torch.randn((B * N, Hq, hd), generator=g, device="cuda").bfloat16(),
          "out": torch.empty((B * N, Hq, hd), dtype=torch.bfloat16, device="cuda"),
          "ctx": torch.from_numpy(ctx).cuda(), "depth": torch.from_numpy(depth).cuda(),
          "path": torch.from_numpy(_paths(parent)).cuda(), "table": torch.from_numpy(table).cuda().long(),
          "width": int(ctx.max()) + N}
    if own:
        st["model"], st["kv"], st["tree"] = _model(B, N, Hq, Hkv, hd, case["window"], int(ctx.max()), 1, pool)
        st["tree"].plan(st["kv"], np.arange(0, B * N + 1, N), parent, ctx, table)
    return st


def _prepare_sample(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    R, V = case["R"], case["V"]
    logits = torch.randn((R, V), generator=g, device="cuda").mul_(case["std"])
    if case["mix"] != "wide":  # the likely continuations stand out of the bulk
        at = (torch.randint(0, V, (R, 1), generator=g, device="cuda") + 641 * torch.arange(200, device="cuda")) % V
        logits.scatter_(1, at, torch.rand((R, 200), generator=g, device="cuda") * 14 + logits.gather(1, at))
    s, f = np.zeros(R, SAMPLER), np.zeros(R, FILTER)
    s["seed"], s["step"] = rng.integers(0, 2 ** 63, R), rng.integers(0, 100000, R)
    f["top_p"] = 1.0
    if case["mix"] == "chat":
        s["temperature"], f["top_k"], f["top_p"] = 0.8, 50, 0.9
    elif case["mix"] == "wide":
        s["temperature"], f["top_p"] = rng.uniform(1.0, 1.6, R), rng.uniform(0.9, 0.99, R)
    else:  # a serving batch: one row in eight greedy, one unfiltered, the others with one, two or three filters
        kind = rng.integers(0, 8, R)
        s["temperature"] = np.where(kind == 0, 0.0, rng.uniform(0.6, 1.2, R))
        f["top_k"] = np.where((kind == 2) | (kind >= 5), rng.integers(1, 200, R), 0)
        f["top_p"] = np.where((kind == 3) | (kind >= 6), rng.uniform(0.8, 0.98, R), 1.0)
        f["min_p"] = np.where((kind == 4) | (kind == 7), rng.uniform(0.02, 0.2, R), 0.0)
    st = {"case": case, "logits": logits, "samplers": s, "filters": f,
          "tokens": torch.empty(R, dtype=torch.int32, device="cuda"),
          "logprobs": torch.empty(R, dtype=torch.float32, device="cuda")}
    for name, a in (("t", s["temperature"].astype("f8")), ("k", f["top_k"].astype("i8")),
                    ("p", f["top_p"].astype("f8")), ("m", f["min_p"].astype("f8")), ("seed", s["seed"].view("i8")),
                    ("step", s["step"].view("i8"))):
        st[name] = torch.from_numpy(np.ascontiguousarray(a)).cuda()[:, None]
    if own:
        from invariant_vd_step_gb300 import vd
        st["workspace"] = vd.sample_workspace(R, V)
    return st


def _prepare_accept(case, seed):
    g, rng = _generator(seed), np.random.default_rng(int(seed))
    B, N, ctx, V = case["B"], case["N"], case["ctx"], 128256
    parent, depth = _trees(rng, B, N, case["chain"])
    if case["chain"] < 2:  # one level of alternatives below the root, all of them rejected
        parent[:, 1:], depth[:, 1:] = 0, 1
    token = rng.integers(0, V, (B, N)).astype(np.int32)
    choice = rng.integers(V, 2 * V, (B, N)).astype(np.int32)
    for b in range(B):  # four nodes in five choose one of their drafted continuations
        for i in range(N):
            children = np.flatnonzero(parent[b] == i)
            if len(children) and case["chain"] > 1 and rng.random() < 0.8:
                choice[b, i] = token[b, rng.choice(children)]
    shared = ctx // PAGE  # full pages of the prefix every request shares; then each request's own
    each = (ctx + N + PAGE - 1) // PAGE - shared
    table = np.zeros((B, shared + each), np.int32)
    order = rng.permutation(shared + B * each)
    table[:, :shared] = order[:shared]
    table[:, shared:] = order[shared:].reshape(B, each)
    pool = torch.empty((case["layers"], shared + B * each, 2, case["Hkv"], PAGE, case["hd"]), dtype=torch.bfloat16,
                       device="cuda")
    pool.normal_(generator=g)
    st = {"case": case, "pool": pool, "token": torch.from_numpy(token).cuda().reshape(-1),
          "choice": torch.from_numpy(choice).cuda().reshape(-1), "parent": torch.from_numpy(parent).cuda().long(),
          "depth": torch.from_numpy(depth).cuda().long(), "path": torch.from_numpy(_paths(parent)).cuda(),
          "table": torch.from_numpy(table).cuda().long(),
          "length": torch.empty(B, dtype=torch.int32, device="cuda"),
          "out": torch.empty((B, case["chain"]), dtype=torch.int32, device="cuda"), "host": (parent, table)}
    if own:
        st["model"], st["kv"], st["tree"] = _model(B, N, 2 * case["Hkv"], case["Hkv"], case["hd"], 0, ctx,
                                                   case["layers"], pool)
        st["tree"].plan(st["kv"], np.arange(0, B * N + 1, N), parent, np.full(B, ctx, np.int32), table)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        if op == "rotary":
            st["rope"].apply(st["x"], st["pos"], st["y"], inverse=st["case"]["inverse"])
            return st["y"]
        if op == "tree":
            st["tree"].attention(st["kv"], 0, st["q"], st["out"])
            return st["out"]
        if op == "sample":
            from invariant_vd_step_gb300 import vd
            vd.sample(st["logits"], st["samplers"], st["filters"], st["tokens"], st["logprobs"], st["workspace"])
            return {"tokens": st["tokens"], "logprobs": st["logprobs"]}
        st["tree"].accept(st["kv"], st["token"], st["choice"], st["length"], st["out"])
        return {"length": st["length"], "out": st["out"], "pool": st["pool"]}
    return {"rotary": _rotary, "tree": _tree, "sample": _sample, "accept": _accept}[op](st)


def _rotary(st):
    case, rot = st["case"], st["case"]["rot"]
    a = st["pos"].double()[:, None] * st["f"]
    mag = 1.0 / st["mag"] if case["inverse"] else st["mag"]
    c, s = (a.cos() * mag).float()[:, None], (a.sin() * (-mag if case["inverse"] else mag)).float()[:, None]
    x = st["x"].float()
    x1, x2 = (x[..., :rot // 2], x[..., rot // 2:rot]) if case["layout"] == "half" else \
        (x[..., 0:rot:2], x[..., 1:rot:2])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.cat([y1, y2], -1) if case["layout"] == "half" else torch.stack([y1, y2], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1).to(st["x"].dtype)


def _tree(st):
    case, W = st["case"], st["width"]
    B, N, Hq, Hkv, hd = case["B"], case["N"], case["Hq"], case["Hkv"], case["hd"]
    slot = torch.arange(W, device="cuda")
    kv = st["pool"][0][st["table"][:, slot // PAGE], :, :, slot % PAGE].float()  # [B][W][2][Hkv][hd]
    q = st["q"].view(B, N, Hkv, Hq // Hkv, hd).float()
    s = torch.einsum("bnhgd,bwhd->bhgnw", q, kv[:, :, 0]) / math.sqrt(hd)
    ctx, at = st["ctx"][:, None, None], slot[None, None]
    pos = ctx + st["depth"][:, :, None]
    seen = at < ctx
    if case["window"]:
        seen = seen & (at > pos - case["window"])
    node = (at - ctx).clamp(0, N - 1).expand(B, N, W)
    drafted = (at >= ctx) & (at < ctx + N) & st["path"].gather(2, node)
    if case["window"]:
        drafted = drafted & (st["depth"][:, None].expand(B, N, N).gather(2, node) + ctx > pos - case["window"])
    s = s.masked_fill(~(seen | drafted)[:, None, None], -math.inf)
    p = (s - s.amax(-1, keepdim=True)).exp()
    o = torch.einsum("bhgnw,bwhd->bnhgd", p, kv[:, :, 1]) / p.sum(-1).permute(0, 3, 1, 2)[..., None]
    return o.reshape(B * N, Hq, hd).bfloat16()


def _philox(block, seed, step):
    """Words of Philox4x32-10 for counter (block, step, 0x5644) under key `seed`, as int64 tensors."""
    M = 0xFFFFFFFF
    c = [block, step & M, (step >> 32) & M, torch.full_like(block, 0x5644)]
    k0, k1 = seed & M, (seed >> 32) & M
    for r in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # modulo 2^64: the 64-bit products
        c = [((p1 >> 32) & M) ^ c[1] ^ k0, p1 & M, ((p0 >> 32) & M) ^ c[3] ^ k1, p0 & M]
        k0, k1 = (k0 + 0x9E3779B9) & M, (k1 + 0xBB67AE85) & M
    return c


def _uniforms(seed, step, V):
    """u [R][V] in float32 (exact): word i % 4 of block i / 4, its upper 24 bits plus a half, times 2^-24."""
    block = torch.arange((V + 3) // 4, device="cuda").expand(len(seed), -1).contiguous()
    w = torch.stack(_philox(block, seed, step), -1).flatten(1)[:, :V]
    return ((w >> 8).float() + 0.5) * 2.0 ** -24


def _sample(st):
    logits, t = st["logits"], st["t"].float()
    greedy = t <= 0
    x = logits / torch.where(greedy, 1.0, t)
    x, index = torch.sort(x, dim=1, descending=True, stable=True)
    rank = torch.arange(x.shape[1], device="cuda")
    keep = (st["k"] == 0) | (rank < st["k"])
    w = torch.where(keep, (x - x[:, :1]).exp(), 0.0).double()
    mass = w.cumsum(1)
    keep = keep & ((rank == 0) | (st["p"] >= 1) | (mass - w < st["p"] * mass[:, -1:]))
    keep = keep & (x - x[:, :1] >= st["m"].float().log())
    g = -torch.log(-torch.log(_uniforms(st["seed"], st["step"], x.shape[1]))).gather(1, index)
    score = torch.where(keep, x + g, -math.inf)
    best = score.amax(1, keepdim=True)
    token = torch.where(score == best, index, x.shape[1]).amin(1, keepdim=True)
    chosen = logits.gather(1, token) / torch.where(greedy, 1.0, t)
    logprob = (chosen - x[:, :1]).double() - torch.where(keep, w, 0.0).sum(1, keepdim=True).log()
    token = torch.where(greedy, index[:, :1], token)
    return {"tokens": token[:, 0].int(), "logprobs": torch.where(greedy, 0.0, logprob)[:, 0].float()}


def _accept(st):
    case, N = st["case"], st["case"]["N"]
    B, W = case["B"], case["chain"]
    token, choice = st["token"].view(B, N), st["choice"].view(B, N)
    up = st["parent"].clamp(min=0)
    hit = token == choice.gather(1, up)
    node = torch.arange(N, device="cuda")
    # the lowest matching child of each parent
    same = (st["parent"][:, :, None] == st["parent"][:, None]) & hit[:, None] & (node[None] < node[:, None])
    hit = (hit & ~same.any(2)) | (node == 0)
    taken = (hit[:, None] | ~st["path"]).all(2)
    length = taken.sum(1)
    depth = torch.arange(W, device="cuda")
    on = taken[:, None] & (st["depth"][:, None] == depth[:, None])  # [B][W][N]
    at = torch.where(on.any(2), on.int().argmax(2), depth)
    out = torch.where(depth < length[:, None], choice.gather(1, at), -1)
    src, dst = case["ctx"] + at, (case["ctx"] + depth).expand(B, W)
    moved = st["pool"][:, st["table"].gather(1, src // PAGE), :, :, src % PAGE]
    st["pool"][:, st["table"].gather(1, dst // PAGE), :, :, dst % PAGE] = moved
    return {"length": length.int(), "out": out.int(), "pool": st["pool"]}


# ---------------------------------------------------------------- work
def work(case):
    if case["op"] == "rotary":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["hd"] * (4 if case["dtype"] == "fp32" else 2) + 4 * case["T"],
                "flops": 3 * n * case["rot"]}
    if case["op"] == "tree":
        B, N, Hq, Hkv, hd = case["B"], case["N"], case["Hq"], case["Hkv"], case["hd"]
        c = (case["ctx_lo"] + case["ctx_hi"]) / 2
        c = min(c, case["window"]) if case["window"] else c
        path = 1 + min(N, max(1, N // 4)) / 2  # keys of a node's path, on average
        return {"bytes": int(B * ((c + N) * Hkv * 4 + 4 * N * Hq) * hd), "flops": int(4 * B * N * Hq * hd * (c + path))}
    if case["op"] == "sample":
        return {"bytes": case["R"] * (case["V"] * 4 + 48), "flops": 4 * case["R"] * case["V"]}
    moved = case["B"] * max(1, case["chain"] // 2)
    return {"bytes": moved * case["layers"] * 2 * 2 * case["Hkv"] * case["hd"] * 2 + case["B"] * case["N"] * 12,
            "flops": case["B"] * case["N"]}


# ---------------------------------------------------------------- float64
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, st)
    if case["op"] == "tree":
        return _exact_tree(case, st)
    if case["op"] == "sample":
        return _exact_sample(case, st)
    return _exact_accept(case, st)


def _exact_rotary(case, st):
    half, x = case["rot"] // 2, st["x"].double()
    if case["layout"] == "half":
        first = torch.arange(half, device="cuda")
        second = first + half
    else:
        first = torch.arange(half, device="cuda") * 2
        second = first + 1
    sign, mag = (-1, 1 / st["mag"]) if case["inverse"] else (1, st["mag"])
    turn = torch.polar(torch.full_like(st["f"], mag).expand(case["T"], -1), sign * st["pos"].double()[:, None] * st["f"])
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_tree(case, st):
    B, N, Hq, Hkv, hd, window = (case[k] for k in ("B", "N", "Hq", "Hkv", "hd", "window"))
    q, outs = st["q"].double().view(B, N, Hkv, Hq // Hkv, hd), []
    for b in range(B):
        c = int(st["ctx"][b])
        pages = st["pool"][0][st["table"][b, :(c + N + PAGE - 1) // PAGE]].double()
        k, v = pages.permute(1, 2, 0, 3, 4).reshape(2, Hkv, -1, hd)[:, :, :c + N]
        # logical positions of the slots: the prefix in order, then each node at its depth
        where = torch.cat([torch.arange(c, device="cuda"), c + st["depth"][b]])
        see = torch.cat([torch.ones((N, c), dtype=torch.bool, device="cuda"), st["path"][b]], 1)
        if window:
            see &= where[None] + window > (c + st["depth"][b])[:, None]
        w = torch.softmax((torch.matmul(q[b].permute(1, 2, 0, 3), k[:, None].transpose(-1, -2)) * hd ** -0.5)
                          .masked_fill(~see, -math.inf), -1)
        outs.append(torch.matmul(w, v[:, None]).permute(2, 0, 1, 3).reshape(N, Hq, hd))
    return torch.cat(outs)


def _exact_sample(case, st):
    tokens, logprobs = [], []
    for r in range(case["R"]):
        row, t, f = st["logits"][r].double(), float(st["samplers"]["temperature"][r]), st["filters"][r]
        if t <= 0:
            tokens.append(int(row.argmax()))
            logprobs.append(0.0)
            continue
        order = torch.argsort(row, descending=True, stable=True)
        if f["top_k"] > 0:
            order = order[:int(f["top_k"])]
        p = torch.softmax(row[order] / t, 0)
        if f["top_p"] < 1:
            before = torch.cat([p.new_zeros(1), p.cumsum(0)[:-1]])
            order = order[(before < float(f["top_p"])) | (before == 0)]
            p = p[:len(order)]
        if f["min_p"] > 0:
            order = order[p >= float(f["min_p"]) * p[0]]
        word = torch.stack(_philox((order // 4)[:, None], st["seed"][r], st["step"][r]))[:, :, 0]
        u = ((word.gather(0, (order % 4)[None])[0] >> 8).double() + 0.5) / 2 ** 24
        x = row[order] / t
        i = int(torch.argmax(x - (-u.log()).log()))
        tokens.append(int(order[i]))
        logprobs.append(float(torch.log_softmax(x, 0)[i]))
    return {"tokens": torch.tensor(tokens, dtype=torch.int32), "logprobs": torch.tensor(logprobs, dtype=torch.float64)}


def _exact_accept(case, st):
    (parent, table), ctx, pool = st["host"], case["ctx"], st["pool"].clone()
    token, choice = (st[k].view(case["B"], case["N"]).cpu().numpy() for k in ("token", "choice"))
    lengths, out = [], np.full((case["B"], case["chain"]), -1, np.int32)
    for b in range(case["B"]):
        path = [0]
        while True:
            nxt = [i for i in range(case["N"]) if parent[b, i] == path[-1] and token[b, i] == choice[b, path[-1]]]
            if not nxt:
                break
            path.append(nxt[0])
        lengths.append(len(path))
        for d, i in enumerate(path):
            out[b, d] = choice[b, i]
            to, at = ctx + d, ctx + i
            pool[:, table[b, to // PAGE], :, :, to % PAGE] = st["pool"][:, table[b, at // PAGE], :, :, at % PAGE]
    return {"length": torch.tensor(lengths, dtype=torch.int32), "out": torch.from_numpy(out), "pool": pool.double()}
