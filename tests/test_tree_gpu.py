"""Token trees on the GPU: attention rows equal to the decoded path bit for bit
and to a float64 oracle, whole tree steps, acceptance, refusals."""

import numpy as np
import pytest
import torch

from gpu_util import bits, f64, ready
from invariant_vd_step_gb300 import synth, vd
from tree_scenario import TreeScenario, make_tree, path_of, tree_spec

pytestmark = pytest.mark.gpu


def check_rows(sc, window=0, layer=0):
    got, ref = sc.attention(layer), sc.decoded(layer)
    np.testing.assert_array_equal(bits(got), bits(ref))
    want, vmax = sc.oracle(window)
    # weights enter P V as two bf16 terms (relative 2^-16 of a weight, whose sum is 1) over fp32 sums, then one
    # rounding to bf16 (half a step: 2^-8 relative)
    tol = 2.0 ** -14 * vmax + 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"max excess {(err - tol).max():.3g}"
    assert sc.model.device_status() == 0


# (query heads, KV heads, head dim): every head dim, groups of 1 to 16 heads
HEADS = [(4, 2, 64), (8, 8, 64), (8, 2, 128), (16, 2, 128), (16, 1, 128), (4, 2, 256), (16, 1, 256), (6, 2, 64)]


@pytest.mark.parametrize("Hq,Hkv,hd", HEADS)
def test_rows_equal_decoded_paths(Hq, Hkv, hd):
    ready()
    # prefixes of none, one, tile and split borders; trees of one node to many row blocks
    trees = [(0, make_tree("random", 5, 1)), (1, make_tree("chain", 1)), (31, make_tree("chain", 4)),
             (32, make_tree("star", 9)), (33, make_tree("random", 17, 2)), (500, make_tree("chain", 40)),
             (511, make_tree("comb", 7)), (512, make_tree("random", 3, 3)), (1030, make_tree("random", 40, 4))]
    check_rows(TreeScenario(tree_spec(Hq, Hkv, hd), trees, seed=Hq + hd))


@pytest.mark.parametrize("window", [1, 5, 33, 600])
@pytest.mark.parametrize("Hq,Hkv,hd", [(4, 2, 64), (8, 2, 128), (4, 2, 256)])
def test_rows_equal_decoded_paths_windows(Hq, Hkv, hd, window):
    ready()
    trees = [(0, make_tree("chain", 40)), (30, make_tree("random", 9, 1)), (513, make_tree("chain", 20)),
             (700, make_tree("random", 33, 2)), (1020, make_tree("comb", 12)), (64, make_tree("chain", 1))]
    check_rows(TreeScenario(tree_spec(Hq, Hkv, hd, window), trees, seed=window), window)


@pytest.mark.parametrize("hd,n", [(64, 256), (128, 128), (256, 96)])
def test_large_trees_and_both_shared_tile_kernels(hd, n):
    ready()
    spec = tree_spec(8, 2, hd)
    sc = TreeScenario(spec, [(1500, make_tree("random", n, 5)), (47, make_tree("random", 64, 6))], seed=hd)
    check_rows(sc)
    tc = sc.attention()
    sc.model.set_attention_prefill(1)  # plans made from here on take mma.sync CTAs
    sc.plan(sc.tree)
    np.testing.assert_array_equal(bits(sc.attention()), bits(tc))


def test_row_does_not_depend_on_the_rest_of_tree_or_batch():
    ready()
    spec = tree_spec(8, 2, 128)
    full = [(700, make_tree("random", 24, 3)), (90, make_tree("star", 6)), (1500, make_tree("chain", 9))]
    sc = TreeScenario(spec, full, seed=4)
    all_rows = sc.attention()
    cu, parent, cached, pt = sc.descriptor()
    for r, keep in ((0, 10), (2, 3), (0, 1)):  # the first nodes of one request, alone
        t = vd.Tree(sc.model, max_nodes=keep)
        t.plan(sc.pool, [0, keep], parent[cu[r]:cu[r] + keep], cached[r:r + 1], pt[r:r + 1])
        out = torch.empty_like(sc.q[:keep])
        t.attention(sc.pool, 0, sc.q[cu[r]:cu[r] + keep].contiguous(), out)
        torch.cuda.synchronize()
        np.testing.assert_array_equal(bits(out), bits(all_rows[cu[r]:cu[r] + keep]))


SPECS = {
    "llama": synth.TINY,
    "gemma": synth.ModelSpec("gemma-tree", 3, 256, 4, 2, 64, 512, 1024, act="geglu", qk_norm=True, rope_theta=1e6,
                             sliding_window=24, local_global_period=3, rms_eps=1e-6, embed_scale=True,
                             norm_offset=True, sandwich_norm=True),
}


def run_path(model, pool, tokens, table, V):
    """Logits of the last position of a token history, prefilled cold."""
    logits = torch.empty((1, V), dtype=torch.float32, device="cuda")
    model.step(pool, vd.StepBatch([(tokens, 0, table)], logit_rows=[len(tokens) - 1]), logits)
    return logits[0]


@pytest.mark.parametrize("name", SPECS)
def test_tree_step_sampling_and_acceptance_equal_plain_decoding(name):
    """A speculative run as a program would make it: plan, step, choose, accept, until each request has its tokens.
    Every node's logits equal a cold forward of its path; the released tokens equal plain decoding."""
    ready()
    spec = SPECS[name]
    V = spec.vocab
    W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=3, gain_std=0.1).items()}
    model = vd.Model(spec, W, max_tokens=256, max_seqs=4, max_logit_rows=64, max_context=256)
    pool = vd.KVPool(model, 96, memory=torch.zeros(model.pool_bytes(96), dtype=torch.uint8, device="cuda"))
    prompts = [synth.make_tokens(n, V, seed=n) for n in (45, 1, 30)]
    temps, new = [0.0, 0.8, 1.3], 12
    perm = synth.page_permutation(96, seed=5)
    tables = [perm[8 * r:8 * r + 8] for r in range(3)]
    spare = perm[40:56]
    # plain decoding
    plain = []
    for r, p in enumerate(prompts):
        h = list(p)
        tok = torch.empty(1, dtype=torch.int32, device="cuda")
        for i in range(new):
            lg = run_path(model, pool, np.array(h, np.int32), spare, V)
            model.sample(lg[None], [(11 + r, i, temps[r])], tok)
            h.append(int(tok.item()))
        plain.append(h[len(p):])
    # speculative: prefill all but the last token, then trees
    hist = [list(p) for p in prompts]
    for r, p in enumerate(prompts):
        if len(p) > 1:
            model.step(pool, vd.StepBatch([(p[:-1], 0, tables[r])]), torch.empty((1, V), device="cuda"))
    rng = np.random.default_rng(0)
    tree = vd.Tree(model, max_nodes=64)
    steps = accepted = 0
    while any(len(h) - len(p) < new for h, p in zip(hist, prompts)):
        parents, toks, depths, cu = [], [], [], [0]
        for r, h in enumerate(hist):
            par = make_tree("random", int(rng.integers(1, 12)), int(rng.integers(1 << 30)))
            done = len(h) - len(prompts[r])
            t = [h[-1]]
            for i in range(1, len(par)):  # drafts: the right token of that position half of the time
                d = len(path_of(par, i)) - 1
                at = done + d - 1
                t.append(plain[r][at] if at < new and rng.random() < 0.6 else int(rng.integers(0, V)))
            parents.append(par)
            toks += t
            depths += [len(path_of(par, i)) - 1 for i in range(len(par))]
            cu.append(cu[-1] + len(par))
        tree.plan(pool, cu, np.concatenate(parents), [len(h) - 1 for h in hist], np.stack(tables), token_ids=toks)
        T = cu[-1]
        logits = torch.empty((T, V), dtype=torch.float32, device="cuda")
        tree.step(pool, logits)
        seq = np.repeat(np.arange(3), np.diff(cu))
        state = [(11 + int(r), len(hist[r]) - len(prompts[r]) + d, temps[r]) for r, d in zip(seq, depths)]
        choice = torch.empty(T, dtype=torch.int32, device="cuda")
        model.sample(logits, state, choice)
        for i in (0, cu[1], T - 1):  # some nodes' logits against a cold forward of their path
            r = int(seq[i])
            path = path_of(parents[r], i - cu[r])
            ref = run_path(model, pool, np.array(hist[r][:-1] + [toks[cu[r] + j] for j in path], np.int32), spare, V)
            assert torch.equal(logits[i].view(torch.int32), ref.view(torch.int32))
        n = torch.empty(3, dtype=torch.int32, device="cuda")
        out = torch.empty((3, 16), dtype=torch.int32, device="cuda")
        tree.accept(pool, None, choice, n, out)
        n, out = n.cpu().numpy(), out.cpu().numpy()
        for r in range(3):
            assert n[r] >= 1 and (out[r, n[r]:] == -1).all()
            hist[r] += [int(x) for x in out[r, :n[r]]]
            accepted += int(n[r]) - 1
        steps += 1
    assert steps < 3 * new and accepted > 0
    for h, p, want in zip(hist, prompts, plain):
        assert h[len(p):len(p) + new] == want
    # the K/V that acceptance left equals the K/V of a cold prefill
    for r, h in enumerate(hist):
        m = len(h) - 1
        run_path(model, pool, np.array(h[:-1], np.int32), spare, V)
        shape = (m, spec.n_kv_heads, spec.head_dim)
        kv = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        for layer in range(spec.n_layers):
            model.copy_kv(pool, layer, tables[r], m, kv[0], kv[1])
            model.copy_kv(pool, layer, spare, m, kv[2], kv[3])
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bits(kv[0]), bits(kv[2]))
            np.testing.assert_array_equal(bits(kv[1]), bits(kv[3]))
    assert model.device_status() == 0


@pytest.mark.parametrize("most", [None, 1, 2, 5])
@pytest.mark.parametrize("layers,Hkv,hd,n", [(1, 1, 64, 1), (3, 2, 64, 40), (2, 8, 128, 33), (2, 2, 256, 1024)])
def test_accept_moves_the_path_and_nothing_else(layers, Hkv, hd, n, most):
    ready()
    spec = tree_spec(2 * Hkv, Hkv, hd, layers=layers)
    W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=1).items()}
    model = vd.Model(spec, W, max_tokens=2 * n, max_seqs=2, max_logit_rows=8, max_context=n + 32)
    P = 2 * (n // 16 + 3)
    pool = vd.KVPool(model, P, memory=torch.zeros(model.pool_bytes(P), dtype=torch.uint8, device="cuda"))
    view = pool.view()
    view.copy_(synth.make_normal_bf16(tuple(view.shape), seed=3).cuda())
    before = view.clone()
    rng = np.random.default_rng(n)
    kinds = ["random", "chain"] if n < 1024 else ["chain", "comb"]
    parents = [make_tree(k, n, 7) for k in kinds]
    cached = np.array([13, 16], np.int32)
    pt = synth.page_permutation(P, seed=2).reshape(2, -1)
    tok = rng.integers(0, 50, 2 * n).astype(np.int32)
    choice = np.full(2 * n, -7, np.int32)
    for r in range(2):  # follow a random child everywhere; some siblings hold the same token
        for i in range(n):
            kids = np.flatnonzero(parents[r] == i)
            if len(kids):
                choice[r * n + i] = tok[r * n + rng.choice(kids)]
    tree = vd.Tree(model, max_nodes=2 * n)
    tree.plan(pool, [0, n, 2 * n], np.concatenate(parents), cached, pt)
    got_n = torch.full((2,), -5, dtype=torch.int32, device="cuda")
    stride = most or n + 3  # a path longer than that ends there
    got = torch.full((2, stride), -5, dtype=torch.int32, device="cuda")
    tree.accept(pool, torch.from_numpy(tok).cuda(), torch.from_numpy(choice).cuda(), got_n, got)
    torch.cuda.synchronize()
    want = before.clone()
    for r in range(2):
        path = [0]
        while len(path) < stride:
            kids = [i for i in np.flatnonzero(parents[r] == path[-1]) if tok[r * n + i] == choice[r * n + path[-1]]]
            if not kids:
                break
            path.append(int(kids[0]))
        assert got_n[r].item() == len(path)
        assert got[r].tolist() == [int(choice[r * n + i]) for i in path] + [-1] * (stride - len(path))
        for d, i in enumerate(path):
            to, at = cached[r] + d, cached[r] + i
            want[:, pt[r, to // 16], :, :, to % 16] = before[:, pt[r, at // 16], :, :, at % 16]
    assert torch.equal(view.view(torch.int16), want.view(torch.int16))


def test_refusals_leave_plan_and_memory_alone():
    ready()
    spec = tree_spec(4, 2, 64)
    sc = TreeScenario(spec, [(20, make_tree("random", 6, 1)), (3, make_tree("chain", 2))], max_tokens=64)
    first = sc.attention()
    cu, parent, cached, pt = sc.descriptor()

    def code(**kw):
        a = dict(cu_nodes=cu, parent=parent, cached_len=cached, page_table=pt)
        a.update(kw)
        with pytest.raises(vd.VDError) as e:
            sc.tree.plan(sc.pool, **a)
        return e.value.code

    def with_(a, i, v):
        a = a.copy()
        a[i] = v
        return a
    assert code(parent=with_(parent, 0, 0)) == 1           # node 0 is the root
    assert code(parent=with_(parent, 3, 3)) == 1           # its own parent
    assert code(parent=with_(parent, 3, -1)) == 1          # a second root
    assert code(parent=with_(parent, 3, 5)) == 1           # a later node
    assert code(cached_len=with_(cached, 0, -1)) == 1
    assert code(cached_len=with_(cached, 0, 10 ** 6)) == 4
    assert code(cached_len=with_(cached, 1, 2 ** 31 - 1)) == 4
    assert code(page_table=pt[:, :1]) == 3
    assert code(page_table=with_(pt, (0, 1), sc.num_pages)) == 3
    assert code(page_table=with_(pt, (0, 1), -1)) == 3
    assert code(page_table=np.stack([pt[0], pt[0]]), cached_len=[20, 20]) == 1  # two nodes in one slot
    assert code(token_ids=np.full(8, spec.vocab)) == 3
    assert code(cu_nodes=np.array([0, 8, 8])) == 1          # a request without nodes
    assert code(cu_nodes=np.array([0, 9, 8])) == 1
    big = vd.Tree(sc.model, max_nodes=4)
    with pytest.raises(vd.VDError) as e:
        sc.plan(big)
    assert e.value.code == 4
    with pytest.raises(vd.VDError):
        vd.Tree(sc.model, max_nodes=0)
    with pytest.raises(vd.VDError) as e:
        vd.Tree(sc.model, max_nodes=65)                     # more than the model's max_tokens
    assert e.value.code == 4
    other = vd.KVPool(sc.model, 4)
    with pytest.raises(vd.VDError):
        sc.tree.attention(other, 0, sc.q, torch.empty_like(sc.q))
    with pytest.raises(vd.VDError):
        sc.tree.attention(sc.pool, 1, sc.q, torch.empty_like(sc.q))
    with pytest.raises(vd.VDError):
        sc.tree.attention(sc.pool, 0, sc.q[:3], torch.empty_like(sc.q))
    with pytest.raises(vd.VDError):
        sc.tree.attention(sc.pool, 0, sc.q.float(), torch.empty_like(sc.q))
    with pytest.raises(vd.VDError):
        sc.tree.step(sc.pool, torch.empty((8, spec.vocab), device="cuda"))  # no token_ids in the plan
    n, out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty((2, 0), dtype=torch.int32, device="cuda")
    ch = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(vd.VDError):
        sc.tree.accept(sc.pool, None, ch, n, out)           # no tokens
    with pytest.raises(vd.VDError) as e:
        sc.tree.accept(sc.pool, ch, ch, n, out)             # out_tokens without room for the root's choice
    assert e.value.code == 4
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    o = torch.empty_like(sc.q)
    caught = []
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        o.zero_()
        try:
            sc.tree.attention(sc.pool, 0, sc.q, o)
        except vd.VDError as e:
            caught.append(e.code)
    assert caught == [2]
    np.testing.assert_array_equal(bits(sc.attention()), bits(first))  # the plan in force still runs
    empty = vd.Tree(sc.model, max_nodes=4)
    empty.plan(sc.pool, [0], [], [], np.zeros((0, 0), np.int32))
    empty.attention(sc.pool, 0, sc.q[:0], sc.q[:0])
    assert sc.model.device_status() == 0


def test_side_stream_alignment_and_closing():
    ready()
    sc = TreeScenario(tree_spec(8, 2, 64), [(40, make_tree("random", 12, 3)), (600, make_tree("chain", 5))], seed=4)
    want = sc.attention()
    out, side = torch.full_like(sc.q, float("nan")), torch.cuda.Stream()
    torch.cuda.synchronize()
    sc.tree.plan(sc.pool, *sc.descriptor(), token_ids=np.arange(17), stream=side)
    sc.tree.attention(sc.pool, 0, sc.q, out, stream=side)
    side.synchronize()
    np.testing.assert_array_equal(bits(out), bits(want))
    # acceptance takes 4-byte aligned arrays only
    L, i32 = vd.lib(), torch.zeros(256, dtype=torch.int32, device="cuda")
    before, at = sc.pool.memory.clone(), i32.data_ptr()
    for shift in ((1, 0, 0), (0, 2, 0), (0, 0, 3)):
        args = [at + 256 * k + s for k, s in enumerate(shift)]
        assert L.vd_tree_accept(sc.tree.h, sc.pool.h, None, *args, 16, None) == vd.VD_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(sc.pool.memory, before) and not i32.any()
    # a model may be closed before its tree, which then only closes
    other = vd.Tree(sc.model, max_nodes=4)
    sc.tree.close()
    with pytest.raises(vd.VDError):
        sc.tree.attention(sc.pool, 0, sc.q, out)
    sc.pool.close()
    sc.model.close()
    with pytest.raises(vd.VDError):
        other.plan(sc.pool, *sc.descriptor())
    other.close()
    other.close()
