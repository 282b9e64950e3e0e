"""Tree kernels launched one behind the other with nothing waited for between them, on windows that leave none of the
shared tiles visible: whole steps, and RoPE + K/V write followed by attention, against the decoded paths."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from invariant_vd_step_gb300 import synth, vd
from tree_scenario import make_tree, path_of, tree_spec

pytestmark = pytest.mark.gpu


class Requests:
    """Requests whose cached prefix ends at least `window` keys into a 32-key tile, each with pages of its own and
    spare pages in which a path is laid out as an ordinary request behind the same prefix."""

    def __init__(self, spec, cached, nodes, seed=0):
        self.spec, self.cached = spec, cached
        self.parents = [make_tree("random" if r % 2 else "chain", n, seed + r) for r, n in enumerate(nodes)]
        self.cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.T = int(self.cu[-1])
        need = [(c + n + 15) // 16 for c, n in zip(cached, nodes)]
        W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=seed, gain_std=0.1).items()}
        B, longest = len(cached), max(c + n for c, n in zip(cached, nodes))
        self.model = vd.Model(spec, W, max_tokens=max(longest, self.T), max_seqs=max(B, 8), max_logit_rows=max(self.T, 8),
                              max_context=longest + 16)
        P = 2 * sum(need)
        mem = torch.zeros(self.model.pool_bytes(P), dtype=torch.uint8, device="cuda")
        self.pool = vd.KVPool(self.model, P, memory=mem)
        perm, k = synth.page_permutation(P, seed=seed + 1), 0
        self.tables, self.spare = [], []
        for n in need:
            self.tables.append(perm[k:k + n])
            self.spare.append(perm[k + n:k + 2 * n])
            k += 2 * n
        self.pt = np.zeros((B, max(need)), np.int32)
        for r, t in enumerate(self.tables):
            self.pt[r, :len(t)] = t
        self.tree = vd.Tree(self.model, max_nodes=self.T)

    def plan(self, token_ids=None):
        self.tree.plan(self.pool, self.cu, np.concatenate(self.parents), self.cached, self.pt, token_ids=token_ids)

    def paths(self, rng):
        """One path of each request, ending at a random node."""
        return [path_of(p, int(rng.integers(0, len(p)))) for p in self.parents]


def below_the_tile(window, rng, tiles):
    return [32 * t + int(rng.integers(window, 32)) for t in tiles]


# few requests: launches of at most one CTA per SM; many: every class of CTA (set_attention_prefill(1): mma.sync)
SIZES = {"few": ([0, 1, 2], [5, 9, 3], 0), "many": ([40, 17, 33, 1, 38, 25, 40, 20, 16, 31], [40] * 9 + [7], 0),
         "many-mma": ([40, 17, 33, 1, 38, 25, 40, 20, 16, 31], [40] * 8 + [12, 7], 1)}


@pytest.mark.parametrize("window", [1, 6, 18, 31])
@pytest.mark.parametrize("size", SIZES)
def test_steps_in_a_row(size, window):
    ready()
    tiles, nodes, kernel = SIZES[size]
    rng = np.random.default_rng(window)
    spec = tree_spec(4, 2, 64, window, layers=3)
    q = Requests(spec, below_the_tile(window, rng, tiles), nodes, seed=window)
    q.model.set_attention_prefill(kernel)
    V = spec.vocab
    for c, own, spare in zip(q.cached, q.tables, q.spare):
        history = synth.make_tokens(c, V, seed=c)
        for t in (own, spare):
            q.model.step(q.pool, vd.StepBatch([(history, 0, t)]), torch.empty((1, V), device="cuda"))
    tokens = [synth.make_tokens(q.T, V, seed=50 + i) for i in range(12)]
    got = [torch.empty((q.T, V), dtype=torch.float32, device="cuda") for _ in tokens]
    torch.cuda.synchronize()
    for toks, out in zip(tokens, got):  # nothing waits in here
        q.plan(toks)
        q.tree.step(q.pool, out)
    for toks, out in zip(tokens, got):
        paths = q.paths(rng)
        b = vd.StepBatch([(toks[q.cu[r] + np.array(p)], q.cached[r], q.spare[r]) for r, p in enumerate(paths)],
                         logit_rows=np.cumsum([len(p) for p in paths]) - 1)
        ref = torch.empty((len(paths), V), dtype=torch.float32, device="cuda")
        q.model.step(q.pool, b, ref)
        rows = [int(q.cu[r]) + p[-1] for r, p in enumerate(paths)]
        np.testing.assert_array_equal(bits(out[rows]), bits(ref))
    assert q.model.device_status() == 0


@pytest.mark.parametrize("window", [1, 13, 31])
@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("Hq,Hkv,hd,layout", [(4, 2, 64, None), (8, 2, 128, "interleaved"), (4, 2, 256, "half")])
def test_rope_then_attention_in_a_row(Hq, Hkv, hd, layout, size, window):
    ready()
    tiles, nodes, kernel = SIZES[size]
    rng = np.random.default_rng(window)
    spec = tree_spec(Hq, Hkv, hd, window)
    q = Requests(spec, below_the_tile(window, rng, tiles), nodes, seed=hd + window)
    q.model.set_attention_prefill(kernel)
    if layout is not None:  # a rope of the model's own choosing, over part of the head where the pairs are neighbours
        q.model.set_rope(vd.Rope(hd, rot_dim=hd // 2 if layout == "interleaved" else 0, layout=layout, theta=5e5))
    view = q.pool.view()
    view.copy_(synth.make_normal_bf16(tuple(view.shape), seed=3).cuda())
    for own, spare in zip(q.tables, q.spare):
        view[:, spare.tolist()] = view[:, own.tolist()]
    q.plan()
    qkv = [synth.make_normal_bf16((q.T, spec.qkv_dim), seed=20 + i).cuda() for i in range(16)]
    rot, out = ([torch.full((q.T, Hq, hd), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in qkv] for _ in range(2))
    torch.cuda.synchronize()
    for x, y, o in zip(qkv, rot, out):  # nothing waits in here
        q.tree.rope_kv(q.pool, 0, x, y)
        q.tree.attention(q.pool, 0, y, o)
    for x, y, o in zip(qkv, rot, out):
        paths = q.paths(rng)
        rows = np.concatenate([q.cu[r] + np.array(p) for r, p in enumerate(paths)])
        b = vd.StepBatch([(np.zeros(len(p), np.int32), q.cached[r], q.spare[r]) for r, p in enumerate(paths)])
        ry, ro = (torch.empty((len(rows), Hq, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        q.model.rope_kv(q.pool, 0, b, x[rows].contiguous(), ry)
        q.model.attention(q.pool, 0, b, ry, ro)
        np.testing.assert_array_equal(bits(y[rows]), bits(ry))
        last = np.cumsum([len(p) for p in paths]) - 1
        np.testing.assert_array_equal(bits(o[rows[last]]), bits(ro[last]))
    assert q.model.device_status() == 0
