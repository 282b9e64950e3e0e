"""Token-tree scenarios: a pool of seeded K/V, trees of seeded shape over
cached prefixes, and, for every node, the same path laid out as an ordinary
request (no test functions here)."""

import numpy as np
import torch

from gpu_util import f64
from invariant_vd_step_gb300 import synth, vd


def tree_spec(Hq, Hkv, hd, window=0, layers=1):
    return synth.ModelSpec(f"tree{Hq}-{Hkv}-{hd}", layers, 256, Hq, Hkv, hd, 256, 512, sliding_window=window,
                           local_global_period=layers + 1 if window else 0)


def make_tree(kind, n, seed=0):
    """Parents of a tree of n nodes: a chain, a star, a comb or a random tree."""
    if kind == "chain":
        return np.arange(-1, n - 1, dtype=np.int32)
    if kind == "star":
        return np.array([-1] + [0] * (n - 1), np.int32)
    if kind == "comb":  # a chain of the even nodes, a leaf on each
        return np.array([-1] + [i - 1 if i % 2 else max(i - 2, 0) for i in range(1, n)], np.int32)
    rng = np.random.default_rng(seed)
    return np.array([-1] + [int(rng.integers(0, i)) for i in range(1, n)], np.int32)


def path_of(parent, i):
    out = []
    while i >= 0:
        out.append(i)
        i = int(parent[i])
    return out[::-1]


class TreeScenario:
    """trees: list of (cached_len, parents).  Each request's slots 0 .. cached + n - 1 hold seeded K/V in pages of
    their own; the pool's other slots hold NaN, so that nothing outside a node's path may enter its row.  (The pages
    of the paths laid out for ordinary attention end in zeros: it gives their masked slots the weight 0.)"""

    def __init__(self, spec, trees, seed=0, extra_pages=0, max_tokens=None):
        self.spec, self.trees = spec, trees
        N = sum(len(p) for _, p in trees)
        need = [(c + len(p) + 15) // 16 for c, p in trees]
        own = [[-(-(c + len(path_of(p, i))) // 16) - c // 16 for i in range(len(p))] for c, p in trees]
        self.num_pages = sum(need) + sum(map(sum, own)) + extra_pages
        W = {k: v.cuda() for k, v in synth.make_weights(spec, seed=seed).items()}
        self.max_context = max(c + len(p) for c, p in trees) + 16
        self.model = vd.Model(spec, W, max_tokens=max_tokens or max(N, 64), max_seqs=max(N, 8), max_logit_rows=max(N, 8),
                              max_context=self.max_context)
        mem = torch.zeros(self.model.pool_bytes(self.num_pages), dtype=torch.uint8, device="cuda")
        self.pool = vd.KVPool(self.model, self.num_pages, memory=mem)
        view = self.pool.view()
        view.fill_(float("nan"))
        perm = synth.page_permutation(self.num_pages, seed=seed + 1)
        k, self.tables, self.K, self.V = 0, [], [], []
        Hkv, hd = spec.n_kv_heads, spec.head_dim
        for r, (c, p) in enumerate(trees):
            t = perm[k:k + need[r]]
            k += need[r]
            self.tables.append(t)
            kv = synth.make_normal_bf16((2, c + len(p), Hkv, hd), seed=100 * seed + r).cuda()
            self.K.append(kv[0])
            self.V.append(kv[1])
            self._write(view, t, kv, 0)
        # every node's path as a request of its own, behind the shared full pages of the prefix
        self.paths = []
        for r, (c, p) in enumerate(trees):
            for i in range(len(p)):
                path = path_of(p, i)
                full = c // 16
                t = np.concatenate([self.tables[r][:full], perm[k:k + own[r][i]]]).astype(np.int32)
                k += own[r][i]
                slots = list(range(16 * full, c)) + [c + j for j in path]
                kv = torch.stack([self.K[r][slots], self.V[r][slots]])
                view[:, t[full:]] = 0
                self._write(view, t, kv, 16 * full)
                self.paths.append((r, i, c + len(path) - 1, t))
        self.q = synth.make_normal_bf16((N, spec.n_heads, spec.head_dim), seed=seed + 9).cuda()
        self.tree = vd.Tree(self.model, max_nodes=N)
        self.plan(self.tree)

    def _write(self, view, table, kv, first):
        for j in range(kv.shape[1]):
            s = first + j
            view[:, table[s // 16], :, :, s % 16] = kv[:, j][None]

    def descriptor(self):
        width = max(len(t) for t in self.tables)
        pt = np.zeros((len(self.tables), width), np.int32)
        for r, t in enumerate(self.tables):
            pt[r, :len(t)] = t
        cu = np.concatenate([[0], np.cumsum([len(p) for _, p in self.trees])]).astype(np.int32)
        return cu, np.concatenate([p for _, p in self.trees]), np.array([c for c, _ in self.trees], np.int32), pt

    def plan(self, tree, token_ids=None):
        tree.plan(self.pool, *self.descriptor(), token_ids=token_ids)

    def attention(self, layer=0):
        out = torch.full_like(self.q, float("nan"))
        self.tree.attention(self.pool, layer, self.q, out)
        torch.cuda.synchronize()
        return out

    def decoded(self, layer=0):
        """Every node's row by the ordinary attention of its path, one decode row per node."""
        out = torch.full_like(self.q, float("nan"))
        b = vd.StepBatch([(np.zeros(1, np.int32), p, t) for _, _, p, t in self.paths])
        self.model.attention(self.pool, layer, b, self.q, out)
        torch.cuda.synchronize()
        return out

    def oracle(self, window):
        """float64 rows, and the largest |v| that each row's request holds."""
        q, rows, vmax = f64(self.q), [], []
        G = self.spec.n_heads // self.spec.n_kv_heads
        for n, (r, i, p, _) in enumerate(self.paths):
            c, parent = self.trees[r]
            slots = list(range(c)) + [c + j for j in path_of(parent, i)]
            slots = slots[max(0, p - window + 1):] if window else slots
            K, V = f64(self.K[r][slots]), f64(self.V[r][slots])
            s = np.einsum("hgd,jhd->hgj", q[n].reshape(-1, G, self.spec.head_dim), K) / np.sqrt(self.spec.head_dim)
            w = np.exp(s - s.max(-1, keepdims=True))
            w /= w.sum(-1, keepdims=True)
            rows.append(np.einsum("hgj,jhd->hgd", w, V).reshape(self.spec.n_heads, -1))
            vmax.append(np.abs(V).max())
        return np.stack(rows), np.array(vmax)[:, None, None]
