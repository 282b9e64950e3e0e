"""Steps over the 8-bit cache as a serving loop makes them: prompts in chunks, decoding, forks that copy the page being
filled, freed and compacted pages; logits bit for bit the same however a history was computed, and against the oracle."""

import numpy as np
import pytest
import torch

import oracle.decoder as od
from gpu_util import assert_logits_close, bits, ready
from invariant_vd_step_gb300 import synth, vd

pytestmark = pytest.mark.gpu

TINY = synth.TINY
WINDOW = synth.TINY.with_(name="tiny-window", sliding_window=40, local_global_period=2, rope_theta_local=1e4)
G16 = synth.TINY.with_(name="tiny-g16", n_heads=16, n_kv_heads=1)


class Server:
    """Requests over one cache and one pool, both shared by reference counts."""

    def __init__(self, spec, fmt, pages8=60, pages16=40, weights=None):
        W = weights or {k: v.cuda() for k, v in synth.make_weights(spec, seed=3, gain_std=0.1).items()}
        self.spec, self.W = spec, W
        self.model = vd.Model(spec, W, max_tokens=256, max_seqs=8, max_logit_rows=256, max_context=512)
        self.cache = vd.KV8Cache(self.model, pages8, fmt)
        mem = torch.zeros(self.model.pool_bytes(pages16), dtype=torch.uint8, device="cuda")
        self.pool = vd.KVPool(self.model, pages16, memory=mem)
        self.pool.view().fill_(float("nan"))
        self.plan = vd.KV8Plan(self.model, 256)
        self.p8, self.p16 = vd.Pages(pages8), vd.Pages(pages16)
        self.seq = {}

    def step(self, work):
        """work: {request: new tokens}.  Logits [T][V] of every new token."""
        rows, cu, toks = list(work), [0], []
        for r in rows:
            s = self.seq.setdefault(r, {"len": 0, "t8": [], "t16": []})
            c, n = s["len"], len(work[r])
            s["t8"] += self.p8.alloc((c + n) // 16 - len(s["t8"])).tolist()
            s["t16"] += self.p16.alloc((c + n + 15) // 16 - c // 16 - len(s["t16"])).tolist()
            cu.append(cu[-1] + n)
            toks += list(work[r])
        pad = lambda k: np.array([self.seq[r][k] + [0] * (40 - len(self.seq[r][k])) for r in rows], np.int32)  # noqa: E731
        logits = torch.empty((cu[-1], self.spec.vocab), dtype=torch.float32, device="cuda")
        self.plan.plan(self.cache, self.pool, cu, [self.seq[r]["len"] for r in rows], pad("t8"), pad("t16"), toks,
                       np.arange(cu[-1]))
        self.plan.step(self.cache, self.pool, logits)
        for r in rows:
            s = self.seq[r]
            done = (s["len"] + len(work[r])) // 16 - s["len"] // 16
            self.p16.release(s["t16"][:done])
            s["t16"] = s["t16"][done:]
            s["len"] += len(work[r])
        torch.cuda.synchronize()
        assert self.model.device_status() == 0
        return {r: logits[cu[i]:cu[i + 1]] for i, r in enumerate(rows)}

    def fork(self, r, children):
        s = self.seq[r]
        full = s["len"] // 16
        t8, src, dst = self.p8.fork(s["t8"][:full], full, len(children))
        assert src.size == 0
        t16, src, dst = self.p16.fork(s["t16"], 0, len(children))
        self.pool.copy_pages(src, dst)
        for i, c in enumerate(children):
            self.seq[c] = {"len": s["len"], "t8": t8[i].tolist(), "t16": t16[i].tolist()}

    def drop(self, r):
        s = self.seq.pop(r)
        self.p8.release(s["t8"])
        self.p16.release(s["t16"])

    def compact(self):
        """Both caches; the pages beyond those in use are overwritten."""
        for pages, key, cache in ((self.p8, "t8", self.cache), (self.p16, "t16", self.pool)):
            flat = np.array([x for s in self.seq.values() for x in s[key]], np.int32)
            src, dst = pages.compact(flat)
            cache.copy_pages(src, dst)
            at = 0
            for s in self.seq.values():
                s[key] = flat[at:at + len(s[key])].tolist()
                at += len(s[key])


def run(server, r, tokens, cuts):
    out, at = [], 0
    for n in cuts:
        out.append(server.step({r: tokens[at:at + n]})[r])
        at += n
    assert at == len(tokens)
    return torch.cat(out)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("spec", [TINY, WINDOW, G16], ids=lambda s: s.name)
def test_histories_give_the_same_bits_however_they_are_computed(spec, fmt):
    ready()
    toks = synth.make_tokens(150, spec.vocab, seed=4)
    sv = Server(spec, fmt)
    want = bits(run(sv, "whole", toks, [150]))
    for cuts in ([16, 16, 118], [1] * 40 + [110], [37, 1, 1, 9, 102], [150 - 3, 1, 1, 1]):
        np.testing.assert_array_equal(bits(run(sv, str(cuts), toks, cuts)), want)
        sv.drop(str(cuts))
    # forks in the middle of a page, decoded side by side with different tokens, then pages freed and compacted
    sv.drop("whole")
    run(sv, "base", toks[:37], [37])
    other = synth.make_tokens(150, spec.vocab, seed=5)
    sv.fork("base", ["a", "b"])
    a, b = [], []
    for i in range(30):
        got = sv.step({"b": other[37 + i:38 + i], "a": toks[37 + i:38 + i]})
        a.append(got["a"])
        b.append(got["b"])
        if i == 12:
            sv.drop("base")
            sv.compact()
            sv.cache.seal(sv.pool, [0], [sv.cache.num_pages - 1])  # a page that is no longer anyone's
    a.append(sv.step({"a": toks[67:150]})["a"])
    np.testing.assert_array_equal(bits(torch.cat(a)), want[37:])
    fresh = Server(spec, fmt, weights=sv.W)
    mixed = np.concatenate([toks[:37], other[37:67]])
    np.testing.assert_array_equal(bits(torch.cat(b)), bits(run(fresh, "b", mixed, [67]))[37:])
    sv.drop("a")
    sv.drop("b")
    assert sv.p8.free == 60 and sv.p16.free == 40


@pytest.mark.parametrize("spec", [TINY, WINDOW], ids=lambda s: s.name)
def test_step_against_the_oracle(spec, monkeypatch):
    """The 64-bit oracle with this cache's attention in place of its own; the step's stated tolerance (int8: a bf16 step
    of K or V moves a code by at most one, which is no more than a bf16 step of the page's largest value)."""
    ready()

    def attention8(q, K, V, positions, window, perturb=None):
        out = np.empty(q.shape)
        full = K.shape[0] // 16 * 16
        dec = []
        for x in (K, V):
            y = x.copy()
            blocks = y[:full].reshape(-1, 16, *y.shape[1:])
            a = np.maximum(np.abs(blocks).max((1, 3), keepdims=True), 2.0 ** -80)
            y[:full] = (np.rint(127 * blocks / a) * a / 127).reshape(y[:full].shape)
            dec.append(y)
        G = q.shape[1] // K.shape[1]
        for t, p in enumerate(positions):
            p = int(p)
            lo, own = (max(0, p - window + 1) if window else 0), p // 16 * 16
            k, v = (np.concatenate([d[lo:own], x[max(lo, own):p + 1]]) for d, x in zip(dec, (K, V)))
            for h in range(q.shape[1]):
                s = k[:, h // G] @ q[t, h] / np.sqrt(q.shape[2])
                w = np.exp(s - s.max())
                out[t, h] = w @ v[:, h // G] / w.sum()
        return od.round_bf16(out)

    monkeypatch.setattr(od, "attention", attention8)
    sv = Server(spec, "int8")
    toks = synth.make_tokens(100, spec.vocab, seed=8)
    got = run(sv, 0, toks, [70, 1, 1, 20, 8]).cpu().numpy().astype(np.float64)
    ref = od.OracleDecoder(spec, synth.weights_to_numpy({k: v.cpu() for k, v in sv.W.items()})).forward_all(toks)
    assert_logits_close(got, ref)
