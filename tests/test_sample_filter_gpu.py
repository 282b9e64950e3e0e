"""Filtered token choice on the GPU against a float64 oracle: filters alone
and together, vocabularies of every size, ties, infinities and NaN, rows whose
cut lies far down, refusals."""

import numpy as np
import pytest
import torch

from filter_oracle import row_choice
from gpu_util import ready
from invariant_vd_step_gb300 import synth, vd

pytestmark = pytest.mark.gpu

# Scores: x = l / T and the sum are each rounded once (2^-24 relative), the two logarithms of G are within 2 ulp of
# values up to 17: below 2^-20 of max(1, |score|).  Masses: float32 exponentials (2 ulp of the result plus the
# rounding of an exponent up to 30, 2^-19 together) and sums that are exact beside them.
SLACK = 2.0 ** -18

FILTERS = [(0, 1.0, 0.0), (1, 1.0, 0.0), (2, 1.0, 0.0), (50, 1.0, 0.0), (50, 0.9, 0.0), (0, 0.9, 0.0), (0, 0.0, 0.0),
           (0, 0.5, 0.05), (0, 1.0, 0.1), (0, 1.0, 1.0), (0, 1.0, 1e-30), (64, 0.95, 0.02), (200, 0.999, 0.0),
           (3000, 1.0, 0.0), (3000, 0.99, 0.0), (10 ** 9, 0.3, 0.0), (70, 0.9999, 1e-6), (0, 0.99999, 0.0)]
TEMPS = [0.7, 1.0, 1.6, 0.0, 0.05]


def rows_of(kind, R, V, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((R, V)) * 2.0).astype(np.float32)
    if kind == "flat":
        x *= 0.05
    elif kind == "ties":        # eight bits of mantissa, as logits that were bf16 have
        x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "sorted":      # the likely tokens side by side
        x.sort(axis=1)
    elif kind == "masked":      # a grammar allows few tokens
        allowed = rng.random((R, V)) < min(1.0, 60.0 / V)
        allowed[:, rng.integers(0, V)] = True
        x[~allowed] = -np.inf
    elif kind == "lowest":      # masked with the type's lowest value
        x[rng.random((R, V)) < 0.9] = np.finfo(np.float32).min
    elif kind == "nan":
        x[rng.random((R, V)) < 0.3] = np.nan
    elif kind == "peak":
        x[:, rng.integers(0, V)] = 60.0
    elif kind == "huge":
        x *= 1e30
    elif kind == "zeros":       # signed zeros tie
        x = np.where(rng.random((R, V)) < 0.5, -0.0, 0.0).astype(np.float32)
    return x


def run(x, samplers, filters, pad=0, shift=0, logprobs=True):
    R, V = x.shape
    buf = torch.full((R, V + pad + shift), 100.0, device="cuda")  # what lies between the rows would win
    view = buf[:, shift:shift + V]
    view.copy_(torch.from_numpy(x))
    tok = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    lp = torch.full((R,), float("nan"), device="cuda") if logprobs else None
    vd.sample(view, samplers, filters, tok, lp)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy() if logprobs else None


def check(x, samplers, filters, tok, lp):
    off = 0
    for r in range(len(x)):
        want, want_lp, may = row_choice(x[r], samplers[r], filters[r], SLACK)
        off += tok[r] != want
        assert int(tok[r]) in may, (r, samplers[r], filters[r], int(tok[r]), want)
        # d and the sum's logarithm, each within a few float32 roundings; a mass near the cut may fall either way
        ls = may[int(tok[r])]
        assert any(abs(lp[r] - l) <= 2.0 ** -19 * max(1.0, abs(l)) + SLACK for l in ls), (r, filters[r], lp[r], ls)
    return off


KINDS = ["normal", "flat", "ties", "equal", "sorted", "masked", "lowest", "nan", "peak", "huge", "zeros"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 1024, 1025, 4096, 32003])
def test_choice_vs_float64(V, kind):
    ready()
    rng = np.random.default_rng(V)
    filters = FILTERS
    samplers = [(int(rng.integers(0, 2 ** 63)) * 2 + 1, int(rng.integers(0, 2 ** 50)), TEMPS[i % len(TEMPS)])
                for i in range(len(filters))]
    off = 0
    for turn in range(2):  # every filter under two temperatures
        x = rows_of(kind, len(filters), V, 10 * V + turn)
        tok, lp = run(x, samplers, filters, pad=[0, 3][turn], shift=[0, 1][turn])
        off += check(x, samplers, filters, tok, lp)
        samplers = [(s, st + 1, TEMPS[(i + 1) % len(TEMPS)]) for i, (s, st, _) in enumerate(samplers)]
    assert off <= 1


@pytest.mark.parametrize("V,kind", [(128256, "normal"), (128256, "flat"), (128256, "sorted"), (128256, "equal"),
                                    (128256, "ties"), (262144, "flat"), (262144, "normal"), (262144, "masked"),
                                    (1 << 21, "normal"), (600001, "ties")])
def test_choice_vs_float64_large_vocabularies(V, kind):
    ready()
    rows = [3, 4, 5, 7, 11, 13, 14, 17] if V < 300000 else [4, 5, 14]
    filters = [FILTERS[i] for i in rows]
    samplers = [(99 + i, i, [0.8, 1.0, 1.5][i % 3]) for i in range(len(rows))]
    x = rows_of(kind, len(rows), V, V)
    tok, lp = run(x, samplers, filters)
    assert check(x, samplers, filters, tok, lp) <= 1


def test_many_wide_rows_back_to_back():
    """Several calls on one workspace with nothing waited for between them: rows that need the wide kernels, the exact
    histograms and only the lists, side by side."""
    ready()
    V, R = 40000, 40
    rng = np.random.default_rng(3)
    kinds = ["flat", "normal", "ties", "sorted", "equal", "masked", "nan", "peak"]
    x = np.concatenate([rows_of(kinds[r % 8], 1, V, r) for r in range(R)])
    f = [FILTERS[int(i)] for i in rng.integers(0, len(FILTERS), R)]
    lg, ws = torch.from_numpy(x).cuda(), vd.sample_workspace(R, V)
    outs = []
    for call in range(6):
        s = [(r, call, TEMPS[(r + call) % len(TEMPS)]) for r in range(R)]
        tok, lp = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
        vd.sample(lg, s, f, tok, lp, ws)
        outs.append((s, tok, lp))
    torch.cuda.synchronize()
    assert sum(check(x, s, f, tok.cpu().numpy(), lp.cpu().numpy()) for s, tok, lp in outs) <= 2


def test_rows_without_filters_get_the_samplers_token():
    ready()
    V = 2048
    spec = synth.TINY.with_(vocab=V)
    m = vd.Model(spec, {k: v.cuda() for k, v in synth.make_weights(spec).items()}, max_tokens=16, max_seqs=4,
                 max_logit_rows=1024, max_context=64)
    x = np.concatenate([rows_of(k, 60, V, 5) for k in KINDS])
    x[0, :], x[1, :], x[2, 17], x[3, [5, 900]] = -np.inf, np.nan, np.inf, np.inf
    R = len(x)
    lg = torch.from_numpy(x).cuda()
    state = [(1000 + r, 3 * r, TEMPS[r % len(TEMPS)]) for r in range(R)]
    a, b, c = (torch.empty(R, dtype=torch.int32, device="cuda") for _ in range(3))
    m.sample(lg, state, a)
    m.sample_filtered(lg, state, None, b)
    m.sample_filtered(lg, state, [(0, 1.0, 0.0)] * R, c, torch.empty(R, device="cuda"))
    assert torch.equal(a, b) and torch.equal(a, c)


def test_infinite_and_missing_logits_under_filters():
    ready()
    V = 5000
    x = rows_of("normal", 8, V, 1)
    x[0], x[1] = -np.inf, np.nan
    x[2, 17] = np.inf
    x[3, [9, 4000]] = np.inf
    x[4], x[4, 4321] = -np.inf, -3.0
    x[5, :2500], x[5, 2500:] = np.nan, -np.inf
    f = [(20, 0.9, 0.0)] * 8
    s = [(r, r, 1.0) for r in range(8)]
    for filt in (f, [(0, 0.9, 0.0)] * 8, [(0, 1.0, 0.2)] * 8, [(4900, 0.99, 1e-9)] * 8):
        tok, lp = run(x, s, filt)
        assert tok[:6].tolist() == [0, 0, 17, 9, 4321, 2500]
        assert lp[0] == lp[1] == lp[5] == 0 and lp[2] == lp[4] == 0 and abs(lp[3] - np.log(0.5)) < 1e-6


@pytest.mark.parametrize("levels,count", [(0, 300), (1, 40), (1, 700), (3, 700), (5, 2500)])
def test_cuts_among_the_few_likely_tokens(levels, count):
    """Likely tokens far above the bulk, so that top-p and min-p cut among them: of any value (levels 0), or of a few
    values each shared by many tokens, up to more than a list's bin takes."""
    ready()
    V, filters = 128256, [(0, 0.3, 0.0), (0, 0.9, 0.0), (0, 0.97, 0.05), (0, 1.0, 0.2), (0, 0.6, 0.5), (0, 0.999, 0.0)]
    rng = np.random.default_rng(count)
    x = rows_of("normal", len(filters), V, count)
    for row in x:
        top = rng.random(count) * 8 if levels == 0 else rng.integers(0, levels, count) * 1.5
        row[rng.permutation(V)[:count]] = 20 + top
    s = [(r, count, [0.7, 1.0, 1.4][r % 3]) for r in range(len(filters))]
    assert check(x, s, filters, *run(x, s, filters)) <= 1


@pytest.mark.parametrize("V,std,R", [(262144, 0.2, 20), (262144, 0.01, 3), (40001, 6.0, 90), (131072, 1.0, 700)])
def test_wide_rows_of_any_spread(V, std, R):
    ready()
    some = np.random.default_rng(V).standard_normal((min(R, 10), V)).astype(np.float32) * np.float32(std)
    x = np.tile(some, (-(-R // len(some)), 1))[:R]
    filters = [[(0, 0.95, 0.0), (0, 0.99, 1e-7), (0, 1.0, 1e-6), (V // 3, 1.0, 0.0), (0, 0.9, 0.0)][r % 5] for r in range(R)]
    s = [(7, r % 10, [1.0, 1.6][r % 2]) for r in range(R)]
    tok, lp = run(x, s, filters)
    assert check(x[:10], s[:10], filters[:10], tok[:10], lp[:10]) <= 1
    for r in range(10, R):  # the same ten rows again
        assert tok[r] == tok[r % 10] and lp[r] == lp[r % 10]


def test_row_alone_equals_row_in_a_batch_and_many_rows():
    ready()
    V, R = 3001, 1100  # more rows than one launch takes
    x = np.tile(rows_of("normal", 50, V, 8), (22, 1))
    filters = [FILTERS[r % len(FILTERS)] for r in range(R)]
    s = [(r % 50, r % 7, TEMPS[r % len(TEMPS)]) for r in range(R)]
    tok, lp = run(x, s, filters)
    for r in (0, 5, 511, 512, 600, 1023, 1024, 1099):
        t1, l1 = run(x[r:r + 1], s[r:r + 1], filters[r:r + 1], pad=8)
        assert t1[0] == tok[r] and l1[0] == lp[r]
    again = run(x, s, filters)
    np.testing.assert_array_equal(again[0], tok)
    np.testing.assert_array_equal(again[1], lp)
    np.testing.assert_array_equal(run(x, s, filters, logprobs=False)[0], tok)


@pytest.mark.parametrize("V", [40001, 131072, 262144])
def test_rows_do_not_depend_on_the_rest_of_the_call(V):
    """A row's token and log-probability, bit for bit, alone and in calls of other rows, which change how many CTAs
    share a row and which kernels a call has."""
    ready()
    kinds = ["normal", "flat", "ties", "equal", "sorted", "normal"]
    x = np.concatenate([rows_of(k, 1, V, i) for i, k in enumerate(kinds)])
    filters = [(0, 0.95, 0.0), (0, 0.9, 0.0), (0, 0.97, 0.0), (50, 1.0, 0.0), (200, 1.0, 1e-4), (V // 5, 1.0, 0.0),
               (0, 1.0, 1e-6), (100, 0.99, 0.0)]
    # every row under every filter: row k of the call is kind k % 6 under filter k // 6
    n = len(kinds) * len(filters)
    xs, fs = x[np.arange(n) % 6], [filters[k // 6] for k in range(n)]
    s = [(5 + k, k, [1.0, 1.7][k % 2]) for k in range(n)]
    tok, lp = run(xs, s, fs)
    for group in (1, 5):
        for k0 in range(0, n, group):
            rows = range(k0, min(n, k0 + group))
            t1, l1 = run(xs[k0:k0 + group], [s[k] for k in rows], [fs[k] for k in rows])
            for k in rows:
                assert t1[k - k0] == tok[k] and l1[k - k0] == lp[k], (group, kinds[k % 6], fs[k])


def test_frequencies_follow_the_filtered_distribution():
    ready()
    V, R = 64, 512
    x = np.tile(np.linspace(3, -3, V).astype(np.float32), (R, 1))
    filt = (20, 0.8, 0.0)
    p = np.exp(x[0, :20].astype(np.float64))
    p /= p.sum()
    n = int(np.searchsorted(np.cumsum(p), 0.8)) + 1
    p = p[:n] / p[:n].sum()
    count = np.zeros(V)
    for step in range(40):
        tok, _ = run(x, [(r, step, 1.0) for r in range(R)], [filt] * R)
        count += np.bincount(tok, minlength=V)
    assert count[n:].sum() == 0
    total = count.sum()
    chi2 = ((count[:n] - total * p) ** 2 / (total * p)).sum()
    assert chi2 < n - 1 + 5 * np.sqrt(2 * (n - 1))  # five standard deviations of its distribution


def test_capture_replays_on_new_logits():
    ready()
    V, R = 128256, 3
    x = torch.randn((R, V), device="cuda")
    s, f = [(1, 2, 0.9), (3, 4, 1.2), (5, 6, 1.0)], [(50, 0.9, 0.0), (0, 0.95, 0.0), (0, 1.0, 0.0)]
    ws = vd.sample_workspace(R, V)
    tok, lp = torch.empty(R, dtype=torch.int32, device="cuda"), torch.empty(R, device="cuda")
    vd.sample(x, s, f, tok, lp, ws)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        vd.sample(x, s, f, tok, lp, ws)
    x.copy_(torch.randn((R, V), device="cuda"))
    g.replay()
    t2, l2 = torch.empty_like(tok), torch.empty_like(lp)
    vd.sample(x, s, f, t2, l2)
    torch.cuda.synchronize()
    assert torch.equal(tok, t2) and torch.equal(lp, l2)


def test_a_models_first_filtered_choice_is_refused_in_a_capture():
    ready()
    V = 4096
    spec = synth.TINY.with_(vocab=V)
    model = vd.Model(spec, {k: v.cuda() for k, v in synth.make_weights(spec).items()}, max_tokens=16, max_seqs=4,
                     max_logit_rows=4, max_context=64)
    x, s, f = torch.randn((2, V), device="cuda"), [(1, 2, 1.0), (3, 4, 0.8)], [(0, 0.9, 0.0), (5, 1.0, 0.0)]
    tok, want = torch.full((2,), -1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    vd.sample(x, s, f, want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
        mark = x + 1  # (a graph is not empty)
        with pytest.raises(vd.VDError):
            model.sample_filtered(x, s, f, tok)
    model.sample_filtered(x, s, f, tok)
    assert torch.equal(tok, want)
    tok.fill_(-1)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        model.sample_filtered(x, s, f, tok)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, want) and mark.shape == x.shape
    model.close()


def test_refusals():
    ready()
    x = torch.zeros((2, 100), device="cuda")
    tok, lp = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    s, f = [(0, 0, 1.0)] * 2, [(5, 0.9, 0.1)] * 2
    vd.sample(x, s, f, tok, lp)
    before = tok.clone()
    bad = [dict(filters=[(-1, 1.0, 0.0)] * 2), dict(filters=[(0, 1.5, 0.0)] * 2), dict(filters=[(0, -0.1, 0.0)] * 2),
           dict(filters=[(0, float("nan"), 0.0)] * 2), dict(filters=[(0, 1.0, 2.0)] * 2),
           dict(filters=[(0, 1.0, float("nan"))] * 2), dict(filters=f[:1]), dict(samplers=s[:1]),
           dict(logits=x.half()), dict(logits=x.cpu()), dict(logits=x.t()), dict(logits=x[0]),
           dict(tokens_out=tok.long()), dict(tokens_out=tok[:1]), dict(logprobs_out=lp.double()),
           dict(logprobs_out=lp.cpu()), dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))]
    for i, kw in enumerate(bad):
        a = dict(logits=x, samplers=s, filters=f, tokens_out=tok, logprobs_out=lp)
        a.update(kw)
        with pytest.raises(vd.VDError):
            vd.sample(**a)
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()
    assert torch.equal(tok, before)
