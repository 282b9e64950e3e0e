"""Filtered token choice in float64, from its definition (no test functions
here): the kept tokens and the scores of a row, with the margins inside which
a float32 implementation may decide either way."""

import numpy as np


def words(index, seed, step):
    """Philox4x32-10 word of each vocabulary index (Salmon et al., SC'11), vectorised."""
    M = np.uint64(0xFFFFFFFF)
    i = np.asarray(index, dtype=np.uint64)
    c = [i // np.uint64(4), np.full_like(i, step & 0xFFFFFFFF), np.full_like(i, step >> 32), np.full_like(i, 0x5644)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for r in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & M, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & M]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c)[(i % np.uint64(4)).astype(int), np.arange(len(i))]


def row_choice(logits, sampler, filt, slack):
    """(token, logprob, may): the choice, its log-probability, and a dict of the tokens that a computation within
    `slack` (relative in masses, absolute in scores) may choose, each with the log-probabilities that it may then have
    (a token whose mass before it is within `slack` of the cut may be kept or not)."""
    seed, step, t = sampler
    k, top_p, min_p = filt
    x = np.asarray(logits, dtype=np.float64)
    real = np.flatnonzero(~np.isnan(x))
    if t <= 0 or len(real) == 0 or x[real].max() == -np.inf:
        tok = int(real[np.argmax(x[real])]) if len(real) else 0
        return tok, 0.0, {tok: [0.0]}
    filtered = (0 < k < len(x)) or top_p < 1 or min_p > 0
    cand = real[x[real] > -np.inf] if filtered else real
    cand = cand[np.lexsort((cand, -x[cand]))]
    if 0 < k < len(x):
        cand = cand[:k]
    top = x[cand[0]]
    with np.errstate(invalid="ignore"):
        d = np.where(x[cand] == top, 0.0, (x[cand] - top) / np.float64(np.float32(t)))
    w = np.exp(d)
    before = (np.cumsum(w) - w) / w.sum()

    def choice(shift):
        keep = np.ones(len(cand), bool)
        if top_p < 1:
            keep &= (before < np.float64(np.float32(top_p)) + shift) | (np.arange(len(cand)) == 0)
        if min_p > 0:
            keep &= (d >= np.log(np.float64(np.float32(min_p))) - shift) | (d == 0)
        kept = cand[keep]
        # the sampler's uniforms as its float32 holds them: from 1/2 on the half rounds to even, and a word of 24 ones
        # in front gives 1, whose score is infinite
        u = np.float64((words(kept, seed, step) >> np.uint64(8)).astype(np.float32) + np.float32(0.5)) / 2.0 ** 24
        with np.errstate(divide="ignore", invalid="ignore"):
            s = x[kept] / np.float64(np.float32(t)) - np.log(-np.log(u))
        s[np.isnan(s)] = -np.inf  # a logit of -inf under an infinite draw: no score beats another
        z = np.log(w[keep].sum())
        near = s >= s.max() - slack * max(1.0, abs(s.max())) if np.isfinite(s.max()) else s == s.max()
        first = int(np.flatnonzero(s == s.max())[0])
        return int(kept[first]), d[keep][first] - z, {int(kept[i]): d[keep][i] - z for i in np.flatnonzero(near)}
    tok, lp, _ = choice(0.0)
    may = {}
    for shift in (0.0, -slack, slack):
        for token, l in choice(shift)[2].items():
            may.setdefault(token, []).append(l)
    return tok, lp, may
