"""How far attention over an 8-bit cache may be from its fp64 oracle, from the
tokens that the call may use alone.  Slots past a sequence's end and blocks that
no table names may hold numbers of any size: none of them widens the bound."""

import numpy as np

import oracle
from parity import to64


def live_top(cache, table, lens, d):
    """Largest |V| of the tokens of each sequence and KV head, [S, Hkv]."""
    v = oracle.kv8_unpack(cache, d)[1]
    out = np.zeros((len(lens), cache.shape[1]))
    for b, n in enumerate(lens):
        j = np.arange(int(n))
        if n:
            out[b] = np.nan_to_num(np.abs(v[np.asarray(table)[b, j // 16], :, j % 16])).max((0, 2))
    return out


def compare_live(o, lse, ref, cache, table, lens, d, what=""):
    """o and lse of a decode or a prefill.  Scores are fp32 sums of exact products,
    off by under 2^-12 with normalised queries and keys: 2 2^-12 of the largest value
    in o.  Numerators rounded to 11 bits: 2^-11 of it.  o's rounding to bf16: 2^-8 |o|.
    The LSE uses the unrounded numerators: 2^-16 covers its fp32 sums, relative to its
    size where that is more than 16."""
    o_ref, lse_ref = ref
    o, lse = to64(o), lse.double().cpu().numpy()
    nan, none = np.isnan(lse_ref), np.isneginf(lse_ref)
    assert np.array_equal(np.isnan(lse), nan), "%s: other rows are NaN" % what
    assert np.array_equal(np.isnan(o).any(-1), nan) and np.array_equal(np.isnan(o).all(-1), nan), what
    assert np.array_equal(np.isneginf(lse), none) and np.all(o[none] == 0), what
    top = live_top(cache, table, lens, d)
    top = np.repeat(top, o.shape[1] // top.shape[1], 1).reshape(top.shape[0], o.shape[1], *[1] * (o.ndim - 2))
    fine = ~nan & ~none
    lim = (2.0 ** -8 * np.abs(o_ref) + 2.0 ** -10 * top)[fine]
    err = np.abs(o - o_ref)[fine]
    assert np.all(err <= lim), "%s: o at %.3g of its bound" % (what, (err / lim).max())
    lerr = np.abs(lse[fine] - lse_ref[fine])
    assert np.all(lerr <= 2.0 ** -16 * np.maximum(1, np.abs(lse_ref[fine]) / 16)), "%s: lse off by %.3g" % (what, lerr.max())


def close_bound(q, cache, table, lens, scale, d, score=2.0 ** -12):
    """A bound of o's error for each element of a prefill's o, [S, Hq, N, d], from the
    weights w of its row (64 bits): scores off by `score`, numerators rounded to
    11 bits: 2 score and 2^-11 of the sum of w |v|; numerators that round to a multiple
    of 2^-32 of the largest w scale (2^-33 of it each, times codes up to 448); and o's
    rounding to bf16."""
    k, v, _ = oracle.kv8_unpack(cache, d)
    at = 2 * oracle.kv8.SLOTS * d
    scales = np.ascontiguousarray(cache[..., at + 4: at + 8]).view("<f4")[..., 0].astype(np.float64)
    S, Hq, N, _ = q.shape
    g = Hq // cache.shape[1]
    lim = np.zeros(q.shape)
    for b in range(S):
        L = int(lens[b])
        j = np.arange(L)
        blk = np.asarray(table)[b, j // 16]
        for h in range(Hq):
            keys, vals, sv = k[blk, h // g, j % 16], v[blk, h // g, j % 16], scales[blk, h // g]
            see = j[None] <= np.arange(L - N, L)[:, None]
            x = np.where(see, scale * (q[b, h] @ keys.T), -np.inf)
            w = np.exp(x - np.maximum(x.max(-1, keepdims=True), -1e300))
            w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
            o = w @ vals
            lim[b, h] = (2.0 ** -8 * np.abs(o) + (2 * score + 2.0 ** -11) * (w @ np.abs(vals))
                         + 2.0 ** -33 * 448 * see.sum(-1, keepdims=True) * (w * sv).max(-1, keepdims=True))
    return lim
