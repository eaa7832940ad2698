"""Reference of the 8-bit paged KV cache — TEST INFRASTRUCTURE ONLY.

A code is an e4m3 number: bit 7 the sign, bits 6 .. 3 an exponent E, bits
2 .. 0 a fraction f; (1 + f/8) 2^(E - 7), or f/8 2^-6 for E = 0; codes 0x7f and
0xff are NaN.  Its value is that times the scale of its (block, head, kind): the
smallest power of two, 2^-64 .. 2^64, under which no finite element of the
block's tokens exceeds 448.

A record holds the 16 token slots of one KV head of one block: K codes [16][d],
V codes [16][d], K scale, V scale (fp32), a 32-bit word of flags (bit s: the
key of slot s has an element that is not finite; bit 16 + s: its value), zeros
up to 32 d + 32 bytes.  Written out element by element here.
"""

import numpy as np

SLOTS = 16
MOST = 448.0


def kv8_record_bytes(d):
    return 2 * SLOTS * d + 32


def kv8_code_values():
    """The fp64 values of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        out[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return out


def kv8_codes(x):
    """The nearest codes of x (fp64, in units of the scale): half to even, at
    most 448; NaN and infinities as 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    pos = kv8_code_values()[:127]                    # ascending
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), MOST)
    hi = np.minimum(np.searchsorted(pos, a), 126)    # pos[hi - 1] < a <= pos[hi]
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def kv8_scale(x):
    """The scale for elements x (any shape): over those that are finite."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    most = x[np.isfinite(x)].max(initial=0.0)
    e = -64
    while e < 64 and most > MOST * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _tail(record, d):
    at = 2 * SLOTS * d
    return record[at: at + 8].view("<f4"), record[at + 8: at + 12].view("<u4")


def kv8_append(cache, k, v, block_table, seq_ids, positions, d):
    """The cache (uint8 [num_blocks, Hkv, bytes], changed in place) after an
    append of rows k, v [T, Hkv, d] (fp64 or fp32 numbers)."""
    value = kv8_code_values()
    rows = {}
    for t, (b, p) in enumerate(zip(seq_ids, positions)):
        if b >= 0:
            rows.setdefault(int(block_table[b][p // SLOTS]), []).append((int(p) % SLOTS, t))
    for phys, members in rows.items():
        for h in range(cache.shape[1]):
            record = cache[phys, h]
            scales, flags = _tail(record, d)
            begun = not any(s == 0 for s, _ in members)
            if not begun:
                record[2 * SLOTS * d + 8:] = 0
            for kind, x in ((0, k), (1, v)):
                codes = record[kind * SLOTS * d: (kind + 1) * SLOTS * d].reshape(SLOTS, d)
                need = kv8_scale([x[t, h] for _, t in members])
                had = float(scales[kind])
                if begun and 2.0 ** -64 <= had <= 2.0 ** 64:
                    now = max(had, need)
                    if now > had:
                        old = value[codes]
                        codes[:] = np.where(np.isnan(old), codes, kv8_codes(old * (had / now)))
                else:
                    now = need
                    codes[:] = 0
                    flags[0] &= ~np.uint32(0xFFFF << (16 * kind))
                for s, t in members:
                    codes[s] = kv8_codes(np.asarray(x[t, h], dtype=np.float64) / now)
                    bit = np.uint32(1 << (16 * kind + s))
                    flags[0] &= ~bit
                    if not np.all(np.isfinite(x[t, h])):
                        flags[0] |= bit
                scales[kind] = now
    return cache


def kv8_unpack(cache, d):
    """Every slot of a cache: fp64 (k, v), each [num_blocks, Hkv, 16, d], and
    which tokens are flagged, [num_blocks, Hkv, 16]."""
    cache = np.ascontiguousarray(cache)
    value, out = kv8_code_values(), []
    tail = np.ascontiguousarray(cache[..., 2 * SLOTS * d: 2 * SLOTS * d + 12]).view("<u4")
    scales = np.ascontiguousarray(tail[..., :2]).view("<f4").astype(np.float64)
    for kind in (0, 1):
        codes = cache[..., kind * SLOTS * d: (kind + 1) * SLOTS * d].reshape(cache.shape[:2] + (SLOTS, d))
        with np.errstate(invalid="ignore"):
            out.append(value[codes] * scales[..., kind, None, None])
    f = tail[..., 2, None]
    flagged = (((f >> np.arange(16, dtype=np.uint32)) | (f >> (16 + np.arange(16, dtype=np.uint32)))) & 1).astype(bool)
    return out[0], out[1], flagged


def prefill_paged_kv8(q, cache, block_table, seq_lens, scale, d):
    """q [S, Hq, N, d]: the last N tokens of each sequence attend to the tokens
    up to themselves.  fp64 (o, lse); a row of no token: 0 and -inf; a row that
    attends to a flagged token: NaN."""
    k, v, flagged = kv8_unpack(cache, d)
    S, Hq, N, _ = q.shape
    Hkv = cache.shape[1]
    o, lse = np.zeros(q.shape), np.full((S, Hq, N), -np.inf)
    for b in range(S):
        L = int(seq_lens[b])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            j = np.arange(L)
            at = (np.asarray(block_table)[b, j // SLOTS], g, j % SLOTS)
            keys, vals, bad = k[at], v[at], flagged[at]
            first = max(0, N - L)                    # rows before it belong to no token
            if first == N:
                continue
            see = np.arange(L)[None] <= np.arange(L - N + first, L)[:, None]
            x = np.where(see, scale * (np.asarray(q[b, h, first:], np.float64) @ np.nan_to_num(keys).T), -np.inf)
            m = x.max(-1, keepdims=True)
            p = np.exp(x - m)
            total = p.sum(-1, keepdims=True)
            spoilt = (see & bad).any(-1)
            o[b, h, first:] = np.where(spoilt[:, None], np.nan, p @ np.nan_to_num(vals) / total)
            lse[b, h, first:] = np.where(spoilt, np.nan, (m + np.log(total))[:, 0])
    return o, lse


def decode_paged_kv8(q, cache, block_table, seq_lens, scale, d):
    """q [S, Hq, d]: one query for each sequence, over all of its tokens."""
    o, lse = prefill_paged_kv8(q[:, :, None], cache, block_table, seq_lens, scale, d)
    return o[:, :, 0], lse[:, :, 0]
