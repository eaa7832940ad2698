"""Reference of the 4-bit paged KV cache — TEST INFRASTRUCTURE ONLY.

Every group of ``group`` consecutive elements of a key or value keeps
min = bf16(lowest), scale = bf16((highest - min) r), r the fp32 number
nearest to 1/15, and a code per element, (x - min) / scale to the nearest whole number (half to even) in
0 .. 15; it stands for code * scale + min.

A record holds the 16 token slots of one KV head of one block:
K codes [16][d/2] bytes, V codes [16][d/2], K parameters [16][d/group] words,
V parameters [16][d/group]; a parameter word has min in its low and scale in
its high 16 bits (bf16 both).  Codes are 4-bit cells, the low half of a byte
first; element e of a key is cell 8 ((d/32) c + w) + i + 4 h of its row with
e = 32 w + 8 i + 2 c + h, element e of a value is cell 8 ((d/64) r + w) + n
with e = r + 8 (8 w + n).  Written out cell by cell here.
"""

import numpy as np

from .definitions import decode_paged

SLOTS = 16


def bf16_bits(x):
    """Bits of fp32 values rounded to bf16 (nearest, ties to even; no NaN)."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint32)


def bf16_value(bits):
    return (np.asarray(bits, dtype=np.uint32) << 16).view(np.float32)


def kv4_record_bytes(d, group):
    return 2 * SLOTS * (d // 2) + 2 * SLOTS * (d // group) * 4


def kv4_quantise(x, group):
    """Rows x [..., d] fp32 (finite) -> (codes [..., d], words [..., d/group])."""
    x = np.asarray(x, dtype=np.float32)
    y = x.reshape(x.shape[:-1] + (-1, group))
    low_bits = bf16_bits(y.min(-1))
    low = bf16_value(low_bits)
    spread = np.maximum(y.max(-1) - low, np.float32(0))
    scale_bits = bf16_bits(spread * (np.float32(1) / np.float32(15)))
    scale_bits[scale_bits < 0x80] = 0
    scale = bf16_value(scale_bits)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((y - low[..., None]) / scale[..., None])
    codes = np.where(scale[..., None] > 0, np.clip(np.nan_to_num(q), 0, 15), 0).astype(np.uint8)
    return codes.reshape(x.shape), (scale_bits << 16) | low_bits


def kv4_values(codes, words, group):
    """The fp64 values of codes [..., d] with parameter words [..., d/group]."""
    scale = bf16_value(np.asarray(words) >> 16).astype(np.float64)
    low = bf16_value(np.asarray(words) & 0xFFFF).astype(np.float64)
    y = codes.reshape(codes.shape[:-1] + (-1, group)).astype(np.float64)
    return (y * scale[..., None] + low[..., None]).reshape(codes.shape)


def kv4_cell(kind, e, d):
    """Cell of element e in a key's (kind 0) or value's (kind 1) row."""
    if kind == 0:
        w, i, c, h = e // 32, e // 8 % 4, e // 2 % 4, e % 2
        return 8 * ((d // 32) * c + w) + i + 4 * h
    w, n, r = e // 64, e // 8 % 8, e % 8
    return 8 * ((d // 64) * r + w) + n


def _offsets(kind, d, group):
    codes = kind * SLOTS * (d // 2)
    params = 2 * SLOTS * (d // 2) + kind * SLOTS * (d // group) * 4
    return codes, params


def kv4_store(record, kind, slot, codes, words, d, group):
    """Writes one row into a record (uint8 array of kv4_record_bytes)."""
    base, par = _offsets(kind, d, group)
    for e in range(d):
        cell = kv4_cell(kind, e, d)
        at, shift = base + slot * (d // 2) + cell // 2, 4 * (cell % 2)
        record[at] = (int(record[at]) & (0xF0 >> shift)) | (int(codes[e]) << shift)
    n = d // group
    record[par + slot * n * 4: par + (slot + 1) * n * 4] = np.asarray(words, dtype="<u4").view(np.uint8)


def kv4_unpack(cache, d, group):
    """Every slot of a cache [num_blocks, Hkv, bytes]: fp64 (k, v), each
    [num_blocks, Hkv, 16, d]."""
    cache = np.ascontiguousarray(cache)
    out = []
    for kind in (0, 1):
        base, par = _offsets(kind, d, group)
        rows = cache[..., base: base + SLOTS * (d // 2)].reshape(cache.shape[:2] + (SLOTS, d // 2))
        cells = np.array([kv4_cell(kind, e, d) for e in range(d)])
        codes = (rows[..., cells // 2] >> (4 * (cells % 2))) & 15
        n = SLOTS * (d // group) * 4
        words = np.ascontiguousarray(cache[..., par: par + n]).view("<u4").reshape(cache.shape[:2] + (SLOTS, d // group))
        with np.errstate(invalid="ignore"):
            out.append(kv4_values(codes, words, group))
    return tuple(out)


def decode_paged_kv4(q, cache, block_table, seq_lens, scale, d, group):
    """attn_decode_paged over what a 4-bit cache stands for (fp64)."""
    k, v = kv4_unpack(cache, d, group)
    return decode_paged(q, k, v, block_table, seq_lens, scale)
