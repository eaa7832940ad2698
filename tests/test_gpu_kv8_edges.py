"""Attention over the 8-bit cache where it can go wrong at the edges of what it
accepts, against the fp64 oracle, held to the values that the call may use."""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import oracle
import workloads
from kv8_bounds import close_bound, compare_live, live_top
from parity import to64
from test_gpu_kv8_attention import DECODES, PREFILLS, case, decode, prefill, ways

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("lens,Hq,Hkv,d", DECODES)
def test_decode_beside_large_garbage(lens, Hq, Hkv, d):
    """Slots past the ends and unused blocks hold the largest numbers."""
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=len(lens) + Hq, garbage=0x7E)
    o, lse = decode(q, cache, table, sl)
    ref = oracle.decode_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,N,d", PREFILLS)
def test_prefill_beside_large_garbage(lens, Hq, Hkv, N, d):
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N, garbage=0x7E)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)
    assert attn.device_status() == 0


def flag(cache, table, b, p, h, kind, d):
    """A NaN in the key (kind 0) or value of head h of sequence b's token p."""
    rec = cache[table[b, p // 16].long(), h]
    rec[(16 * kind + p % 16) * d + p % d] = 0x7F
    word = rec[32 * d + 8: 32 * d + 12].view(torch.int32)
    word |= 1 << (16 * kind + p % 16) if 16 * kind + p % 16 < 31 else -2 ** 31


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,N", [(2, 2, 300), (3, 1, 200), (2, 1, 520)])
def test_flagged_tokens_where_the_query_tiles_end_apart(Hq, Hkv, N, d):
    """The two query tiles of 128 rows that a CTA works on see different numbers of
    key tiles.  Flags in the last key tile that the first sees, in its last key, just
    behind, in the second's last one, and in none."""
    first = 100 + 127                                # last key of the first query tile: of key tile 1 of 128
    flagged = [200, first, first + 1, 255, 256, 99 + min(N, 256), None, 100 + N - 1, 0]
    lens = [100 + N] * len(flagged)
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N)
    for b, p in enumerate(flagged):
        if p is not None:
            flag(cache, table, b, p, b % Hkv, b % 2, d)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)
    assert attn.device_status() == 0


def wide(i, kind):
    """log2 of block i's V scale."""
    return {"down": 64 if i < 9 else -64, "up": -64 if i < 9 else 64, "in turn": 64 if i % 2 else -64, "one": 64 if i == 9 else -64,
            "first": 64 if i == 0 else -64, "zeros": -64 if i % 3 else 60, "near": 36 if i % 2 else -64, "three": (-64, 0, 64)[i % 3],
            "small": -30 if i % 5 else -64}[kind]


@pytest.mark.parametrize("kind", ["down", "up", "in turn", "one", "first", "zeros", "near", "three", "small"])
@pytest.mark.parametrize("N,d", [(40, 128), (40, 64), (300, 64), (3, 128)])
def test_value_scales_from_one_end_of_their_range_to_the_other(kind, N, d):
    """Every V scale is accepted beside every other one: the weights of the tokens with
    small values, which dominate the softmax sum where those with large ones have the
    lower scores, are not lost.  ("zeros": blocks of no value at all have 2^-64.)"""
    Hq, Hkv = 2, 1
    lens = [420, 330]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N + d, N=N, garbage=None)
    for b in range(2):
        for i in range(-(-lens[b] // 16)):
            rec = cache[table[b, i].long(), 0]
            tail = rec[32 * d: 32 * d + 8].view(torch.float32)
            tail[0] *= 4.0                           # scores that differ by some ten log2 units
            tail[1] = 2.0 ** wide(i, kind)
            if kind == "zeros" and i % 3:
                rec[16 * d: 32 * d] = 0
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    q64, c = q.double().numpy(), cache.numpy()
    o_ref, lse_ref = oracle.prefill_paged_kv8(q64, c, table.numpy(), lens, d ** -0.5, d)
    # With keys four times as large as normalised ones the scores are off by under
    # 2^-10, and so is the LSE.
    lim = close_bound(q64, c, table.numpy(), lens, d ** -0.5, d, score=2.0 ** -10)
    for times in ways(2, Hq, Hkv, N, d):
        o, lse = prefill(args, times)
        err = np.abs(to64(o) - o_ref)
        lerr = np.abs(lse.double().cpu().numpy() - lse_ref).max()
        assert lerr <= 2.0 ** -10, "%d times: lse off by %.3g" % (times, lerr)
        assert np.all(err <= lim), "%d times: o at %.3g of its bound" % (times, (err / np.maximum(lim, 1e-300)).max())
    assert attn.device_status() == 0


def test_wide_value_scales_in_many_units():
    """More units to a CTA than its list of rows to be computed again is long."""
    d, Hq, Hkv, N = 64, 2, 2, 100
    lens = [33, 48, 20, 41, 32]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=4, N=N, garbage=None)
    for b in range(len(lens)):
        for i in range(-(-lens[b] // 16)):
            for h in range(Hkv):
                tail = cache[table[b, i].long(), h, 32 * d: 32 * d + 8].view(torch.float32)
                tail[0] *= 4.0
                tail[1] = 2.0 ** wide(i, "in turn")
    times = 70 * 152 // (len(lens) * Hkv) + 1
    assert attn.attn_prefill_paged_kv8_workspace_size(times * len(lens), Hq, Hkv, N, d) == 0
    q64, c = q.double().numpy(), cache.numpy()
    o_ref, lse_ref = oracle.prefill_paged_kv8(q64, c, table.numpy(), lens, d ** -0.5, d)
    lim = torch.from_numpy(close_bound(q64, c, table.numpy(), lens, d ** -0.5, d, score=2.0 ** -10)).to(DEV)
    o, lse = attn.attn_prefill_paged_kv8(*(x.to(DEV).repeat(times, *[1] * (x.dim() - 1)) if x is not cache else x.to(DEV)
                                           for x in (q, cache, table, sl)))
    torch.cuda.synchronize()
    err = (o.double().view(times, *o_ref.shape) - torch.from_numpy(o_ref).to(DEV)).abs()
    lse, ref = lse.double().view(times, *lse_ref.shape), torch.from_numpy(lse_ref).to(DEV)
    none = torch.isneginf(ref)
    assert torch.all(torch.isneginf(lse) == none) and torch.all(err <= lim)
    assert ((lse - ref).abs()[:, ~none] <= 2.0 ** -10).all() and attn.device_status() == 0


def in_tiles(S, Hq, Hkv, N, d):
    return attn.attn_prefill_paged_kv8_workspace_size(S, Hq, Hkv, N, d) == 0


def along(L, d, e, w, N, vscale):
    """Keys of one sequence along a vector of signs, of sizes w (one head), queries 2^e
    of it: all products and sums of a score are exact."""
    table, _, _, nb = workloads.token_map([0], [L], 1)
    cache = workloads.kv8_cache(nb, 1, attn.kv8_record_bytes(d), d, 2)
    sign = torch.where(torch.rand(d, generator=torch.Generator().manual_seed(5)) < 0.5, -1.0, 1.0)
    codes = (torch.tensor(w)[:, None] * sign).to(torch.float8_e4m3fn).view(torch.uint8)
    for p in range(L):
        rec = cache[table[0, p // 16].long(), 0]
        rec[p % 16 * d: (p % 16 + 1) * d] = codes[p]
        rec[32 * d: 32 * d + 8].view(torch.float32)[:] = torch.tensor([1.0, vscale(p // 16)])
    q = (sign * 2.0 ** e).to(torch.bfloat16).expand(1, 2, N, d).contiguous()
    return q, cache, table, torch.tensor([L], dtype=torch.int32)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("N", [1, 3, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_every_size(d, N, sign):
    """One key weighs more than all others by some 2^-5 of scores of 2^14 .. 2^94 log2
    units, of either sign: o is its value.  (Numerators rounded to 11 bits and o to bf16;
    a score of exact sums is off by its three products' roundings, and the LSE by two
    more: 5 2^-24 of it and the sum's 2^-24.  In tiles NaN from 2^40 on.)"""
    L = 200
    size = [1.0 + (i * 7 % 5) / 8 for i in range(L)] if sign > 0 else [1.25 + (i * 7 % 5) / 8 for i in range(L)]
    size[50], size[120] = (1.625, 1.75) if sign > 0 else (1.125, 1.0)
    for e in (10, 14, 18, 20, 21, 22, 23, 24, 25, 27, 29, 31, 32, 33, 36, 45, 60, 90):
        q, cache, table, sl = along(L, d, e, [sign * s for s in size], N, lambda i: 2.0 ** (i % 4 - 6))
        o_ref, lse_ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), [L], d ** -0.5, d)
        for times in ways(1, 2, 1, N, d):
            o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
            if np.abs(lse_ref).min() / np.log(2) >= 2.0 ** 40 and in_tiles(times, 2, 1, N, d):
                assert torch.isnan(o).all() and torch.isnan(lse).all()
                continue
            assert np.all(np.abs(to64(o) - o_ref) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(o_ref)), (e, times)
            assert np.all(np.abs(lse.double().cpu().numpy() / lse_ref - 1) <= 6 * 2.0 ** -24), (e, times)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N", [1, 3, 64])
def test_the_same_large_score_twice(N):
    """Two keys of the same score, the largest, beside V scales that differ: the mean of
    their values."""
    L, d = 200, 128
    size = [1.0] * L
    size[50] = size[120] = 1.75
    for e in (24, 28, 34):
        q, cache, table, sl = along(L, d, e, size, N, lambda i: 2.0 ** (i % 4 - 6))
        o_ref, lse_ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), [L], d ** -0.5, d)
        v = np.abs(oracle.kv8_unpack(cache.numpy(), d)[1]).max()
        for times in ways(1, 2, 1, N, d):
            o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
            assert np.all(np.abs(to64(o) - o_ref) <= 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -11 * v), (e, times)
            assert np.all(np.abs(lse.double().cpu().numpy() / lse_ref - 1) <= 6 * 2.0 ** -24), (e, times)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N", [1, 3, 64])
@pytest.mark.parametrize("d", [64, 128])
def test_a_score_of_zero_beside_scores_beyond_fp32(d, N):
    """A key of zeros in a block of the largest scale, under queries of 2^90: the others'
    scores are minus infinity in fp32, and o is its value."""
    L = 40
    size = [-1.0] * L
    size[20] = 0.0
    q, cache, table, sl = along(L, d, 90, size, N, lambda i: 2.0 ** -6)
    cache[:, :, 32 * d: 32 * d + 4].view(torch.float32)[:] = 2.0 ** 64
    sees = np.arange(L - N, L) >= 20
    v = oracle.kv8_unpack(cache.numpy(), d)[1][table[0, 1], 0, 4]
    for times in ways(1, 2, 1, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        o, lse = to64(o)[:, :, sees], lse.double().cpu().numpy()[:, :, sees]
        assert np.all(np.abs(o - v) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(v)) and np.all(lse == 0.0), times
    assert attn.device_status() == 0


def without(q, cache, table, lens, missing, d):
    """The oracle's o and LSE where the blocks `missing` of each sequence are left out."""
    k, v, _ = oracle.kv8_unpack(cache, d)
    S, Hq, N, _ = q.shape
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(S):
        j = np.array([p for p in range(lens[b]) if p // 16 not in missing[b]], dtype=int)
        for h in range(Hq):
            g = h // (Hq // cache.shape[1])
            keys, vals = (x[np.asarray(table)[b, j // 16], g, j % 16] for x in (k, v))
            for i in range(N):
                see = j <= lens[b] - N + i
                if see.any():
                    x = d ** -0.5 * (keys[see] @ q[b, h, i])
                    w = np.exp(x - x.max())
                    o[b, h, i], lse[b, h, i] = w @ vals[see] / w.sum(), x.max() + np.log(w.sum())
    return o, lse


@pytest.mark.parametrize("Hq,Hkv,N,d", [(4, 2, 64, 64), (2, 1, 40, 128), (2, 2, 270, 64), (3, 3, 2, 128)])
def test_blocks_outside_the_pool_are_left_out(Hq, Hkv, N, d):
    """In either way through a batch: single blocks, the whole first tile of keys, all of
    them, the last one."""
    lens = [300, 300, 290, 100, 280, 333]
    missing = [{1, 3, 17}, set(range(8)), set(range(19)), {0, 6}, {0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11}, set()]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N)
    bad = table.clone()
    for b, gone in enumerate(missing):
        for i in gone:
            bad[b, i] = (-1, cache.shape[0], 2 ** 31 - 1)[i % 3]
    ref = without(q.double().numpy(), cache.numpy(), table.numpy(), lens, missing, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, bad, sl)], times)
        assert attn.device_status() == attn.ATTN_DEV_BAD_BLOCK
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)


@pytest.mark.parametrize("N", [3, 64])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [0, 14, 24])
def test_blocks_of_zeros_that_were_never_written(N, d, size):
    """Keys and values of zero, whatever scale the zeros are: blocks of a pool as it is
    allocated, in either way through a batch."""
    Hq, Hkv = 2, 1
    lens = [200, 150, 90]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N, garbage=None)
    cache[..., 32 * d + 4: 32 * d + 8] = (cache[..., 32 * d + 4: 32 * d + 8].contiguous().view(torch.float32)
                                          * 2.0 ** size).view(torch.uint8)
    for b, i in ((0, 0), (0, 5), (1, 2), (1, 3), (2, 5)):
        cache[table[b, i].long()] = 0
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(3, Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)
    assert attn.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_are_not_in_use(d):
    """Queries of any bits at all (rows of padding that nobody has written) beside others,
    in tiles: the others are what they are beside zeros (to the bounds of two results: 32
    rows may have their stabilisers moved together), and the call takes no longer (such
    scores are beyond those that are computed key by key)."""
    Hq, Hkv, N, S = 4, 2, 300, 24
    lens = [2000] * S
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=3, N=N)
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    assert in_tiles(S, Hq, Hkv, N, d)
    junk = torch.randint(-2 ** 15, 2 ** 15, (S, Hq, 200, d), generator=torch.Generator().manual_seed(1)).to(torch.int16)
    runs = []
    for fill in (torch.zeros(S, Hq, 200, d, dtype=torch.bfloat16), junk.view(torch.bfloat16)):
        args[0][:, :, :200] = fill.to(DEV)
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            o, lse = attn.attn_prefill_paged_kv8(*args)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        runs.append((o[:, :, 200:].clone(), lse[:, :, 200:].clone(), min(times)))
    (o, lse, _), (o2, lse2, _) = runs
    top = live_top(cache.numpy(), table.numpy(), lens, d).max()
    assert torch.isfinite(o).all() and attn.device_status() == 0
    assert torch.all((o.float() - o2.float()).abs() <= 2 * (2.0 ** -8 * o.float().abs() + 2.0 ** -10 * top))
    assert torch.all((lse - lse2).abs() <= 2.0 ** -15)
    assert runs[1][2] < 3 * runs[0][2], runs
