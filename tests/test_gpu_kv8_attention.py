"""Attention over the 8-bit paged cache on the GPU, against the fp64 oracle:
one query per sequence, and the last N tokens of each.

Bounds.  q, codes and scales enter exactly and the scores are fp32 sums: with
these inputs their error is under 2^-12, and 2 2^-12 of max|V| in O.  Numerators
are rounded to 11 bits: 2^-11 of max|V|.  Then O's own rounding to bf16, 2^-8 |O|.  The LSE uses the unrounded numerators: 2^-16 covers the fp32
sums, relative to its size where that is more than 16.
"""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import oracle
import workloads
from parity import to64
from test_gpu_rope import map_case, randn, views

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def case(lens, Hq, Hkv, d, seed, N=None, garbage=0xFF):
    """Queries, a cache whose slots past the ends (and unused blocks) are
    garbage, table, lengths (CPU)."""
    table, ids, pos, nb = workloads.token_map([0] * len(lens), lens, seed, spare_blocks=2)
    cache = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed + 1)
    if garbage is not None:
        used = set()
        for b, n in enumerate(lens):
            for i in range(-(-n // 16)):
                used.add(int(table[b, i]))
                for slot in range(max(0, n - 16 * i), 16):
                    for kind in (0, 1):
                        at = (16 * kind + slot) * d
                        cache[table[b, i].long(), :, at: at + d] = garbage
        for p in set(range(nb)) - used:
            cache[p] = garbage
    shape = (len(lens), Hq, d) if N is None else (len(lens), Hq, N, d)
    return randn(seed + 2, *shape), cache, table, torch.tensor(lens, dtype=torch.int32)


def prefill(args, times=1, **kw):
    """The call on GPU tensors, its batch `times` over: the copies come out alike."""
    q, cache, table, lens = args
    S = q.shape[0]
    o, lse = attn.attn_prefill_paged_kv8(q.repeat(times, 1, 1, 1), cache, table.repeat(times, 1), lens.repeat(times), **kw)
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0))
    for i in range(1, times):
        assert same(o[i * S: i * S + S], o[:S]) and same(lse[i * S: i * S + S], lse[:S])
    return o[:S], lse[:S]


def ways(S, Hq, Hkv, N, d):
    """How often a batch has to be repeated for each way through it: passes over the
    cache, which use a workspace, and tiles of query rows, for many rows in all,
    which use none."""
    found = {}
    for r in list(range(1, 25)) + [50, 100, 200, 500]:
        found.setdefault(attn.attn_prefill_paged_kv8_workspace_size(S * r, Hq, Hkv, N, d) == 0, r)
    return list(found.values())


def compare(o, lse, ref, cache, d, what=""):
    o_ref, lse_ref = ref
    o, lse = to64(o), lse.double().cpu().numpy()
    nan = np.isnan(lse_ref)
    assert np.array_equal(np.isnan(lse), nan) and np.array_equal(np.isnan(o).any(-1), nan), what
    assert np.array_equal(np.isnan(o).all(-1), nan), what
    none = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), none) and np.all(o[none] == 0), what
    top = max(np.nanmax(np.abs(np.where(np.isfinite(x), x, 0))) for x in oracle.kv8_unpack(cache, d)[1:2])
    fine = ~nan & ~none
    lim = 2.0 ** -8 * np.abs(o_ref[fine]) + 2.0 ** -10 * top
    err = np.abs(o[fine] - o_ref[fine])
    assert np.all(err <= lim), "%s: O at %.3g of its bound" % (what, (err / lim).max())
    lerr = np.abs(lse[fine] - lse_ref[fine])
    assert np.all(lerr <= 2.0 ** -16 * np.maximum(1, np.abs(lse_ref[fine]) / 16)), "%s: LSE off by %.3g" % (what, lerr.max())


def decode(q, cache, table, lens, scale=None, **kw):
    o, lse = attn.attn_decode_paged_kv8(*(x.to(DEV) for x in (q, cache, table, lens)), scale=scale, **kw)
    torch.cuda.synchronize()
    return o, lse


DECODES = [  # lens, Hq, Hkv, d
    ([1], 1, 1, 64), ([100], 12, 2, 128), ([16, 17, 15, 0, 33], 6, 3, 64), ([0, 0, 0], 4, 2, 128),
    ([700, 1, 250, 64], 16, 1, 128), ([300, 0, 31], 32, 2, 64), ([1000, 2000], 5, 1, 128), ([40] * 70, 8, 8, 64),
    ([20000, 3], 12, 2, 128), ([3, 9000, 0, 5000], 24, 2, 64), ([123] * 9, 10, 2, 128), ([5, 48, 512], 9, 1, 64),
]


@pytest.mark.parametrize("lens,Hq,Hkv,d", DECODES)
@pytest.mark.parametrize("ctas", [0, 1, 7])
def test_decode_against_the_oracle(lens, Hq, Hkv, d, ctas):
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=len(lens) + Hq)
    scale = d ** -0.5
    attn.set_decode_max_ctas(ctas)
    try:
        o, lse = decode(q, cache, table, sl)
    finally:
        attn.set_decode_max_ctas(0)
    assert attn.device_status() == 0
    ref = oracle.decode_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, scale, d)
    compare(o, lse, ref, cache.numpy(), d)


PREFILLS = [  # lens, Hq, Hkv, N, d
    ([1], 1, 1, 1, 64), ([5], 4, 2, 2, 128), ([3, 0, 40, 7], 12, 2, 4, 128), ([100, 2, 33], 6, 3, 5, 64),
    ([700, 90], 8, 1, 16, 128), ([50, 51, 0, 1], 4, 4, 50, 64), ([260, 100, 300], 6, 2, 130, 128),
    ([400, 128, 129], 3, 1, 128, 64), ([513, 17], 5, 5, 257, 128), ([2000], 16, 2, 3, 128), ([1500, 30], 20, 1, 1, 64),
    ([1029, 1300], 2, 1, 1029, 64), ([200, 600, 50], 32, 2, 7, 128), ([64] * 20, 12, 2, 2, 128),
]


@pytest.mark.parametrize("lens,Hq,Hkv,N,d", PREFILLS)
@pytest.mark.parametrize("garbage", [0xFF, 0x7E])
def test_prefill_against_the_oracle(lens, Hq, Hkv, N, d, garbage):
    """Rows of sequences shorter than N among them; garbage past the ends is NaN
    or the largest numbers."""
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N, garbage=garbage)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        assert attn.device_status() == 0
        compare(o, lse, ref, cache.numpy(), d, what="%d times" % times)


@pytest.mark.parametrize("ctas", [1, 7])
@pytest.mark.parametrize("d,N", [(128, 9), (64, 20)])
def test_passes_over_few_ctas(ctas, d, N):
    """Several groups of rows of several sequences, split over a few CTAs."""
    lens = [700, 0, 33, 1200]
    q, cache, table, sl = case(lens, 12, 2, d, seed=2, N=N)
    attn.set_decode_max_ctas(ctas)
    try:
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)])
    finally:
        attn.set_decode_max_ctas(0)
    assert attn.device_status() == 0
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    compare(o, lse, ref, cache.numpy(), d)


def test_the_two_ways_are_both_tested():
    both = [c for c in PREFILLS if len(ways(len(c[0]), *c[1:])) == 2]
    assert {c[4] for c in both} == {64, 128} and {c[3] >= 256 for c in both} == {True, False}


def test_a_query_alone_is_a_decode():
    lens = [100, 0, 1, 517]
    q, cache, table, sl = case(lens, 12, 2, 128, seed=3)
    a = decode(q, cache, table, sl)
    b = attn.attn_prefill_paged_kv8(*(x.to(DEV) for x in (q[:, :, None], cache, table, sl)))
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0][:, :, 0]) and torch.equal(a[1], b[1][:, :, 0])


@pytest.mark.parametrize("N", [None, 4, 60])
@pytest.mark.parametrize("d", [64, 128])
def test_flagged_tokens(N, d):
    """A row that attends to a token with a NaN in that head is NaN, o and lse;
    rows that do not see it, other heads and other sequences are as ever."""
    Hq, Hkv = 6, 3
    lens = [100, 61, 60, 200]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=9, N=N)
    for b, p, h, kind in ((0, 99, 0, 0), (1, 10, 1, 1), (2, 58, 2, 1), (2, 40, 0, 0), (3, 150, 1, 1), (3, 170, 1, 0)):
        rec = cache[table[b, p // 16].long(), h]
        rec[(16 * kind + p % 16) * d + 5] = 0x7F
        word = rec[32 * d + 8: 32 * d + 12].view(torch.int32)
        word |= 1 << (16 * kind + p % 16)
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    f = oracle.decode_paged_kv8 if N is None else oracle.prefill_paged_kv8
    ref = f(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    assert np.isnan(ref[1]).any() and not np.isnan(ref[1]).all()
    for times in (0,) if N is None else ways(4, Hq, Hkv, N, d):
        o, lse = attn.attn_decode_paged_kv8(*args) if N is None else prefill(args, times)
        torch.cuda.synchronize()
        compare(o, lse, ref, cache.numpy(), d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N,times", [(None, 0), (3, 1), (64, 1), (64, 50)])
def test_bad_blocks_and_lengths_are_reported(N, times):
    """A block outside the pool counts as keys and values of zero in tiles, and
    is left out by the others; a length outside the table is clamped.  What is
    beside them is as ever."""
    d, Hq, Hkv = 64, 4, 2
    lens = [90, 50, 200]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=5, N=N)
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    call = attn.attn_decode_paged_kv8 if N is None else lambda *x: prefill(x, times)
    good, _ = call(*args)
    bad = table.clone()
    bad[0, 1], bad[0, 3] = cache.shape[0], -1
    got, _ = call(args[0], args[1], bad.to(DEV), args[3])
    torch.cuda.synchronize()
    assert attn.device_status() == attn.ATTN_DEV_BAD_BLOCK
    assert torch.equal(got[1:], good[1:]) and torch.isfinite(got[0]).all()
    wrong = sl.clone()
    wrong[1], wrong[2] = -3, 16 * table.shape[1] + 1
    got, _ = call(args[0], args[1], args[2], wrong.to(DEV))
    torch.cuda.synchronize()
    assert attn.device_status() & attn.ATTN_DEV_BAD_SEQLEN
    assert torch.equal(got[0], good[0])


@pytest.mark.parametrize("N", [None, 2, 33, 66])
@pytest.mark.parametrize("qs,ks,vs", [(1.0, 0, 0), (2.0 ** 20, -30, 40), (2.0 ** -30, 20, -60), (1e-36, 64, 64), (0.0, 0, 0),
                                      (6.0, 1, -3)])
def test_values_of_every_size(N, qs, ks, vs):
    d, Hq, Hkv = 64, 4, 2
    lens = [300, 37]
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=6, N=N, garbage=None)
    q = (q.float() * qs).to(BF)
    tail = cache[..., 32 * d: 32 * d + 8].contiguous().view(torch.float32)
    tail = tail * 256 / 8 * torch.tensor([2.0 ** ks, 2.0 ** vs])
    tail = tail.clamp(2.0 ** -64, 2.0 ** 64)
    cache[..., 32 * d: 32 * d + 8] = tail.contiguous().view(torch.uint8)
    scale = d ** -0.5 * (2.0 ** 10 if qs == 2.0 ** 20 else 1.0)
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    f = oracle.decode_paged_kv8 if N is None else oracle.prefill_paged_kv8
    ref = f(q.double().numpy(), cache.numpy(), table.numpy(), lens, np.float32(scale).astype(np.float64), d)
    for times in (0,) if N is None else ways(2, Hq, Hkv, N, d):
        o, lse = attn.attn_decode_paged_kv8(*args, scale=scale) if N is None else prefill(args, times, scale=scale)
        torch.cuda.synchronize()
        compare(o, lse, ref, cache.numpy(), d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N", [None, 2, 40])
def test_scores_that_jump(N):
    """Keys along q whose scores climb by hundreds of log2 units block by block,
    and fall again; scales of V that differ by 2^30 from block to block."""
    d, Hq, Hkv = 128, 2, 1
    L = 900
    q, cache, table, sl = case([L], Hq, Hkv, d, seed=8, N=N, garbage=None)
    q = q[:, :1].expand_as(q).contiguous()
    nblk = -(-L // 16)
    e = torch.zeros(nblk)
    e[10:14], e[20], e[40:] = torch.tensor([1.0, 3.0, 5.0, 5.0]), 7.0, 2.0
    for i in range(nblk):
        rec = cache[table[0, i].long(), 0]
        t = rec[32 * d: 32 * d + 8].view(torch.float32)
        t[0] *= 2.0 ** float(e[i])
        t[1] *= 2.0 ** (30 * (i % 3 - 1))
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    f = oracle.decode_paged_kv8 if N is None else oracle.prefill_paged_kv8
    o_ref, lse_ref = f(q.double().numpy(), cache.numpy(), table.numpy(), [L], d ** -0.5, d)
    # Scores up to some 1000 (their fp32 sums are off by up to 128 2^-24 of the
    # sum of their terms' sizes, 2^-9 here), so weights by 2^-8.
    top = np.abs(oracle.kv8_unpack(cache.numpy(), d)[1]).max()
    for times in (0,) if N is None else ways(1, Hq, Hkv, N, d):
        o, lse = attn.attn_decode_paged_kv8(*args) if N is None else prefill(args, times)
        torch.cuda.synchronize()
        assert np.all(np.abs(to64(o) - o_ref) <= 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -6 * top)
        assert np.all(np.abs(lse.double().cpu().numpy() - lse_ref) <= 2.0 ** -9)
    assert attn.device_status() == 0


@pytest.mark.parametrize("N", [None, 3, 64])
def test_workspaces_levels_streams_and_graphs(N):
    """Garbage and reused workspaces, both early-plan levels, given outputs, a
    given stream, a captured graph replayed on other contents: the same bits."""
    d, Hq, Hkv = 128, 12, 2
    more = 2 if N == 64 else 1                       # (enough for tiles)
    lens = [4000, 17, 0, 900, 900, 2500] * more
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=4, N=N)
    args = [x.to(DEV) for x in (q, cache, table, sl)]
    call = attn.attn_decode_paged_kv8 if N is None else attn.attn_prefill_paged_kv8
    need = (attn.attn_decode_paged_kv8_workspace_size(len(lens), Hq, Hkv, d) if N is None
            else attn.attn_prefill_paged_kv8_workspace_size(len(lens), Hq, Hkv, N, d))
    assert (need == 0) == (N == 64)
    o, lse = call(*args)
    for fill in (0, 0xFF, 0x5A):
        ws = torch.full((need + 16,), fill, dtype=torch.uint8, device=DEV)
        for level in (0, 1, 2):
            attn.set_decode_early_plan(level)
            try:
                got = call(*args, workspace=ws, o=torch.full_like(o, 3.0), lse=torch.full_like(lse, 3.0))
            finally:
                attn.set_decode_early_plan(0)
            assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(*args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], o) and call(*args, return_lse=False)[1] is None
    q2 = (args[0] * 0.5).clone()
    ws, out, lse2 = torch.empty(need, dtype=torch.uint8, device=DEV), torch.zeros_like(o), torch.zeros_like(lse)
    live, lens2 = args[0].clone(), args[3].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(live, *args[1:3], lens2, workspace=ws, o=out, lse=lse2)
        call(live, *args[1:3], lens2, workspace=ws, o=out, lse=lse2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o) and torch.equal(lse2, lse)
    live.copy_(q2)
    lens2.copy_(torch.tensor([64, 3000, 5, 0, 1, 16] * more, dtype=torch.int32).clamp(max=sl))
    graph.replay()
    want = call(q2, *args[1:3], lens2)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse2, want[1])
    assert attn.device_status() == 0


def test_a_prompt_in_chunks_then_drafts_then_steps():
    """The operators as they are used together: a prompt goes in by chunks, each
    attending to the cache it has just been put into, then draft tokens that are
    verified and partly taken back, then single tokens.  Every step against the
    oracle on the cache as it then is."""
    d, Hq, Hkv, S = 128, 6, 2, 3
    f = workloads.rope_inv_freq(d).to(DEV)
    nb = 60
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    table = perm.view(S, 20)
    kv = torch.full((nb, Hkv, attn.kv8_record_bytes(d)), 0xFF, dtype=torch.uint8, device=DEV)
    at = [0] * S
    seed = 0
    for N in (40, 100, 4, 4, 1, 1):
        seed += 1
        ids = torch.arange(S, dtype=torch.int32).repeat_interleave(N)
        pos = torch.cat([torch.arange(a, a + N) for a in at]).to(torch.int32)
        x = randn(seed, S * N, (Hq + 2 * Hkv) * d).to(DEV)
        turned = attn.kv8_append_paged(*views(x, Hq, Hkv, d), kv, table.to(DEV), ids.to(DEV), pos.to(DEV), inv_freq=f)
        at = [a + N for a in at]
        lens = torch.tensor(at, dtype=torch.int32)
        q = turned.view(S, N, Hq, d).transpose(1, 2).contiguous()
        if N == 1:
            o, lse = attn.attn_decode_paged_kv8(q[:, :, 0].contiguous(), kv, table.to(DEV), lens.to(DEV))
            o, lse = o[:, :, None], lse[:, :, None]
        else:
            o, lse = attn.attn_prefill_paged_kv8(q, kv, table.to(DEV), lens.to(DEV))
        torch.cuda.synchronize()
        ref = oracle.prefill_paged_kv8(to64(q), kv.cpu().numpy(), table.numpy(), at, d ** -0.5, d)
        compare(o, lse, ref, kv.cpu().numpy(), d, what="N %d" % N)
        if N == 4:                                   # some drafts are not taken
            at = [a - b for a, b in zip(at, (0, 1, 3))]
    assert attn.device_status() == 0


def test_cache_beyond_32_bits():
    d, Hq, Hkv = 128, 16, 8
    rec = attn.kv8_record_bytes(d)
    nb = 5 * 2 ** 30 // (Hkv * rec)
    small = workloads.kv8_cache(4, Hkv, rec, d, seed=3)
    kv = torch.zeros(nb, Hkv, rec, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[0, nb - 1, 2 ** 32 // (Hkv * rec), nb // 2]], dtype=torch.int32)
    kv[table[0].long().to(DEV)] = small.to(DEV)
    q = randn(4, 1, Hq, 40, d)
    lens = torch.tensor([61], dtype=torch.int32)
    for n in (1, 2, 40):
        x = q[:, :, :n].contiguous()
        ref = oracle.prefill_paged_kv8(x.double().numpy(), small.numpy(), np.array([[0, 1, 2, 3]]), [61], d ** -0.5, d)
        for times in ways(1, Hq, Hkv, n, d):
            o, lse = prefill([y.to(DEV) for y in (x, kv, table, lens)], times)
            compare(o, lse, ref, small.numpy(), d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("S,Hq,Hkv,N,d", [(300, 4, 2, 64, 64), (260, 2, 1, 300, 128), (250, 1, 1, 1250, 64)])
def test_more_sequences_and_query_blocks_than_are_ordered(S, Hq, Hkv, N, d):
    """In tiles, beyond the numbers of sequences and of query blocks that the kernel
    orders by their cost; most sequences shorter than their N rows."""
    lens = [(37 * i) % 41 for i in range(S)]
    lens[7], lens[S - 1] = 333, 130
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N)
    assert attn.attn_prefill_paged_kv8_workspace_size(S, Hq, Hkv, N, d) == 0
    o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)])
    assert attn.device_status() == 0
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    compare(o, lse, ref, cache.numpy(), d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [0, 1])
def test_every_code(kind, d):
    """Keys (or values) that take every code in every dimension.  A row that sees
    one token has its value, rounded to bf16, which holds every e4m3 number."""
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    L = len(codes)
    N, Hq = 260, 2
    table, _, _, nb = workloads.token_map([0], [L], 5)
    cache = workloads.kv8_cache(nb, 1, attn.kv8_record_bytes(d), d, 6)
    for p in range(L):
        at = (16 * kind + p % 16) * d
        cache[table[0, p // 16].long(), 0, at: at + d] = codes[(p + torch.arange(d)) % L]
    q = randn(7, 1, Hq, N, d)
    sl = torch.tensor([L], dtype=torch.int32)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), [L], d ** -0.5, d)
    for times in ways(1, Hq, 1, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare(o, lse, ref, cache.numpy(), d)
        # The row that sees the first token alone.
        assert torch.equal(o[0, :, N - L].cpu(), torch.from_numpy(ref[0][0, :, N - L]).to(BF))
    assert attn.device_status() == 0
