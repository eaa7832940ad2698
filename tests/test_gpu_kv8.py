"""The 8-bit paged cache on the GPU: append and read-back against the oracle's
record format.

Values without rotation reach the quantiser exactly, and its steps are exact
products with powers of two and one rounding: records equal the oracle's byte
for byte.  Rotated keys are those of the fp32 formula (cos and sin rounded from
64 bits, products and sums rounded one by one).
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


def dev(*xs):
    return [x.to(DEV) for x in xs]


def append_both(cache, k, v, table, ids, pos, d, **kw):
    """The same append by the kernel and by the oracle; the records' bytes."""
    kv = torch.as_tensor(cache).to(DEV)
    attn.kv8_append_paged(None, *dev(k, v), kv, *dev(table, ids, pos), **kw)
    torch.cuda.synchronize()
    want = oracle.kv8_append(np.array(cache), k.double().numpy(), v.double().numpy(), table.numpy(), ids.numpy(),
                             pos.numpy(), d)
    return kv.cpu().numpy(), want


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("ctx,new", [([0], [1]), ([0, 13, 40, 5], [1, 37, 9, 3]), ([15, 16, 17, 0], [1, 16, 15, 32]),
                                     ([0, 700, 3], [300, 5, 1])])
def test_rows_are_the_oracles_bytes(d, Hkv, ctx, new):
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, 2, Hkv, d, 41, padding=3)
    k, v = k.clone(), v.clone()
    T = int((ids >= 0).sum())
    gen = torch.Generator().manual_seed(5)
    grow = torch.exp2(torch.randint(-3, 6, (ids.numel(), Hkv, 1), generator=gen).float())
    k *= grow.to(BF)                               # many scales have to grow
    v *= (grow / 1024).to(BF)
    k[0, 0] = 0.0
    v[T - 1, 0, ::3] *= 2.0 ** -12                 # subnormal codes
    rec = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2)
    got, want = append_both(rec, k, v, table, ids, pos, d)
    assert attn.device_status() == 0
    assert np.array_equal(got, want)
    kv = torch.tensor(got, device=DEV)
    k64, v64, _ = oracle.kv8_unpack(got, d)
    rk, rv = attn.kv8_read_paged(kv, *dev(table, ids[:T], pos[:T]), d)
    torch.cuda.synchronize()
    at = table[ids[:T].long(), (pos[:T] // 16).long()].long().numpy(), pos[:T].numpy() % 16
    for out, ref in ((rk, k64), (rv, v64)):
        assert np.array_equal(to64(out), ref[at[0], :, at[1]])


@pytest.mark.parametrize("d", [64, 128])
def test_every_half_way_value_goes_to_the_even_code(d):
    """All values half-way between two codes (they have 5 bits: exact in bf16),
    times scales of every size."""
    vals = oracle.kv8_code_values()[:127]
    mid = np.concatenate([(vals[1:] + vals[:-1]) / 2, -(vals[1:] + vals[:-1]) / 2])
    T, Hkv = 32, 2
    gen = np.random.default_rng(3)
    x = gen.choice(mid, (T, Hkv, d))
    x[:, :, 0] = 448.0
    x *= 2.0 ** gen.integers(-60, 60, (2, 1, Hkv, 1)).repeat(16, 1).reshape(T, Hkv, 1)
    x = torch.tensor(x).to(BF)
    table = torch.arange(2, dtype=torch.int32)[None]
    pos = torch.arange(T, dtype=torch.int32)
    cache = np.zeros((2, Hkv, attn.kv8_record_bytes(d)), np.uint8)
    got, want = append_both(cache, x, x, table, torch.zeros_like(pos), pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0


def test_scales_at_the_ends_of_their_range():
    d, Hkv = 64, 1
    tops = [0.0, 1e-38, 2.0 ** -64 * 448, 2.0 ** -56, 448.0, 449.0, 2.0 ** 64 * 448, 3e38, 2.0 ** 70]
    tops = torch.tensor(tops).to(BF)
    x = randn(3, len(tops) * 16, Hkv, d).float().clamp(-1, 1) * tops.float().repeat_interleave(16)[:, None, None]
    x = x.to(BF)
    x[::16, 0, 0] = tops
    T = x.shape[0]
    table = torch.arange(len(tops), dtype=torch.int32)[None]
    pos = torch.arange(T, dtype=torch.int32)
    cache = np.full((len(tops), Hkv, attn.kv8_record_bytes(d)), 0xAB, np.uint8)      # garbage that is begun anew
    got, want = append_both(cache, x, x, table, torch.zeros_like(pos), pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0


@pytest.mark.parametrize("garbage", [0x00, 0x7F, 0xFF, 0x3C])
def test_a_block_never_begun(garbage):
    """A row for another slot than the first, in a block whose scales are none:
    the slots not written become zeros.  (The last one has scales of 2^-6: there
    the codes are kept.)"""
    d = 128
    table = torch.tensor([[1]], dtype=torch.int32)
    pos = torch.tensor([4, 5, 6], dtype=torch.int32)
    x = randn(8, 3, 2, d) * 4096
    cache = np.full((3, 2, attn.kv8_record_bytes(d)), garbage, np.uint8)
    if garbage == 0x3C:
        cache.view("<f4")[..., 8 * d: 8 * d + 2] = 2.0 ** -6
    got, want = append_both(cache, x, x, table, torch.zeros_like(pos), pos, d)
    n = 32 * d + 12                                # (what follows the flags is not the row's)
    assert np.array_equal(got[..., :n], want[..., :n]) and np.array_equal(got[::2], cache[::2])


def test_elements_that_are_not_finite_are_flagged_and_alone():
    d, Hkv = 128, 3
    ctx, new = [0, 9], [40, 30]
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, 2, Hkv, d, 17)
    k, v = k.clone(), v.clone()
    k[3, 0, 5], k[17, 1, 127], v[3, 0, 0], v[50, 2, 64] = float("nan"), float("inf"), float("-inf"), float("nan")
    k[44, 0], v[69, 1] = float("nan"), float("inf")
    rec = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2)
    got, want = append_both(rec, k, v, table, ids, pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0
    assert oracle.kv8_unpack(got, d)[2].sum() == 5           # (row 3's key and value are one token's)
    # Written again with numbers, the flags go.
    k[torch.isnan(k) | torch.isinf(k)] = 1.0
    v[torch.isnan(v) | torch.isinf(v)] = 1.0
    got, want = append_both(got, k, v, table, ids, pos, d)
    assert np.array_equal(got, want) and not oracle.kv8_unpack(got, d)[2].any()


def test_token_by_token_and_in_pieces():
    """One sequence appended in pieces of many sizes: the oracle's bytes after
    every step; and the same bytes again when the last step is repeated."""
    d, Hkv = 64, 2
    table, ids, pos, nb, x, q, k, v = map_case([0], [100], 2, Hkv, d, 7)
    k = (k * torch.exp2(torch.arange(100).float() / 9)[:, None, None].to(BF)).contiguous()
    cache = np.zeros((nb, Hkv, attn.kv8_record_bytes(d)), np.uint8)
    at = 0
    for n in [1, 1, 1, 13, 3, 17, 1, 1, 30, 2, 14, 16]:
        s = slice(at, at + n)
        cache, want = append_both(cache, k[s], v[s], table, ids[s], pos[s], d)
        assert np.array_equal(cache, want), at
        again, _ = append_both(cache, k[s], v[s], table, ids[s], pos[s], d)
        assert np.array_equal(again, cache)
        at += n
    assert at == 100 and attn.device_status() == 0


@pytest.mark.parametrize("S,new,Hkv,d", [(700, 9, 2, 64), (5, 1300, 3, 128), (2500, 1, 1, 128), (40, 160, 5, 64)])
def test_many_rows(S, new, Hkv, d):
    """Windows of every width, several of them to a CTA, runs that end outside
    their window."""
    gen = np.random.default_rng(S)
    ctx = gen.integers(0, 60, S).tolist()
    lens = gen.integers(1, new + 1, S).tolist()
    table, ids, pos, nb, x, q, k, v = map_case(ctx, lens, 1, Hkv, d, S, padding=5)
    rec = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2)
    got, want = append_both(rec, k, v, table, ids, pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0


@pytest.mark.parametrize("d,rot,il,axes", [(128, 128, False, 1), (64, 32, True, 1), (128, 48, False, 3), (64, 64, True, 2)])
def test_rotated_records_are_those_of_the_fp32_formula(d, rot, il, axes):
    """cos and sin rounded from 64 bits, products and sums rounded to fp32 one by
    one, then the quantiser: the same bytes, and queries as rope_fwd turns them.
    (One angle in 200 may be an ulp off, and one value in 2^18 is near enough to
    the edge of a code for that to matter: about 0.01 of these 200 thousand.)"""
    ctx, new, Hkv, Hq = [3, 70000], [700, 100], 2, 5
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, Hq, Hkv, d, 91)
    f = workloads.rope_inv_freq(rot)
    kw = dict(inv_freq=f.to(DEV), interleaved=il)
    at = pos[:, None].expand(-1, rot // 2)
    if axes > 1:
        pair_axis = [i % axes for i in range(rot // 2)]
        p = torch.stack([pos // 100, pos % 100, -pos][:axes]).to(torch.int32)
        kw.update(pair_axis=pair_axis, rope_positions=p.to(DEV))
        at = p[pair_axis].T
    a = at.double().numpy() * f.double().numpy()
    c, s = (w.astype(np.float32)[:, None] for w in (np.cos(a), np.sin(a)))
    y = k.float().numpy().copy()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = u * c - w * s, w * c + u * s
    kv = torch.zeros(nb, Hkv, attn.kv8_record_bytes(d), dtype=torch.uint8, device=DEV)
    xd = x.to(DEV)
    qo = attn.kv8_append_paged(*views(xd, Hq, Hkv, d), kv, *dev(table, ids, pos), **kw)
    turned, _ = attn.rope_fwd(views(xd, Hq, Hkv, d)[0].transpose(0, 1)[None], None,
                              kw.get("rope_positions", pos.to(DEV)), f.to(DEV), kw.get("pair_axis"), il)
    torch.cuda.synchronize()
    want = oracle.kv8_append(np.zeros(tuple(kv.shape), np.uint8), y.astype(np.float64), v.double().numpy(),
                             table.numpy(), ids.numpy(), pos.numpy(), d)
    assert attn.device_status() == 0
    assert np.array_equal(kv.cpu().numpy(), want)
    assert torch.equal(turned[0].transpose(0, 1), qo)


def test_order_of_sequences_padding_and_views():
    """Sequences in any order, padding between them, strided rows, no queries,
    queries in place: what the batch's rows say, whatever lies beside them."""
    d, Hq, Hkv = 64, 3, 2
    table, ids, pos, nb, x, q, k, v = map_case([4, 0, 31], [20, 7, 2], Hq, Hkv, d, 5)
    order = torch.cat([torch.arange(20, 27), torch.arange(27, 29), torch.arange(0, 20)])
    ids2 = torch.cat([ids[order[:7]], torch.tensor([-1, -7], dtype=torch.int32), ids[order[7:]]])
    pos2 = torch.cat([pos[order[:7]], torch.tensor([-5, 9], dtype=torch.int32), pos[order[7:]]])
    wide = torch.zeros(31, 2, (Hq + 2 * Hkv) * d + 8, dtype=BF)
    wide[:, 1, 8:] = torch.cat([x[order[:7]], randn(1, 2, x.shape[1]), x[order[7:]]])
    wide = wide.to(DEV)
    qv, kk, vv = views(x.to(DEV), Hq, Hkv, d)
    f = workloads.rope_inv_freq(d).to(DEV)
    rec = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2).to(DEV)
    a, b = rec.clone(), rec.clone()
    qa = attn.kv8_append_paged(qv, kk, vv, a, *dev(table, ids, pos), inv_freq=f)
    rows = wide[:, 1, 8:]
    qb = rows[:, : Hq * d].unflatten(1, (Hq, d))
    before = qb.clone()
    attn.kv8_append_paged(qb, rows[:, Hq * d: (Hq + Hkv) * d].unflatten(1, (Hkv, d)),
                               rows[:, (Hq + Hkv) * d:].unflatten(1, (Hkv, d)), b, *dev(table, ids2, pos2), inv_freq=f,
                               q_out=qb)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    assert torch.equal(a, b) and not torch.equal(a, rec)
    assert torch.equal(qb[7:9], before[7:9])
    assert torch.equal(torch.cat([qb[:7], qb[9:]]), qa[order])
    c = rec.clone()
    assert attn.kv8_append_paged(None, kk, vv, c, *dev(table, ids, pos), inv_freq=f) is None
    torch.cuda.synchronize()
    assert torch.equal(a, c)


def test_bad_rows_are_reported_and_skipped():
    d, Hq, Hkv = 64, 2, 2
    table = torch.tensor([[0, 1], [2, 99], [-1, 3]], dtype=torch.int32)
    ids = torch.tensor([0, 0, 3, 1, 1, 2, 2, 0, 0], dtype=torch.int32)
    pos = torch.tensor([0, 1, 0, 15, 16, 3, 16, 32, -1], dtype=torch.int32)
    good = [0, 1, 3, 6]
    x = randn(2, 9, (Hq + 2 * Hkv) * d).to(DEV)
    q, k, v = views(x, Hq, Hkv, d)
    rec = workloads.kv8_cache(4, Hkv, attn.kv8_record_bytes(d), d, seed=2)
    kv = rec.to(DEV)
    q_out = torch.full((9, Hq, d), 7.0, dtype=BF, device=DEV)
    attn.kv8_append_paged(q, k, v, kv, *dev(table, ids, pos), q_out=q_out)
    torch.cuda.synchronize()
    assert attn.device_status() == attn.ATTN_DEV_BAD_BLOCK | attn.ATTN_DEV_BAD_SEQID | attn.ATTN_DEV_BAD_SEQLEN
    want = oracle.kv8_append(rec.numpy().copy(), k[good].double().cpu().numpy(), v[good].double().cpu().numpy(),
                             table.numpy(), ids[good].numpy(), pos[good].numpy(), d)
    assert np.array_equal(kv.cpu().numpy(), want)
    bad = [i for i in range(9) if i not in good]
    assert torch.all(q_out[bad] == 7.0) and torch.equal(q_out[good], q[good])
    k_out = torch.full((9, Hkv, d), 7.0, dtype=BF, device=DEV)
    v_out = k_out.clone()
    attn.kv8_read_paged(kv, *dev(table, ids, pos), d, k=k_out, v=v_out)
    torch.cuda.synchronize()
    assert attn.device_status() == attn.ATTN_DEV_BAD_BLOCK | attn.ATTN_DEV_BAD_SEQID | attn.ATTN_DEV_BAD_SEQLEN
    assert torch.all(k_out[bad] == 7.0) and torch.all(v_out[bad] == 7.0) and not torch.any(k_out[good] == 7.0)


def test_reading_in_any_order_and_the_same_row_twice():
    d, Hkv = 128, 2
    table, ids, pos, nb, _, _, _, _ = map_case([0, 0], [70, 33], 1, Hkv, d, 3)
    cache = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=4)
    k64, v64, _ = oracle.kv8_unpack(cache.numpy(), d)
    pick = torch.randint(0, 103, (500,), generator=torch.Generator().manual_seed(1))
    i, p = ids[pick], pos[pick]
    k, v = attn.kv8_read_paged(*dev(cache, table, i, p), d)
    torch.cuda.synchronize()
    phys = table[i.long(), (p // 16).long()].long().numpy()
    assert np.array_equal(to64(k), k64[phys, :, p.numpy() % 16]) and np.array_equal(to64(v), v64[phys, :, p.numpy() % 16])
    assert attn.device_status() == 0


def test_records_beyond_32_bits():
    """A pool of 5 GB: blocks on both sides of 2^32 bytes."""
    d, Hkv = 128, 8
    rec = attn.kv8_record_bytes(d)
    nb = 5 * 2 ** 30 // (Hkv * rec)
    kv = torch.zeros(nb, Hkv, rec, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[0, nb - 1, 2 ** 32 // (Hkv * rec), nb // 2]], dtype=torch.int32)
    pos = torch.arange(64, dtype=torch.int32)
    k, v = randn(1, 64, Hkv, d), randn(2, 64, Hkv, d)
    ids = torch.zeros_like(pos)
    attn.kv8_append_paged(None, *dev(k, v), kv, *dev(table, ids, pos))
    small = np.zeros((4, Hkv, rec), np.uint8)
    want = oracle.kv8_append(small, k.double().numpy(), v.double().numpy(), np.array([[0, 1, 2, 3]]), ids.numpy(), pos.numpy(), d)
    rk, _ = attn.kv8_read_paged(kv, *dev(table, ids, pos), d)
    torch.cuda.synchronize()
    assert np.array_equal(kv[table[0].long().to(DEV)].cpu().numpy(), want)
    k64 = oracle.kv8_unpack(want, d)[0]
    assert np.array_equal(to64(rk), k64.transpose(0, 2, 1, 3).reshape(64, Hkv, d)) and attn.device_status() == 0


def test_captured_append_and_read():
    """A decode step's append and a read-back in a graph, replayed on changed
    contents."""
    d, Hq, Hkv = 128, 4, 2
    table, ids, pos, nb, x, _, _, _ = map_case([17, 3, 200], [1, 1, 1], Hq, Hkv, d, 12)
    rec = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2).to(DEV)
    kv, xd, q_out = rec.clone(), x.to(DEV), torch.zeros(3, Hq, d, dtype=BF, device=DEV)
    table, ids, pos = dev(table, ids, pos)
    k, v = (torch.zeros(3, Hkv, d, dtype=BF, device=DEV) for _ in range(2))
    f = workloads.rope_inv_freq(d).to(DEV)

    def step():
        attn.kv8_append_paged(*views(xd, Hq, Hkv, d), kv, table, ids, pos, inv_freq=f, q_out=q_out)
        attn.kv8_read_paged(kv, table, ids, pos, d, k=k, v=v)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        xd.copy_(randn(seed, *x.shape))
        pos += 1
        kv.copy_(rec)
        graph.replay()
        got = [t.clone() for t in (kv, q_out, k, v)]
        kv.copy_(rec)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (kv, q_out, k, v)))
    assert attn.device_status() == 0
