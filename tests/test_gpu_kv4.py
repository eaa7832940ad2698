"""The 4-bit paged cache on the GPU: append and read-back against the oracle's
record format, the decode over it against the fp64 oracle.

Bounds.  Values without rotation reach the quantiser exactly, and its steps
are single fp32 operations: records equal the oracle's byte for byte.  Rotated
keys differ from the fp64 rotation by 2^-20 (|x| + |y|) (see test_gpu_rope) and
stand within half a step of it, plus the roundings of min and scale.

Decode: the scores' error is fp32's, well under 2^-12; a numerator and its
product with the V scale are rounded together to 11 bits (2^-11, fp16's
half step), so O is within 2^-10 max|V| before its bf16 rounding (2^-8 |O|).
The LSE uses the unrounded numerators: 2^-16 covers the fp32 sums.
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


# ------------------------------------------------------------ append and read
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_unrotated_rows_are_the_oracles_bytes(d, group, Hkv):
    ctx, new = [0, 13, 40], [1, 37, 9]
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, 2, Hkv, d, 41, padding=2)
    k, v = k.clone(), v.clone()
    k[0, 0, :group] = 3.0                          # a constant group
    k[1, 0] = 0.0
    v[2, 0, :group] *= 1e-30                       # tiny and huge ranges
    v[3, 0, :group] *= 1e30
    v[4, 0, :group] = torch.arange(group).to(BF)   # many half-way codes
    v[5, 0, :group] = 100 + torch.arange(group).to(BF) / 64
    rec = workloads.kv4_cache(nb, Hkv, attn.kv4_record_bytes(d, group), d, group, seed=2)
    kv = rec.to(DEV)
    attn.rope_append_paged_kv4(None, *dev(k, v), kv, *dev(table, ids, pos), group)
    want = rec.numpy().copy()
    T = int((ids >= 0).sum())
    vals = np.zeros((2, T, Hkv, d))
    for kind, src in ((0, k), (1, v)):
        codes, words = oracle.kv4_quantise(src[:T].float().numpy(), group)
        vals[kind] = oracle.kv4_values(codes, words, group)
        for t in range(T):
            phys = int(table[ids[t], pos[t] // 16])
            for h in range(Hkv):
                oracle.kv4_store(want[phys, h], kind, int(pos[t]) % 16, codes[t, h], words[t, h], d, group)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    assert np.array_equal(kv.cpu().numpy(), want)
    rk, rv = attn.kv4_read_paged(kv, *dev(table, ids[:T], pos[:T]), d, group)
    torch.cuda.synchronize()
    for got, ref in ((rk, vals[0]), (rv, vals[1])):
        assert np.all(np.abs(to64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -23 * 15 * np.abs(ref).max(-1, keepdims=True))


@pytest.mark.parametrize("d,group", [(64, 32), (128, 64)])
def test_half_way_values_go_to_the_even_code(d, group):
    """Groups from lowest to lowest + 15 scales whose values all lie half-way
    between two codes, exactly: (k + 1/2) scale with scale = 1, 3, 5 or 7
    times a power of two fits in bf16's 8 bits."""
    T, Hkv = 160, 2
    gen = torch.Generator().manual_seed(3)
    shape = (T, Hkv, d // group)
    scale = 2.0 * torch.randint(0, 4, shape, generator=gen) + 1
    scale = scale.double() * 2.0 ** torch.randint(-100, 100, shape, generator=gen).double()
    first = -torch.randint(0, 2, shape, generator=gen).double() * 8          # lowest, in scales
    steps = torch.randint(0, 15, (*shape, group), generator=gen).double() + 0.5
    steps[..., 0], steps[..., 1] = 0.0, 15.0
    x = ((steps + first[..., None]) * scale[..., None]).reshape(T, Hkv, d)
    assert torch.equal(x.to(BF).double(), x)
    codes, words = oracle.kv4_quantise(x.float().numpy(), group)
    whole = steps.reshape(T, Hkv, d).numpy()
    assert np.array_equal(codes, np.rint(whole).astype(codes.dtype))         # half to even
    want = np.zeros((T // 16, Hkv, attn.kv4_record_bytes(d, group)), np.uint8)
    for t in range(T):
        for h in range(Hkv):
            for kind in (0, 1):
                oracle.kv4_store(want[t // 16, h], kind, t % 16, codes[t, h], words[t, h], d, group)
    kv = torch.zeros(want.shape, dtype=torch.uint8, device=DEV)
    x = x.to(BF).to(DEV)
    table = torch.arange(T // 16, dtype=torch.int32, device=DEV)[None]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    attn.rope_append_paged_kv4(None, x, x, kv, table, torch.zeros_like(pos), pos, group)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    assert np.array_equal(kv.cpu().numpy(), want)


@pytest.mark.parametrize("d,group,rot,il", [(128, 64, 128, False), (64, 32, 32, True)])
def test_rotated_records_are_those_of_the_fp32_formula(d, group, rot, il):
    """cos and sin rounded from 64 bits, products and sums rounded to fp32 one by
    one, then the quantiser: the same bytes.  (One angle in 200 may be an ulp
    off, and one value in 2^20 is near enough to the edge of a code for that to
    matter: under 0.01 of these 200 thousand.)"""
    ctx, new, Hkv = [3, 70000], [700, 100], 2
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, 1, Hkv, d, 91)
    f = workloads.rope_inv_freq(rot)
    a = pos.double().numpy()[:, None] * f.double().numpy()
    c, s = (w.astype(np.float32)[:, None] for w in (np.cos(a), np.sin(a)))
    y = k.float().numpy().copy()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, rot // 2), slice(rot // 2, rot))
    u, w = y[..., first].copy(), y[..., second].copy()
    y[..., first], y[..., second] = u * c - w * s, w * c + u * s
    kv = torch.zeros(nb, Hkv, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
    attn.rope_append_paged_kv4(None, *dev(k, v), kv, *dev(table, ids, pos), group, f.to(DEV), interleaved=il)
    torch.cuda.synchronize()
    want = np.zeros(tuple(kv.shape), np.uint8)
    for kind, src in ((0, y), (1, v.float().numpy())):
        codes, words = oracle.kv4_quantise(src, group)
        for t in range(pos.numel()):
            phys = int(table[ids[t], pos[t] // 16])
            for h in range(Hkv):
                oracle.kv4_store(want[phys, h], kind, int(pos[t]) % 16, codes[t, h], words[t, h], d, group)
    assert np.array_equal(kv.cpu().numpy(), want)


@pytest.mark.parametrize("d,group,rot,il,axes", [(128, 32, 128, False, 1), (128, 64, 64, True, 1),
                                                 (64, 32, 64, False, 3), (64, 64, 32, True, 2)])
def test_rotated_rows_stand_for_the_rotation(d, group, rot, il, axes):
    Hq, Hkv = 6, 2
    table, ids, pos, nb, x, q, k, v = map_case([0, 5, 900], [3, 120, 1], Hq, Hkv, d, 51, padding=1)
    T = int((ids >= 0).sum())
    f = workloads.rope_inv_freq(rot)
    axis = rp = None
    if axes > 1:
        axis = [p % axes for p in range(rot // 2)]
        rp = torch.stack([pos // 9, pos % 9, pos % 5][:axes]).to(torch.int32)
    kv = workloads.kv4_cache(nb, Hkv, attn.kv4_record_bytes(d, group), d, group, seed=3).to(DEV)
    kc, vc = (torch.zeros(nb, Hkv, 16, d, dtype=BF, device=DEV) for _ in range(2))
    m = dev(table, ids, pos)
    kw = dict(inv_freq=f.to(DEV), rope_positions=None if rp is None else rp.to(DEV), pair_axis=axis, interleaved=il)
    qo = torch.zeros(ids.numel(), Hq, d, dtype=BF, device=DEV)
    qb = torch.zeros_like(qo)
    xd = x.to(DEV)
    attn.rope_append_paged_kv4(*views(xd, Hq, Hkv, d), kv, *m, group, q_out=qo, **kw)
    attn.rope_append_paged(*views(xd, Hq, Hkv, d), kc, vc, *m, q_out=qb, **kw)
    rk, rv = attn.kv4_read_paged(kv, m[0], m[1][:T], m[2][:T], d, group)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    assert torch.equal(qo, qb)                     # the same queries as the bf16 append
    ref = oracle.rope_rotate(to64(k[:T].transpose(0, 1)), (pos[None] if rp is None else rp).numpy()[:, :T], f.numpy(),
                             axis, il).swapaxes(0, 1)
    y = ref.reshape(T, Hkv, -1, group)
    step = np.repeat((y.max(-1) - y.min(-1)) / 15, group, -1).reshape(ref.shape)
    big = np.repeat(np.abs(y).max(-1), group, -1).reshape(ref.shape)
    # half a step (itself rounded, 2^-8), min and 15 scales rounded (2^-8 of at most 2 big each), bf16 on reading
    lim = step / 2 * (1 + 2.0 ** -7) + 5 * 2.0 ** -8 * big + 2.0 ** -18 * big
    assert np.all(np.abs(to64(rk) - ref) <= lim)
    codes, words = oracle.kv4_quantise(v[:T].float().numpy(), group)
    vals = oracle.kv4_values(codes, words, group)
    assert np.all(np.abs(to64(rv) - vals) <= 2.0 ** -8 * np.abs(vals) + 1e-5)


def test_non_finite_groups_poison_themselves_only():
    d, group = 128, 32
    k, v = randn(61, 3, 2, d), randn(62, 3, 2, d)
    k[0, 0, 5] = float("inf")
    k[0, 1, 64] = float("nan")
    v[1, 0, 127] = float("-inf")
    v[2, 1, 32:64] = 3e38
    v[2, 1, 33] = -3e38                            # a range beyond fp32
    table, ids, pos = torch.tensor([[0]]).int(), torch.zeros(3).int(), torch.arange(3).int()
    kv = torch.zeros(1, 2, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
    m = dev(table, ids, pos)
    attn.rope_append_paged_kv4(None, *dev(k, v), kv, *m, group)
    rk, rv = attn.kv4_read_paged(kv, *m, d, group)
    torch.cuda.synchronize()
    bk, bv = torch.zeros(3, 2, d, dtype=torch.bool), torch.zeros(3, 2, d, dtype=torch.bool)
    bk[0, 0, :32] = bk[0, 1, 64:96] = bv[1, 0, 96:] = bv[2, 1, 32:64] = True
    assert torch.equal(torch.isnan(rk.float().cpu()), bk) and torch.equal(torch.isnan(rv.float().cpu()), bv)


# --------------------------------------------------------------------- decode
def decode_case(lens, Hq, Hkv, d, group, seed, max_blocks=None, **kw):
    table, _, _, nb = workloads.token_map([0] * len(lens), lens, seed, spare_blocks=1)
    if max_blocks is not None:
        table = torch.nn.functional.pad(table, (0, max_blocks - table.shape[1]), value=-1)
    rec = workloads.kv4_cache(nb, Hkv, attn.kv4_record_bytes(d, group), d, group, seed + 1, **kw)
    # Slots past a sequence's end hold NaN parameters: using them would show.
    for b, n in enumerate(lens):
        if n % 16:
            phys = int(table[b, n // 16])
            for kind in (0, 1):
                par = 16 * d + kind * 16 * (d // group) * 4
                rec[phys, :, par + (n % 16) * (d // group) * 4: par + 16 * (d // group) * 4] = 0xFF
    return randn(seed + 2, len(lens), Hq, d), rec, table, torch.tensor(lens, dtype=torch.int32)


def check_decode(o, lse, q, rec, table, lens, scale, d, group, what=""):
    ro, rl = oracle.decode_paged_kv4(to64(q), rec.numpy(), table.numpy(), lens.numpy(), scale, d, group)
    _, v = oracle.kv4_unpack(rec.numpy(), d, group)
    vmax = np.nanmax(np.abs(v[np.unique(table.numpy()[table.numpy() >= 0])])) if (table >= 0).any() else 0.0
    err = np.abs(to64(o) - ro)
    lim = 2.0 ** -8 * np.abs(ro) + 2.0 ** -10 * vmax
    assert np.all(err <= lim), "%s: O at %.3g of its bound" % (what, (err / lim).max())
    if lse is not None:
        fin = np.isfinite(rl)
        assert np.array_equal(to64(lse)[~fin], rl[~fin])
        if fin.any():
            assert np.abs(to64(lse)[fin] - rl[fin]).max() <= 2.0 ** -16 * max(1.0, np.abs(rl[fin]).max()), what
    return ro, rl


def run(q, rec, table, lens, group, scale=None, **kw):
    d = q.shape[-1]
    o, lse = attn.attn_decode_paged_kv4(*dev(q, rec, table, lens), group, scale=scale, **kw)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    return o, lse


LENS = [1, 15, 16, 17, 31, 32, 33, 100, 0, 255, 256, 257, 700, 4096, 3]


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 2), (8, 1), (9, 1), (32, 2), (15, 5)])
def test_ragged_lengths(Hq, Hkv, d, group):
    case = decode_case(LENS, Hq, Hkv, d, group, seed=70 + Hq + d + group)
    scale = workloads.default_scale(d)
    o, lse = run(*case, group, scale)
    check_decode(o, lse, *case, scale, d, group, "ragged")
    assert torch.all(o[8] == 0) and torch.all(torch.isneginf(lse[8]))


@pytest.mark.parametrize("n", [1, 2, 16, 17, 500, 20000])
def test_one_sequence(n):
    case = decode_case([n], 6, 1, 128, 32, seed=90)
    o, lse = run(*case, 32, 0.09)
    check_decode(o, lse, *case, 0.09, 128, 32, "one sequence")


@pytest.mark.parametrize("S,Hq,Hkv,d,group,most", [
    (1, 8, 1, 128, 32, 700), (7, 15, 3, 128, 32, 110), (20, 16, 2, 64, 64, 600), (76, 4, 2, 128, 64, 400),
    (152, 1, 1, 64, 32, 300), (153, 1, 1, 64, 32, 300), (38, 64, 4, 64, 32, 250), (30, 9, 3, 128, 32, 1600),
    (50, 2, 2, 64, 32, 17), (3, 32, 2, 128, 64, 90), (100, 6, 3, 128, 32, 100), (110, 4, 4, 64, 64, 130),
    (300, 2, 2, 128, 64, 60), (900, 2, 2, 64, 32, 33), (100, 64, 4, 64, 32, 100), (250, 36, 4, 64, 64, 70),
    (95, 32, 2, 128, 32, 200)])
def test_a_team_of_warps_to_each_run_or_equal_shares(S, Hq, Hkv, d, group, most):
    """Up to as many (sequence, KV head) runs as warps, short ones: each is some
    warps', or cut into equal shares, on either side of the rule."""
    g = torch.Generator().manual_seed(S)
    for lens in ([most] * S, torch.randint(0, most + 1, (S,), generator=g).tolist(),
                 torch.randint(most - most // 4, most + 1, (S,), generator=g).tolist()):
        q, rec, table, lens = decode_case(lens, Hq, Hkv, d, group, seed=S + 1)
        check_decode(*run(q, rec, table, lens, group), q, rec, table, lens, d ** -0.5, d, group)


def test_few_short_runs_among_many_empty_sequences():
    """More sequences than the plan has entries, most of them empty."""
    lens = [0] * 2500
    for i, n in ((0, 40), (1, 3), (1023, 200), (1024, 1), (1025, 333), (2048, 16), (2499, 17)):
        lens[i] = n
    q, rec, table, lens = decode_case(lens, 4, 2, 128, 32, seed=9)
    check_decode(*run(q, rec, table, lens, 32), q, rec, table, lens, 128 ** -0.5, 128, 32)


def test_many_sequences_and_heads():
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 300, (500,), generator=gen).tolist()
    case = decode_case(lens, 16, 8, 64, 32, seed=95, max_blocks=40)
    o, lse = run(*case, 32, 0.125)
    check_decode(o, lse, *case, 0.125, 64, 32, "many")


def test_more_sequences_than_the_plan_caches():
    lens = [(7 * b) % 40 for b in range(2500)]
    case = decode_case(lens, 2, 1, 64, 64, seed=97)
    o, lse = run(*case, 64, 0.125)
    check_decode(o, lse, *case, 0.125, 64, 64, "2500 sequences")


@pytest.mark.parametrize("scale,spread", [(1e-6, 0.2), (40.0, 0.2), (0.3, 2.5)])
def test_wide_ranges(scale, spread):
    """Tiny and large caches, and V scales over many orders of magnitude (the
    weights' power of two has to follow them); large keys give a softmax that
    jumps from token to token."""
    case = decode_case([300, 4000, 77], 8, 2, 128, 32, seed=99, scale=scale, spread=spread)
    s = 0.09 / max(scale, 1.0)
    o, lse = run(*case, 32, s)
    check_decode(o, lse, *case, s, 128, 32, "wide")


def test_first_token_dominates_and_queries_of_mixed_size():
    q, rec, table, lens = decode_case([600, 33], 8, 1, 128, 64, seed=101)
    q = q.float()
    q[0, 1] *= 1e-20
    q[0, 2] = 0.0
    q[0, 3, 0] = 300.0                             # one large element beside small ones
    q[1, :, :] *= 20.0
    q = q.to(BF)
    o, lse = run(q, rec, table, lens, 64, 0.09)
    check_decode(o, lse, q, rec, table, lens, 0.09, 128, 64, "mixed queries")


def test_zero_values_and_constant_groups():
    q, rec, table, lens = decode_case([70, 18], 4, 2, 64, 32, seed=103)
    d, group = 64, 32
    words = rec[..., 16 * d:].view(torch.int32)
    n = 16 * (d // group)
    words[:, 0, n:] = 0                            # head 0: every V value is 0
    words[:, 1, n:] &= 0xFFFF                      # head 1: scale 0, each V group constant at min
    o, lse = run(q, rec, table, lens, group, 0.1)
    check_decode(o, lse, q, rec, table, lens, 0.1, d, group, "constant")
    assert torch.all(o[:, :2] == 0)


def test_a_poisoned_key_shows_in_its_heads_only():
    q, rec, table, lens = decode_case([200, 40], 8, 2, 128, 32, seed=105)
    want, want_l = run(q, rec, table, lens, 32, 0.1)
    phys = int(table[0, 3])
    par = rec[phys, 1, 16 * 128:].view(torch.int32)
    par[4 * 2] = 0x7FC07FC0                        # K parameters of slot 2, group 0
    o, lse = run(q, rec, table, lens, 32, 0.1)
    assert torch.isnan(o[0, 4:].float()).all() and torch.isnan(lse[0, 4:]).all()
    assert torch.equal(o[0, :4], want[0, :4]) and torch.equal(o[1], want[1]) and torch.equal(lse[1], want_l[1])


def test_bad_table_entries_are_reported_and_skipped():
    q, rec, table, lens = decode_case([100, 50], 4, 2, 64, 32, seed=107)
    bad = table.clone()
    bad[0, 2] = rec.shape[0] + 5
    bad[1, 0] = -7
    attn.device_status()
    o, lse = attn.attn_decode_paged_kv4(*dev(q, rec, bad, lens), 32, scale=0.1)
    torch.cuda.synchronize()
    assert attn.device_status() == attn.ATTN_DEV_BAD_BLOCK
    k, v = oracle.kv4_unpack(rec.numpy(), 64, 32)
    for b, gone in ((0, 2), (1, 0)):
        at = [(int(table[b, p // 16]), p % 16) for p in range(int(lens[b])) if p // 16 != gone]
        for h in range(4):
            kk = np.stack([k[i, h // 2, s] for i, s in at])
            vv = np.stack([v[i, h // 2, s] for i, s in at])
            s = kk @ to64(q[b, h]) * 0.1
            p = np.exp(s - s.max())
            assert np.abs(to64(o[b, h]) - p @ vv / p.sum()).max() <= 2.0 ** -7 * np.abs(vv).max()
    wrong = lens.clone()
    wrong[0] = table.shape[1] * 16 + 1
    wrong[1] = -3
    o, lse = attn.attn_decode_paged_kv4(*dev(q, rec, table, wrong), 32, scale=0.1)
    torch.cuda.synchronize()
    assert attn.device_status() & attn.ATTN_DEV_BAD_SEQLEN
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1]))


def test_shared_prefix_blocks():
    """Two sequences whose tables share physical blocks."""
    q, rec, table, lens = decode_case([320, 320], 4, 1, 128, 64, seed=109)
    table = table.clone()
    table[1, :15] = table[0, :15]
    o, lse = run(q, rec, table, lens, 64, 0.1)
    check_decode(o, lse, q, rec, table, lens, 0.1, 128, 64, "shared prefix")


def test_repeats_bit_for_bit_and_lse_is_optional():
    case = decode_case([3000, 1, 4096, 64, 777, 2048, 0, 1500], 12, 2, 128, 32, seed=111)
    ws = torch.full((attn.attn_decode_paged_kv4_workspace_size(8, 12, 2, 128),), 0xA5, dtype=torch.uint8, device=DEV)
    first, lse = run(*case, 32, 0.1, workspace=ws)
    for _ in range(5):
        o, l = run(*case, 32, 0.1, workspace=ws)
        assert torch.equal(o, first) and torch.equal(l, lse)
    o, none = run(*case, 32, 0.1, return_lse=False)
    assert none is None and torch.equal(o, first)


# ------------------------------------------------------- the operators together
def test_prefill_then_decode_steps():
    """A prompt through rope_fwd and attn_fwd, its keys and values into the
    4-bit cache, then decode steps that append and attend: every step against
    the fp64 softmax over what the cache stands for, and the 4-bit result near
    the bf16 cache's."""
    S, Hq, Hkv, d, group, prompt, steps = 3, 8, 2, 128, 32, [45, 16, 7], 4
    f = workloads.rope_inv_freq(d).to(DEV)
    table, ids, pos, nb = workloads.token_map([0] * S, [n + steps for n in prompt], seed=5)
    kv = torch.zeros(nb, Hkv, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
    kc, vc = (torch.zeros(nb, Hkv, 16, d, dtype=BF, device=DEV) for _ in range(2))
    keep = torch.cat([torch.arange(n + steps) < n for n in prompt])
    x = randn(120, int(keep.sum()), (Hq + 2 * Hkv) * d).to(DEV)
    m = [table.to(DEV), ids[keep].to(DEV), pos[keep].to(DEV)]
    q4 = attn.rope_append_paged_kv4(*views(x, Hq, Hkv, d), kv, *m, group, inv_freq=f)
    qb = attn.rope_append_paged(*views(x, Hq, Hkv, d), kc, vc, *m, inv_freq=f)
    # the same prompt by the training path: rotate head-major, attend
    at = 0
    for b, n in enumerate(prompt):
        q, k, v = (t[at:at + n].transpose(0, 1)[None] for t in views(x, Hq, Hkv, d))
        qr, kr = attn.rope_fwd(q, k, torch.arange(n, dtype=torch.int32, device=DEV), f)
        torch.cuda.synchronize()
        assert torch.equal(qr[0].transpose(0, 1), qb[at:at + n]) and torch.equal(qr[0].transpose(0, 1), q4[at:at + n])
        rows = torch.arange(n)
        assert torch.equal(kc[table[b].long()[rows // 16], :, rows % 16], kr[0].transpose(0, 1))
        at += n
    ws = torch.empty(attn.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d), dtype=torch.uint8, device=DEV)
    lens = torch.tensor(prompt, dtype=torch.int32)
    seqs = torch.arange(S, dtype=torch.int32, device=DEV)
    for t in range(steps):
        y = views(randn(130 + t, S, (Hq + 2 * Hkv) * d).to(DEV), Hq, Hkv, d)
        p = lens.to(DEV)
        q4 = attn.rope_append_paged_kv4(*y, kv, m[0], seqs, p, group, inv_freq=f)
        qb = attn.rope_append_paged(*y, kc, vc, m[0], seqs, p, inv_freq=f)
        lens += 1
        o4, l4 = attn.attn_decode_paged_kv4(q4, kv, m[0], lens.to(DEV), group, workspace=ws)
        ob, _ = attn.attn_decode_paged(qb, kc, vc, m[0], lens.to(DEV))
        torch.cuda.synchronize()
        assert attn.device_status() == 0
        check_decode(o4, l4, q4.cpu(), kv.cpu(), table, lens, d ** -0.5, d, group, "step %d" % t)
        # a value is off by at most half a step of a range of at most 2 max|v|, the scores by less than 1
        assert (o4.float() - ob.float()).abs().max() < 2.0
    # the chunked-prefill route: cached tokens back to bf16 blocks
    n = int(lens[0])
    seq0, rows = torch.zeros(n, dtype=torch.int32, device=DEV), torch.arange(n, dtype=torch.int32, device=DEV)
    rk, rv = attn.kv4_read_paged(kv, m[0], seq0, rows, d, group)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    attn.rope_append_paged(None, rk, rv, k2, v2, m[0], seq0, rows)
    o2, _ = attn.attn_decode_paged(q4[:1].contiguous(), k2, v2, m[0][:1].contiguous(), lens[:1].to(DEV))
    torch.cuda.synchronize()
    assert (o2[0].float() - o4[0].float()).abs().max() <= 2e-2


def test_captured_step_replays_and_two_graphs_share_a_workspace():
    S, Hq, Hkv, d, group = 5, 12, 2, 128, 32
    q, rec, table, lens = decode_case([4000, 17, 333, 0, 2100], Hq, Hkv, d, group, seed=141)
    f = workloads.rope_inv_freq(d).to(DEV)
    kv, tab, ln = dev(rec, table, lens)
    x = randn(142, S, (Hq + 2 * Hkv) * d).to(DEV)
    ids = torch.tensor([0, 1, 2, -1, 4], dtype=torch.int32, device=DEV)
    at = (ln - 1).clamp(min=0)
    ws = torch.empty(attn.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d), dtype=torch.uint8, device=DEV)

    def step(qo, o, lse):
        attn.rope_append_paged_kv4(*views(x, Hq, Hkv, d), kv, tab, ids, at, group, inv_freq=f, q_out=qo)
        attn.attn_decode_paged_kv4(qo, kv, tab, ln, group, o=o, lse=lse, workspace=ws)

    bufs = [(torch.zeros(S, Hq, d, dtype=BF, device=DEV), torch.empty(S, Hq, d, dtype=BF, device=DEV),
             torch.empty(S, Hq, device=DEV)) for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*bufs[0])
        want = [t.clone() for t in bufs[0][1:]]
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for b in bufs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*b)
        graphs.append(g)
    for _ in range(3):
        for g, b in zip(graphs, bufs[1:]):
            b[1].zero_()
            g.replay()
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    for b in bufs[1:]:
        assert torch.equal(b[1], want[0]) and torch.equal(b[2], want[1])


def test_calls_see_inputs_written_just_before_on_their_stream():
    S, Hq, Hkv, d, group = 4, 8, 2, 64, 32
    cases = [decode_case([900, 5, 64, 333], Hq, Hkv, d, group, seed=150 + i) for i in range(3)]
    side = torch.cuda.Stream()
    q, rec, tab, ln = (torch.empty_like(t, device=DEV) for t in cases[0])
    on_dev = [dev(*c) for c in cases]
    torch.cuda.synchronize()
    outs = []
    with torch.cuda.stream(side):
        for c in on_dev:
            for dst, src in zip((q, rec, tab, ln), c):
                dst.copy_(src)
            outs.append(attn.attn_decode_paged_kv4(q, rec, tab, ln, group))
    side.synchronize()
    for c, (o, lse) in zip(on_dev, outs):
        ro, rl = attn.attn_decode_paged_kv4(*c, group)
        torch.cuda.synchronize()
        assert torch.equal(o, ro) and torch.equal(lse, rl)


@pytest.mark.parametrize("early", [0, 1, 2])
def test_early_plan_sees_tokens_appended_just_before(early):
    """The append that runs just before the decode, on the same stream, writes
    the newest slots and the queries; lengths and table come from the host."""
    S, Hq, Hkv, d, group = 6, 12, 2, 128, 32
    q, rec, table, lens = decode_case([700, 64, 17, 1500, 1, 333], Hq, Hkv, d, group, seed=170)
    f = workloads.rope_inv_freq(d).to(DEV)
    tab, ln = dev(table, lens)
    ids, at = torch.arange(S, dtype=torch.int32, device=DEV), ln - 1
    steps = [randn(171 + i, S, (Hq + 2 * Hkv) * d).to(DEV) for i in range(3)]
    want = []
    kv = rec.to(DEV)
    for x in steps:
        qo = attn.rope_append_paged_kv4(*views(x, Hq, Hkv, d), kv, tab, ids, at, group, inv_freq=f)
        torch.cuda.synchronize()
        want.append(attn.attn_decode_paged_kv4(qo, kv, tab, ln, group))
        torch.cuda.synchronize()
    kv = rec.to(DEV)
    torch.cuda.synchronize()
    got = []
    try:
        attn.set_decode_early_plan(early)
        for x in steps:
            qo = attn.rope_append_paged_kv4(*views(x, Hq, Hkv, d), kv, tab, ids, at, group, inv_freq=f)
            got.append(attn.attn_decode_paged_kv4(qo, kv, tab, ln, group))
        torch.cuda.synchronize()
    finally:
        attn.set_decode_early_plan(0)
    assert attn.device_status() == 0
    for (o, l), (ro, rl) in zip(got, want):
        assert torch.equal(o, ro) and torch.equal(l, rl)


def test_long_cache_beyond_32_bit_offsets():
    """Records past 2^32 bytes from the start of the pool: append, read and
    decode address them."""
    d, group, Hkv = 128, 32, 8
    rec = attn.kv4_record_bytes(d, group)
    nb = (1 << 32) // (Hkv * rec) + 40
    kv = torch.zeros(nb, Hkv, rec, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[nb - 1, 3, nb - 2]], dtype=torch.int32, device=DEV)
    ids, pos = torch.zeros(40, dtype=torch.int32, device=DEV), torch.arange(40, dtype=torch.int32, device=DEV)
    k, v = randn(160, 40, Hkv, d).to(DEV), randn(161, 40, Hkv, d).to(DEV)
    attn.rope_append_paged_kv4(None, k, v, kv, table, ids, pos, group)
    rk, rv = attn.kv4_read_paged(kv, table, ids, pos, d, group)
    q = randn(162, 1, Hkv, d).to(DEV)
    o, _ = attn.attn_decode_paged_kv4(q, kv, table, torch.tensor([40], dtype=torch.int32, device=DEV), group)
    torch.cuda.synchronize()
    small = kv[[nb - 1, 3, nb - 2]].cpu()
    ro, _ = oracle.decode_paged_kv4(to64(q), small.numpy(), np.array([[0, 1, 2]]), [40], d ** -0.5, d, group)
    assert np.abs(to64(o) - ro).max() <= 2.0 ** -8 * np.abs(ro).max() + 2.0 ** -10 * 6
    assert (rk.float() - k.float()).abs().max() < 0.5 and (rv.float() - v.float()).abs().max() < 0.5
    assert attn.device_status() == 0
