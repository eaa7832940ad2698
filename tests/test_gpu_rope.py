"""Rotary positions and the paged appends on the GPU, against the fp64 oracle.

Bound of a rotated value x cos a - y sin a: the angle is formed to 2^-32
turns, cos and sin are good to 1 ulp, and three fp32 roundings follow: under
2^-20 (|x| + |y|).  Then one rounding to bf16, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import oracle
import workloads
from parity import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF)


def bound(ref, x, rot, interleaved):
    """2^-8 |ref| + 2^-20 (|x| + |y|) with y the partner of x."""
    a = np.abs(to64(x))
    y = a.copy()
    half = rot // 2
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a[..., 1:rot:2], a[..., 0:rot:2]
    else:
        y[..., :half], y[..., half:rot] = a[..., half:rot], a[..., :half]
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * (a + y) + 1e-30


def check(got, ref, x, rot, interleaved, what):
    err = np.abs(to64(got) - ref)
    lim = bound(ref, x, rot, interleaved)
    assert np.all(err <= lim), "%s: %.3g of the bound" % (what, (err / lim).max())
    assert np.array_equal(to64(got)[..., rot:], to64(x)[..., rot:]), what + ": unrotated part changed"


CASES = [  # B, Hq, Hk, N, d, rot, axes, interleaved
    (1, 1, 1, 1, 64, 64, 1, False),
    (2, 12, 2, 37, 128, 128, 1, False),
    (1, 5, 3, 130, 64, 32, 1, True),
    (3, 4, 4, 17, 128, 16, 1, False),
    (1, 16, 1, 257, 128, 128, 3, False),
    (2, 3, 2, 65, 64, 64, 2, True),
    (1, 7, 7, 1001, 64, 48, 4, False),
    (1, 2, 2, 3000, 128, 96, 1, True),
]


@pytest.mark.parametrize("B,Hq,Hk,N,d,rot,axes,il", CASES)
@pytest.mark.parametrize("back", [False, True])
def test_rotation_against_the_oracle(B, Hq, Hk, N, d, rot, axes, il, back):
    gen = torch.Generator().manual_seed(N)
    q, k = randn(N, B, Hq, N, d), randn(N + 1, B, Hk, N, d)
    # ordinary, negative and very far positions
    pos = torch.randint(-50, 5000, (axes, B, N), generator=gen)
    pos[:, :, ::3] += 1 << 20
    pos[:, :, -1] = 2 ** 31 - 1
    pos = pos.to(torch.int32)
    f = workloads.rope_inv_freq(rot)
    axis = None if axes == 1 else [int(a) for a in torch.randint(0, axes, (rot // 2,), generator=gen)]
    func = attn.rope_bwd if back else attn.rope_fwd
    p = pos.to(DEV)
    qo, ko = func(q.to(DEV), k.to(DEV), p[0] if axes == 1 else p, f.to(DEV), pair_axis=axis, interleaved=il)
    torch.cuda.synchronize()
    assert qo.is_contiguous() and qo.shape == q.shape and ko.shape == k.shape
    for b in range(B):
        for x, y, what in ((q, qo, "q"), (k, ko, "k")):
            ref = oracle.rope_rotate(to64(x[b]), pos[:, b].numpy(), f.numpy(), axis, il, inverse=back)
            check(y[b], ref, x[b], rot, il, "%s batch %d" % (what, b))


def test_merged_projection_strided_in_and_out():
    """Token-major views of one merged buffer to head-major tensors, and the
    gradients back into such views of one buffer."""
    B, N, Hq, Hk, d = 2, 53, 6, 2, 128
    x = randn(3, B, N, (Hq + 2 * Hk) * d)
    f = workloads.rope_inv_freq(d)
    pos = torch.arange(N, dtype=torch.int32)
    xd = x.to(DEV)

    def parts(t):
        return (t[..., : Hq * d].view(B, N, Hq, d).transpose(1, 2),
                t[..., Hq * d: (Hq + Hk) * d].view(B, N, Hk, d).transpose(1, 2))

    q, k = parts(xd)
    qo, ko = attn.rope_fwd(q, k, pos.to(DEV), f.to(DEV))
    grad = torch.zeros_like(xd)
    gq, gk = parts(grad)
    attn.rope_bwd(qo, ko, pos.to(DEV), f.to(DEV), dq=gq, dk=gk)
    torch.cuda.synchronize()
    hq, hk = parts(x)
    for src, got, back in ((hq, qo, gq), (hk, ko, gk)):
        ref = oracle.rope_rotate(to64(src), pos.numpy(), f.numpy())
        check(got, ref, src.contiguous(), d, False, "merged")
        ref = oracle.rope_rotate(to64(got), pos.numpy(), f.numpy(), inverse=True)
        check(back, ref, got.cpu(), d, False, "merged back")
    assert torch.all(grad[..., (Hq + Hk) * d:] == 0)
    # in place, in the merged buffer: the values' part untouched
    y = xd.clone()
    q2, k2 = parts(y)
    attn.rope_fwd(q2, k2, pos.to(DEV), f.to(DEV), q_out=q2, k_out=k2)
    torch.cuda.synchronize()
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(y[..., (Hq + Hk) * d:], xd[..., (Hq + Hk) * d:])


def test_broadcast_inputs_and_queries_only():
    B, N, H, d = 3, 20, 4, 64
    one = randn(5, 1, 1, N, d).to(DEV)
    pos = torch.randint(0, 99, (B, N), dtype=torch.int32).to(DEV)
    f = workloads.rope_inv_freq(d).to(DEV)
    qo, none = attn.rope_fwd(one.expand(B, H, N, d), None, pos, f)
    full, _ = attn.rope_fwd(one.expand(B, H, N, d).contiguous(), None, pos, f)
    torch.cuda.synchronize()
    assert none is None and torch.equal(qo, full)
    shared, _ = attn.rope_fwd(one.expand(B, H, N, d), None, pos[:1].expand(B, N), f)
    again, _ = attn.rope_fwd(one.expand(B, H, N, d), None, pos[0], f)
    torch.cuda.synchronize()
    assert torch.equal(shared, again)


def test_infinities_and_nan_stay_in_their_pairs():
    d, rot = 64, 32
    q = randn(6, 1, 2, 5, d)
    q[0, 0, 1, 3] = float("inf")
    q[0, 1, 2, 40] = float("nan")                 # in the part that passes through
    f = workloads.rope_inv_freq(rot)
    f[5] = float("inf")
    qo, _ = attn.rope_fwd(q.to(DEV), None, torch.arange(5, dtype=torch.int32).to(DEV), f.to(DEV))
    torch.cuda.synchronize()
    bad = torch.zeros(q.shape, dtype=torch.bool)
    bad[..., [5, 21]] = True
    bad[0, 0, 1, [3, 19]] = True
    bad[0, 1, 2, 40] = True
    finite = torch.isfinite(qo.float().cpu())
    assert torch.equal(~finite, bad)


def test_gradient_by_differences():
    """The derivative of sum(g * rope(x)) along single elements, from calls on
    exactly representable steps."""
    d, N = 64, 9
    x, g = randn(7, 1, 1, N, d), randn(8, 1, 1, N, d)
    f, pos = workloads.rope_inv_freq(d).to(DEV), torch.arange(N, dtype=torch.int32).to(DEV)
    dx, _ = attn.rope_bwd(g.to(DEV), None, pos, f)
    for e in (0, 7, 31, 32, 63):
        up = torch.zeros_like(x)
        up[..., e] = 1.0                          # the map is linear: its value on a unit step is the difference
        y, _ = attn.rope_fwd(up.to(DEV), None, pos, f)
        num = (y.double() * g.to(DEV).double()).sum(-1).cpu()
        # y is rounded to bf16 (2 terms, 2^-8 of each), dx once
        lim = 2.0 ** -8 * (2 * g.abs().amax().item() + num.abs()) + 1e-6
        assert torch.all((dx[..., e].double().cpu() - num).abs() <= lim)


def map_case(ctx, new, Hq, Hkv, d, seed, padding=0):
    table, ids, pos, nb = workloads.token_map(ctx, new, seed, padding, spare_blocks=2)
    T = ids.numel()
    x = randn(seed + 1, T, (Hq + 2 * Hkv) * d)
    q, k, v = x[:, : Hq * d].view(T, Hq, d), x[:, Hq * d: (Hq + Hkv) * d].view(T, Hkv, d), x[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    return table, ids, pos, nb, x, q, k, v


def views(x, Hq, Hkv, d):
    T = x.shape[0]
    return (x[:, : Hq * d].view(T, Hq, d), x[:, Hq * d: (Hq + Hkv) * d].view(T, Hkv, d),
            x[:, (Hq + Hkv) * d:].view(T, Hkv, d))


APPENDS = [  # ctx, new, Hq, Hkv, d, rot, axes, interleaved, padding
    ([0], [1], 1, 1, 64, 64, 1, False, 0),
    ([31, 0, 16, 700], [1, 1, 1, 1], 12, 2, 128, 128, 1, False, 3),
    ([5, 0, 100], [40, 0, 33], 6, 3, 64, 32, 1, True, 0),
    ([15, 17], [300, 129], 16, 1, 128, 128, 3, False, 11),
    ([3], [2500], 5, 5, 128, 64, 1, False, 0),
]


@pytest.mark.parametrize("ctx,new,Hq,Hkv,d,rot,axes,il,padding", APPENDS)
def test_append_against_the_oracle(ctx, new, Hq, Hkv, d, rot, axes, il, padding):
    table, ids, pos, nb, x, q, k, v = map_case(ctx, new, Hq, Hkv, d, 11, padding)
    order = torch.randperm(ids.numel(), generator=torch.Generator().manual_seed(1))   # tokens in any order
    ids, pos, x = ids[order], pos[order], x[order]
    q, k, v = views(x, Hq, Hkv, d)
    f = workloads.rope_inv_freq(rot)
    axis = rp = None
    if axes > 1:
        axis = [p % axes for p in range(rot // 2)]
        rp = torch.stack([pos // 64, pos % 64 // 8, pos % 8][:axes]).to(torch.int32)
    kc, vc = randn(12, nb, Hkv, 16, d), randn(13, nb, Hkv, 16, d)
    kd, vd = kc.to(DEV), vc.to(DEV)
    qd, kk, vv = views(x.to(DEV), Hq, Hkv, d)
    keep = randn(14, ids.numel(), Hq, d)
    qo = keep.to(DEV)
    out = attn.rope_append_paged(qd, kk, vv, kd, vd, table.to(DEV), ids.to(DEV), pos.to(DEV), inv_freq=f.to(DEV),
                                 rope_positions=None if rp is None else rp.to(DEV), pair_axis=axis, interleaved=il,
                                 q_out=qo)
    torch.cuda.synchronize()
    assert out is qo and attn.device_status() == 0
    at = (pos[None] if rp is None else rp).numpy()
    live = (ids >= 0).numpy()
    qr = oracle.rope_rotate(to64(q.transpose(0, 1)), at, f.numpy(), axis, il).swapaxes(0, 1)
    kr = oracle.rope_rotate(to64(k.transpose(0, 1)), at, f.numpy(), axis, il).swapaxes(0, 1)
    check(qo.cpu()[live], qr[live], q[live], rot, il, "q")
    assert torch.equal(qo.cpu()[~live], keep[~live])                 # padding rows as they were
    phys = table.long()[ids.long().clamp(min=0), pos.long() // 16]
    got_k = kd.cpu()[phys, :, pos.long() % 16][live]
    check(got_k, kr[live], k[live], rot, il, "k")
    vc[phys[live], :, pos.long()[live] % 16] = v[live]
    assert torch.equal(vd.cpu(), vc)                                 # values exact, every other slot untouched
    kc[phys[live], :, pos.long()[live] % 16] = got_k
    assert torch.equal(kd.cpu(), kc)


def test_append_without_queries_or_rotation():
    table, ids, pos, nb, x, q, k, v = map_case([4, 0], [20, 3], 4, 2, 64, 21)
    kd, vd = (torch.zeros(nb, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2))
    a = [t.to(DEV) for t in (table, ids, pos)]
    assert attn.rope_append_paged(None, k.to(DEV), v.to(DEV), kd, vd, *a) is None
    qo = attn.rope_append_paged(q.to(DEV), k.to(DEV), v.to(DEV), kd, vd, *a)
    torch.cuda.synchronize()
    assert torch.equal(qo.cpu(), q)
    phys = table.long()[ids.long(), pos.long() // 16]
    assert torch.equal(kd.cpu()[phys, :, pos.long() % 16], k) and torch.equal(vd.cpu()[phys, :, pos.long() % 16], v)


@pytest.mark.parametrize("group", [None, 32])
def test_bad_rows_are_reported_and_skipped(group):
    """A sequence beyond the table, positions outside it, a table entry outside
    the pool: flagged, nothing written for those rows, the others unharmed."""
    T, Hq, Hkv, d, nb = 6, 4, 2, 64, 5
    table = torch.tensor([[0, 1], [2, 99]], dtype=torch.int32)
    ids = torch.tensor([0, 1, 2, 0, 1, 0], dtype=torch.int32)
    pos = torch.tensor([3, 5, 0, -1, 20, 32], dtype=torch.int32)
    x = randn(31, T, (Hq + 2 * Hkv) * d).to(DEV)
    q, k, v = views(x, Hq, Hkv, d)
    f = workloads.rope_inv_freq(d).to(DEV)
    qo = torch.zeros(T, Hq, d, dtype=BF, device=DEV)
    args = (table.to(DEV), ids.to(DEV), pos.to(DEV))
    attn.device_status()
    if group is None:
        kc = torch.zeros(nb, Hkv, 16, d, dtype=BF, device=DEV)
        vc = torch.zeros_like(kc)
        attn.rope_append_paged(q, k, v, kc, vc, *args, inv_freq=f, q_out=qo)
        torch.cuda.synchronize()
        written = vc.cpu()
        want = torch.zeros(nb, Hkv, 16, d, dtype=BF)
        want[0, :, 3], want[2, :, 5] = v[0].cpu(), v[1].cpu()
        assert torch.equal(written, want)
    else:
        kv = torch.zeros(nb, Hkv, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
        attn.rope_append_paged_kv4(q, k, v, kv, *args, group, inv_freq=f, q_out=qo)
        torch.cuda.synchronize()
        assert torch.all(kv[[1, 3, 4]] == 0) and torch.any(kv[0] != 0) and torch.any(kv[2] != 0)
        rk = torch.full((T, Hkv, d), 7.0, dtype=BF, device=DEV)
        rv = rk.clone()
        flags = attn.ATTN_DEV_BAD_SEQID | attn.ATTN_DEV_BAD_SEQLEN | attn.ATTN_DEV_BAD_BLOCK
        assert attn.device_status() == flags
        attn.kv4_read_paged(kv, *args, d, group, k=rk, v=rv)
        torch.cuda.synchronize()
        assert torch.all(rk[2:] == 7) and torch.all(rv[2:] == 7) and torch.all(rk[:2] != 7)
    assert attn.device_status() == attn.ATTN_DEV_BAD_SEQID | attn.ATTN_DEV_BAD_SEQLEN | attn.ATTN_DEV_BAD_BLOCK
    assert torch.all(qo[:2].float().abs().sum(-1) > 0) and torch.all(qo[2:] == 0)


def test_offsets_beyond_32_bits():
    """Rows more than 2^31 elements from the start of their tensor: head-major
    rotation of a long sequence, and an append of token rows far apart."""
    d, N = 64, (1 << 25) + 1000
    f = workloads.rope_inv_freq(d).to(DEV)
    q = torch.zeros(1, 2, N, d, dtype=BF, device=DEV)
    tail = randn(41, 1, 2, 700, d).to(DEV)
    q[:, :, -700:] = tail
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    out, _ = attn.rope_fwd(q, None, pos, f, q_out=q)
    small, _ = attn.rope_fwd(tail, None, pos[-700:], f)
    torch.cuda.synchronize()
    assert torch.equal(out[:, :, -700:], small) and not out[:, :, :1000].any()
    del q, out
    T, wide, Hkv = 33000, 1 << 16, 2
    x = torch.zeros(T, wide, dtype=BF, device=DEV)
    k, v = x[:, : Hkv * d].view(T, Hkv, d), x[:, 512: 512 + Hkv * d].view(T, Hkv, d)
    k[-50:], v[-50:] = randn(42, 50, Hkv, d).to(DEV), randn(43, 50, Hkv, d).to(DEV)
    table = torch.arange(-(-T // 16), dtype=torch.int32, device=DEV)[None]
    ids, at = torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    kc, vc = (torch.ones(table.shape[1], Hkv, 16, d, dtype=BF, device=DEV) for _ in range(2))
    attn.rope_append_paged(None, k, v, kc, vc, table, ids, at)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    rows = torch.arange(T - 50, T)
    assert torch.equal(kc[rows // 16, :, rows % 16], k[-50:]) and torch.equal(vc[rows // 16, :, rows % 16], v[-50:])
    assert not kc[0].any()
