"""Refusals of the rotary-position and 4-bit-cache calls (CPU): the C entry
points on the host before any device is touched, and the binding before the
library."""

import ctypes
import os
import re

import pytest
import torch

import exact_attention_47_gb300 as attn
from exact_attention_47_gb300 import _binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class _Heads(ctypes.Structure):
    """attn_heads_t"""

    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64), ("stride_token", ctypes.c_int64),
                ("stride_head", ctypes.c_int64), ("heads", ctypes.c_int)]


class _Rope(ctypes.Structure):
    """attn_rope_t"""

    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("positions", ctypes.c_void_p), ("axes", ctypes.c_int), ("stride_axis", ctypes.c_int64),
                ("stride_batch", ctypes.c_int64), ("pair_axis", ctypes.c_char_p)]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(attn.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return attn.load_library()


def test_declared_and_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn47.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:rope|kv4)_[a-z_0-9]+|attn_decode_paged_kv4[a-z_]*)\s*\(", text))
    assert names == {"rope_fwd", "rope_bwd", "rope_append_paged", "rope_append_paged_kv4", "kv4_record_bytes",
                     "kv4_read_paged", "attn_decode_paged_kv4", "attn_decode_paged_kv4_workspace_size"}
    for n in names:
        assert hasattr(lib, n) and n in _binding._SIGS


def test_packed_structures_match_the_header():
    """The binding packs the two structures as bytes: the same size (but for
    the tail padding) and fields as the C ones."""
    h = _Heads.from_buffer_copy(_binding._HEADS.pack(0x10, 1, 2, 3, 4) + bytes(4))
    assert (h.data, h.stride_batch, h.stride_token, h.stride_head, h.heads) == (0x10, 1, 2, 3, 4)
    assert _binding._ROPE.size == ctypes.sizeof(_Rope)
    r = _Rope.from_buffer_copy(_binding._ROPE.pack(0x20, 64, 1, 0x30, 3, 5, 6, 0))
    assert (r.inv_freq, r.rot, r.interleaved, r.positions, r.axes) == (0x20, 64, 1, 0x30, 3)
    assert (r.stride_axis, r.stride_batch, r.pair_axis) == (5, 6, None)


def heads(at, H=2, N=16, d=64, batch=None, token=None, head=None):
    token = H * d if token is None else token
    return _Heads(at, N * token if batch is None else batch, token, d if head is None else head, H)


def rope(rot=64, axes=1, pos=0x9000000, inv=0x8000000, axis=None, stride_axis=16):
    return _Rope(inv, rot, 0, pos, axes, stride_axis, 0, axis)


def ref(x):
    return ctypes.byref(x) if x is not None else None


Q, K, QO, KO = 0x1000000, 0x2000000, 0x3000000, 0x4000000


def fwd(lib, q=None, k=0, qo=None, ko=0, r=None, B=1, N=16, d=64, func="rope_fwd"):
    q = heads(Q) if q is None else q
    k = heads(K) if k == 0 else k
    qo = heads(QO) if qo is None else qo
    ko = heads(KO) if ko == 0 else ko
    r = rope() if r is None else r
    return getattr(lib, func)(ref(q), ref(k), ref(qo), ref(ko), ref(r), B, N, d, None)


@pytest.mark.parametrize("func", ["rope_fwd", "rope_bwd"])
def test_rope_refusals(lib, func):
    def call(**kw):
        return fwd(lib, func=func, **kw)

    assert call(d=96) == UNSUPPORTED
    assert call(B=-1) == INVALID
    assert call(r=rope(rot=24)) == UNSUPPORTED and call(r=rope(rot=0)) == UNSUPPORTED
    assert call(r=rope(rot=80)) == UNSUPPORTED                       # beyond d
    assert call(r=rope(axes=5)) == UNSUPPORTED and call(r=rope(axes=0)) == UNSUPPORTED
    assert call(r=rope(axes=2, axis=bytes([0] * 31 + [2]))) == INVALID
    assert call(r=rope(pos=None)) == INVALID and call(r=rope(inv=None)) == INVALID
    assert call(r=rope(stride_axis=-1)) == INVALID
    assert call(q=heads(Q + 8)) == INVALID                           # misaligned
    assert call(q=heads(Q, token=100)) == INVALID                    # stride not a multiple of 8
    assert call(q=heads(Q, token=-128)) == INVALID
    assert call(q=heads(Q, token=1 << 34)) == UNSUPPORTED
    assert call(q=heads(Q, H=3), qo=heads(QO, H=2)) == INVALID
    assert call(qo=heads(QO, token=64)) == INVALID                   # output rows overlap
    assert "overlap" in lib.attn_last_error().decode()
    assert call(qo=heads(QO, token=0)) == INVALID
    assert call(ko=None) == INVALID                                  # k without k_out
    assert call(qo=heads(Q, token=256)) == INVALID                   # over its input with other strides
    assert call(qo=heads(Q + 128)) == INVALID                        # shifted over its input
    assert call(qo=heads(K)) == INVALID                              # over k
    assert call(ko=heads(QO)) == INVALID                             # over q_out
    assert call(B=0) == OK and call(N=0) == OK


def test_merged_parts_are_told_apart(lib):
    """q and k inside one merged buffer, rotated in place: not refused for
    overlapping (the call then fails on the missing device, not on arguments)."""
    q, k = heads(Q, token=512), heads(Q + 2 * 128, token=512)
    assert fwd(lib, q=q, k=k, qo=q, ko=k) not in (INVALID, UNSUPPORTED, OK)
    k2 = heads(Q + 2 * 64, token=512)                                # starts inside q's rows
    assert fwd(lib, q=q, k=k2, qo=q, ko=k2) == INVALID


def passes(lib, status):
    """The arguments are accepted: the call got as far as the missing device or,
    where there is one, to these addresses not being its memory."""
    return status == 3 or (status == INVALID and
                           re.search("is not (device memory|memory of device)", lib.attn_last_error().decode()) is not None)


def part(at, H, token, head=64, batch=0, d=64):
    return _Heads(at, batch, token, head, H)


@pytest.mark.parametrize("token", [0, 512])
def test_merged_parts_of_one_token_a_batch_are_told_apart(lib, token):
    """A decode step's [B, 1, (Hq + 2 Hkv) d]: one token, whose stride means
    nothing."""
    q, k = part(Q, 2, token, batch=512), part(Q + 2 * 128, 2, token, batch=512)
    assert passes(lib, fwd(lib, q=q, k=k, qo=q, ko=k, B=4, N=1))
    over = part(Q + 2 * 64, 2, token, batch=512)
    assert fwd(lib, q=q, k=over, qo=q, ko=over, B=4, N=1) == INVALID
    last = part(Q + 2 * 448, 2, token, batch=512)                    # its second head is the next batch's first
    assert fwd(lib, q=q, k=last, qo=q, ko=last, B=4, N=1) == INVALID


def test_head_major_parts_are_told_apart(lib):
    """Heads of one [B, H, N, d] buffer."""
    B, N, d = 3, 16, 64
    for k_first, ok in ((2, True), (1, False), (4, False)):          # of 5 heads, q has 2, k 2
        q = part(Q, 2, d, head=N * d, batch=5 * N * d)
        k = part(Q + 2 * k_first * N * d, 2, d, head=N * d, batch=5 * N * d)
        st = fwd(lib, q=q, k=k, qo=q, ko=k, B=B, N=N)
        assert passes(lib, st) == ok and st != UNSUPPORTED
    # q and k as halves of every token of a head: [B, H, N, 2, d]
    q, k = (part(Q + 2 * i * d, 2, 2 * d, head=2 * N * d, batch=4 * N * d) for i in range(2))
    assert passes(lib, fwd(lib, q=q, k=k, qo=q, ko=k, B=B, N=N))


@pytest.mark.parametrize("B,N", [(1, 1), (1, 7), (3, 7), (3, 1)])
def test_parts_interleaved_by_head_are_told_apart(lib, B, N):
    """A projection seen as [B, N, H, 3, d]."""
    H, d = 5, 64
    qkv = [part(Q + 2 * i * d, H, 3 * H * d, head=3 * d, batch=3 * N * H * d) for i in range(3)]
    for func in ("rope_fwd", "rope_bwd"):
        assert passes(lib, fwd(lib, q=qkv[0], k=qkv[1], qo=qkv[0], ko=qkv[1], B=B, N=N, func=func))
        apart = [heads(QO, H=H, N=N), heads(KO, H=H, N=N)]
        assert passes(lib, fwd(lib, q=apart[0], k=apart[1], qo=qkv[0], ko=qkv[1], B=B, N=N, func=func))
        near = part(Q + 2 * (d + 8), H, 3 * H * d, head=3 * d, batch=3 * N * H * d)   # 8 elements into the third part
        assert fwd(lib, q=qkv[0], k=qkv[1], qo=qkv[2], ko=near, B=B, N=N, func=func) == INVALID
    if B == 1:
        assert passes(lib, append(lib, q=qkv[0], k=qkv[1], v=qkv[2], qo=qkv[0], T=N))
        assert append(lib, q=qkv[0], k=qkv[1], v=qkv[2], qo=qkv[2], T=N) == INVALID


def test_views_are_told_apart_as_their_elements_are(lib):
    """Random small views in one buffer against sets of their elements."""
    import random
    rng = random.Random(5)
    B, N, d = 2, 3, 64
    seen = [0, 0]
    for _ in range(3000):
        base = rng.choice([64, 128, 192, 384])
        steps = [base, base * rng.choice([2, 3, 5]), base * rng.choice([6, 8, 15])]
        views = []
        for v in range(2):
            token, head, batch = rng.sample(steps, 3) if rng.random() < 0.5 else steps
            views.append(part(Q + 2 * 8 * rng.randrange(0, 600), rng.choice([1, 2, 4]), token, head, batch))

        def elements(v):
            return [(v.data - Q) // 2 + b * v.stride_batch + n * v.stride_token + h * v.stride_head + e
                    for b in range(B) for n in range(N) for h in range(v.heads) for e in range(0, d, 8)]

        mine, other = (elements(v) for v in views)
        if len(set(mine)) < len(mine):
            continue                                                 # rows of the output that overlap each other
        q = part(0x40000000, views[0].heads, 4 * 64, batch=12 * 64)
        st = fwd(lib, q=q, k=views[1], qo=views[0], ko=part(0x50000000, views[1].heads, 4 * 64, batch=12 * 64), B=B, N=N)
        if st == INVALID and "rows overlap each other" in lib.attn_last_error().decode():
            continue
        shares = not set(mine).isdisjoint(other)
        assert passes(lib, st) != shares and st not in (UNSUPPORTED, OK)
        seen[shares] += 1
    assert min(seen) > 200


KC, VC, TAB, IDS, POS = (ctypes.c_void_p(0x20000000 + i * 0x1000000) for i in range(5))


def append(lib, q=0, k=None, v=None, qo=0, r=0, kc=KC, vc=VC, T=8, S=2, d=64, bs=16, mb=4, nb=8, ids=IDS, group=None):
    q = heads(Q, N=T) if q == 0 else q
    k = heads(K, N=T) if k is None else k
    v = heads(K + 0x100000, N=T) if v is None else v
    qo = heads(QO, N=T) if qo == 0 else qo
    r = rope() if r == 0 else r
    if group is not None:
        return lib.rope_append_paged_kv4(ref(q), ref(k), ref(v), ref(qo), ref(r), kc, group, TAB, ids, POS, T, S, d, bs,
                                         mb, nb, None)
    return lib.rope_append_paged(ref(q), ref(k), ref(v), ref(qo), ref(r), kc, vc, TAB, ids, POS, T, S, d, bs, mb, nb,
                                 None)


@pytest.mark.parametrize("group", [None, 32, 64])
def test_append_refusals(lib, group):
    def call(**kw):
        return append(lib, group=group, **kw)

    assert call(bs=8) == UNSUPPORTED and call(d=80) == UNSUPPORTED
    assert call(T=-1) == INVALID and call(S=0) == INVALID and call(mb=0) == INVALID and call(nb=0) == INVALID
    assert call(mb=1 << 27) == UNSUPPORTED
    assert call(v=heads(K + 0x100000, H=3)) == INVALID
    assert call(qo=None) == INVALID
    assert call(kc=None) == INVALID and call(kc=ctypes.c_void_p(0x20000008)) == INVALID
    assert call(ids=None) == INVALID and call(ids=ctypes.c_void_p(0x20000002)) == INVALID
    assert call(qo=heads(K)) == INVALID                              # q_out over k
    assert call(kc=ctypes.c_void_p(K)) == INVALID                    # cache over k
    assert call(r=rope(rot=40)) == UNSUPPORTED
    assert call(r=rope(axes=3, pos=None, axis=bytes(32))) == INVALID
    if group is None:
        assert call(vc=KC) == INVALID
    assert call(T=0) == OK


def test_group_is_checked(lib):
    assert append(lib, group=16) == UNSUPPORTED and append(lib, group=128) == UNSUPPORTED
    assert lib.kv4_record_bytes(128, 16) == 0 and lib.kv4_record_bytes(96, 32) == 0
    for d in (64, 128):
        for g in (32, 64):
            assert lib.kv4_record_bytes(d, g) == 16 * d + 128 * (d // g)


def read(lib, kv=KC, k=0x5000000, v=0x6000000, T=8, S=2, Hkv=2, d=64, group=32, bs=16, mb=4, nb=8):
    return lib.kv4_read_paged(kv, group, TAB, IDS, POS, k, v, T, S, Hkv, d, bs, mb, nb, None)


def test_read_refusals(lib):
    assert read(lib, group=48) == UNSUPPORTED and read(lib, d=32) == UNSUPPORTED and read(lib, bs=32) == UNSUPPORTED
    assert read(lib, T=-1) == INVALID and read(lib, Hkv=0) == INVALID
    assert read(lib, k=None) == INVALID and read(lib, v=0x6000004) == INVALID
    assert read(lib, v=0x5000010) == INVALID                         # k and v overlap
    assert read(lib, k=0x20000000) == INVALID                        # over the cache
    assert read(lib, T=0) == OK


def decode(lib, S=2, Hq=12, Hkv=2, d=128, group=32, bs=16, mb=4, nb=8, scale=0.1, ws=0x7000000, ws_bytes=None,
           o=0x5000000):
    need = lib.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d)
    return lib.attn_decode_paged_kv4(Q, KC, TAB, IDS, S, Hq, Hkv, d, group, bs, mb, nb, scale, o, None, ws,
                                     need if ws_bytes is None else ws_bytes, None)


def test_decode_refusals(lib):
    assert decode(lib, group=128) == UNSUPPORTED and decode(lib, d=80) == UNSUPPORTED and decode(lib, bs=8) == UNSUPPORTED
    assert decode(lib, Hq=34) == UNSUPPORTED and decode(lib, mb=1 << 27) == UNSUPPORTED
    assert decode(lib, Hq=13) == INVALID and decode(lib, S=-1) == INVALID and decode(lib, nb=0) == INVALID
    assert decode(lib, scale=0.0) == INVALID and decode(lib, scale=float("inf")) == INVALID
    assert decode(lib, o=None) == INVALID and decode(lib, ws=None) == INVALID and decode(lib, ws=0x7000008) == INVALID
    assert decode(lib, ws_bytes=64) == WORKSPACE
    assert decode(lib, o=0x7000000) == INVALID and "overlaps" in lib.attn_last_error().decode()
    assert decode(lib, S=0) == OK
    size = lib.attn_decode_paged_kv4_workspace_size
    assert size(5, 12, 2, 128) == size(500, 12, 2, 128) == 256 * 8 + 512 * 6 * 130 * 4
    assert size(0, 12, 2, 128) == 0


def test_decode_outputs_keep_off_the_inputs(lib):
    """O and LSE over the queries, the cache, the table, the lengths or each
    other: other warps may still be reading there."""
    need = lib.attn_decode_paged_kv4_workspace_size(2, 12, 2, 128)

    def call(o, lse):
        return lib.attn_decode_paged_kv4(Q, KC, TAB, IDS, 2, 12, 2, 128, 32, 16, 4, 8, 0.1, o, lse, 0x7000000, need, None)

    assert call(0x5000000, 0x6000000) not in (INVALID, UNSUPPORTED, OK)      # apart: it fails on the missing device
    for at in (Q, KC.value + 256, TAB.value, IDS.value):
        assert call(at, None) == INVALID and "o overlaps" in lib.attn_last_error().decode()
        assert call(0x5000000, at) == INVALID and "lse overlaps" in lib.attn_last_error().decode()
    assert call(0x5000000, 0x5000000 + 2 * 12 * 128 * 2 - 4) == INVALID


def test_read_outputs_keep_off_the_token_map(lib):
    for at in (TAB.value, IDS.value, POS.value):
        assert read(lib, k=at) == INVALID and "overlap" in lib.attn_last_error().decode()
        assert read(lib, v=at) == INVALID


@pytest.mark.parametrize("func", ["rope_fwd", "rope_bwd"])
def test_rotations_keep_off_positions_and_frequencies(lib, func):
    """Other warps may still be reading there."""
    B, N, d, far = 2, 16, 64, 0x9000000
    for axes, stride_axis, stride_batch in ((1, 0, 16), (1, 0, 0), (3, 64, 16)):
        r = _Rope(0x8000000, 64, 0, far, axes, stride_axis, stride_batch, bytes(32) if axes > 1 else None)
        assert passes(lib, fwd(lib, r=r, B=B, func=func))
        last = far + 4 * ((axes - 1) * stride_axis + (B - 1) * stride_batch) + 4 * (N - 4)   # the last 16 bytes
        for at in (far, last, 0x8000000, 0x8000000 + 112):
            for kw in (dict(qo=heads(at)), dict(ko=heads(at))):
                assert fwd(lib, r=r, B=B, func=func, **kw) == INVALID
                assert "overlaps" in lib.attn_last_error().decode()
    # between the positions of two axes, or among rows with room between them: apart
    r = _Rope(0x8000000, 64, 0, far, 2, 1 << 20, 0, bytes(32))
    assert passes(lib, fwd(lib, r=r, func=func, qo=heads(far + (1 << 20))))
    assert passes(lib, fwd(lib, r=rope(pos=QO + 256), func=func, qo=heads(QO, token=512)))


@pytest.mark.parametrize("group", [None, 32])
def test_appends_keep_off_what_they_read(lib, group):
    T, d = 8, 64
    cache = 8 * 2 * 16 * d * 2
    r = rope()
    for at in (TAB.value, TAB.value + 16, IDS.value, POS.value, POS.value + 16, 0x8000000, 0x9000000):
        assert append(lib, group=group, qo=heads(at, N=T), r=r) == INVALID
        assert "q_out overlaps" in lib.attn_last_error().decode()
        assert append(lib, group=group, kc=ctypes.c_void_p(at), r=r) == INVALID
        assert "the cache overlaps" in lib.attn_last_error().decode()
        if group is None:
            assert append(lib, vc=ctypes.c_void_p(at - cache + 16), r=r) == INVALID
    own = _Rope(0x8000000, 64, 0, None, 1, 0, 0, None)               # turned by the cache's positions
    for x in (r, own, None):
        assert passes(lib, append(lib, group=group, r=x))


# ------------------------------------------------------------------ binding
class _OnCuda0(torch.Tensor):
    """A CPU tensor that claims to be on cuda:0 (it never reaches the library)."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 0)


def dev(shape, dtype):
    return torch.Tensor._make_subclass(_OnCuda0, torch.zeros(shape, dtype=dtype))


@pytest.fixture
def no_library_calls(monkeypatch, lib):
    def refuse(func, device, *args):
        raise AssertionError("%s reached the library with bad arguments" % func)

    monkeypatch.setattr(_binding, "_call", refuse)


def test_binding_refuses_rope(no_library_calls):
    q, k, f, pos = dev((2, 4, 8, 64), BF), dev((2, 2, 8, 64), BF), dev((32,), F32), dev((8,), I32)
    out = dict(q_out=dev((2, 4, 8, 64), BF), k_out=dev((2, 2, 8, 64), BF))
    for bad, match in [
        (dict(q=dev((2, 4, 8, 64), F32)), "q must be torch.bfloat16"),
        (dict(q=torch.zeros((2, 4, 8, 64), dtype=BF)), "q must be a CUDA tensor"),
        (dict(q=dev((4, 8, 64), BF)), r"q must be \[B, H, N, d\]"),
        (dict(k=dev((2, 2, 9, 64), BF)), "k must be"),
        (dict(q=dev((2, 4, 8, 128), BF)[..., ::2]), "contiguous last dimension"),
        (dict(positions=dev((9,), I32)), "positions of an axis"),
        (dict(positions=dev((8,), torch.int64)), "positions must be torch.int32"),
        (dict(positions=dev((3, 9), I32), pair_axis=[0] * 32), "positions of an axis"),
        (dict(pair_axis=[0] * 31, positions=dev((3, 8), I32)), "pair_axis has 31"),
        (dict(inv_freq=dev((32,), BF)), "inv_freq must be torch.float32"),
        (dict(q_out=dev((2, 4, 8, 128), BF)), "q_out must have shape"),
        (dict(k=None), "k_out without its input"),
    ]:
        args = dict(dict(q=q, k=k, positions=pos, inv_freq=f), **out, **{})
        args.update(bad)
        with pytest.raises(ValueError, match=match):
            attn.rope_fwd(**args)
    with pytest.raises(ValueError):
        attn.rope_fwd(q, k, dev((3, 8), I32), f, pair_axis=[300] * 32, **out)


def test_binding_refuses_append_read_decode(no_library_calls):
    T, S, Hq, Hkv, d = 6, 2, 4, 2, 64
    rec = attn.kv4_record_bytes(d, 32)
    base = dict(q=dev((T, Hq, d), BF), k=dev((T, Hkv, d), BF), v=dev((T, Hkv, d), BF), block_table=dev((S, 4), I32),
                seq_ids=dev((T,), I32), positions=dev((T,), I32), inv_freq=dev((32,), F32), q_out=dev((T, Hq, d), BF))
    bf = dict(k_cache=dev((9, Hkv, 16, d), BF), v_cache=dev((9, Hkv, 16, d), BF))
    k4 = dict(kv_cache=dev((9, Hkv, rec), U8), group=32)
    shared = [(dict(v=dev((T, Hkv + 1, d), BF)), "same shape"), (dict(seq_ids=dev((T + 1,), I32)), "seq_ids must have"),
              (dict(positions=dev((T,), torch.int64)), "positions must be torch.int32"),
              (dict(block_table=dev((S,), I32)), "block_table must be"), (dict(q=None), "q_out without q"),
              (dict(inv_freq=None, rope_positions=dev((T,), I32)), "need inv_freq"),
              (dict(pair_axis=[0] * 32), "needs positions"), (dict(q=dev((T, Hq, 128), BF)), "q must be")]
    for func, own, more in (
            (attn.rope_append_paged, bf, [(dict(v_cache=dev((8, Hkv, 16, d), BF)), "caches"),
                                          (dict(k_cache=dev((9, 1, 16, d), BF), v_cache=dev((9, 1, 16, d), BF)), "k's heads")]),
            (attn.rope_append_paged_kv4, k4, [(dict(kv_cache=dev((9, Hkv, rec + 16), U8)), "kv_cache must be"),
                                              (dict(kv_cache=dev((9, Hkv, rec), torch.int8)), "kv_cache must be torch.uint8"),
                                              (dict(kv_cache=dev((9, 3, rec), U8)), "k's heads"), (dict(group=16), "groups of 32 or 64")])):
        for bad, match in shared + more:
            with pytest.raises(ValueError, match=match):
                func(**dict(base, **own, **{}) | bad)
    r = dict(kv_cache=k4["kv_cache"], block_table=base["block_table"], seq_ids=base["seq_ids"],
             positions=base["positions"], d=d, group=32, k=dev((T, Hkv, d), BF), v=dev((T, Hkv, d), BF))
    for bad, match in [(dict(d=128), "kv_cache must be"), (dict(k=dev((T, Hkv, 128), BF)), "k must have shape"),
                       (dict(seq_ids=dev((T, 1), I32)), "seq_ids must be")]:
        with pytest.raises(ValueError, match=match):
            attn.kv4_read_paged(**(r | bad))
    need = attn.attn_decode_paged_kv4_workspace_size(S, Hq, Hkv, d)
    c = dict(q=dev((S, Hq, d), BF), kv_cache=k4["kv_cache"], block_table=base["block_table"], seq_lens=dev((S,), I32),
             group=32, o=dev((S, Hq, d), BF), lse=dev((S, Hq), F32), workspace=dev((need,), U8))
    for bad, match in [(dict(group=64), "kv_cache must be"), (dict(seq_lens=dev((3,), I32)), "seq_lens must have"),
                       (dict(workspace=dev((need - 16,), U8)), "workspace has"), (dict(o=dev((S, Hq, 128), BF)), "o must have")]:
        with pytest.raises(ValueError, match=match):
            attn.attn_decode_paged_kv4(**(c | bad))


def test_fast_calls_leave_the_unusual_to_the_binding(lib):
    """CPU tensors, other types and counts: None each time, nothing raised."""
    fast = _binding._fast()
    f32, i32 = torch.zeros(8), torch.zeros(8, dtype=I32)
    for f, n in ((fast.rope, 9), (fast.append, 14), (fast.read, 8), (fast.decode, 10)):
        for fill in (None, True, 3, 2 ** 80, "x", f32, i32, torch.zeros((2, 4, 8, 64), dtype=BF), f32.to("meta")):
            for count in (0, n - 1, n, n + 1):
                assert f(*[fill] * count) is None
    q = torch.zeros((2, 4, 8, 64), dtype=BF)
    assert fast.rope(False, q, None, i32, torch.zeros(32), None, False, None, None) is None
    with pytest.raises(TypeError):
        fast.bind(1)
    with pytest.raises(ValueError):
        fast.bind(*[0] * 8)
