"""The 8-bit cache's entry points refuse bad arguments on the host before any
device is touched, and the binding before the library.  CPU."""

import ctypes

import pytest
import torch

import exact_attention_47_gb300 as attn
from exact_attention_47_gb300 import _binding
from test_rope_kv4_checks import (BF, F32, I32, INVALID, K, OK, Q, QO, U8, UNSUPPORTED, WORKSPACE, dev,  # noqa: F401
                                  heads, lib, no_library_calls, passes, ref, rope)

V, TAB, IDS, POS, KV, OUT = 0x5000000, 0x6000000, 0x6100000, 0x6200000, 0x20000000, 0x7000000


def test_exported_and_sized(lib):  # noqa: F811
    for n in ("kv8_record_bytes", "kv8_append_paged", "kv8_read_paged", "attn_decode_paged_kv8", "attn_prefill_paged_kv8",
              "attn_decode_paged_kv8_workspace_size", "attn_prefill_paged_kv8_workspace_size"):
        assert hasattr(lib, n) and n in _binding._SIGS
    assert lib.kv8_record_bytes(128) == 4128 and lib.kv8_record_bytes(64) == 2080
    assert lib.kv8_record_bytes(96) == 0 and lib.kv8_record_bytes(0) == 0
    with pytest.raises(ValueError, match="8-bit cache has d 64 or 128"):
        attn.kv8_record_bytes(32)


def append(lib, q=0, k=0, v=0, qo=0, r=None, kv=KV, tab=TAB, ids=IDS, pos=POS, T=16, S=2, d=64, bs=16, mb=4, nb=8):  # noqa: F811
    q, k, v, qo = (heads(at) if h == 0 else h for at, h in ((Q, q), (K, k), (V, v), (QO, qo)))
    return lib.kv8_append_paged(ref(q), ref(k), ref(v), ref(qo), ref(r), kv, tab, ids, pos, T, S, d, bs, mb, nb, None)


def test_append_refusals(lib):  # noqa: F811
    assert passes(lib, append(lib)) and passes(lib, append(lib, q=None, qo=None, r=rope(pos=None)))
    assert append(lib, d=96) == UNSUPPORTED and append(lib, bs=32) == UNSUPPORTED
    assert append(lib, T=-1) == INVALID and append(lib, S=0) == INVALID and append(lib, nb=0) == INVALID
    assert append(lib, kv=None) == INVALID and append(lib, kv=KV + 8) == INVALID
    assert append(lib, tab=None) == INVALID and append(lib, ids=IDS + 2) == INVALID
    assert append(lib, mb=1 << 28) == UNSUPPORTED
    assert append(lib, q=None) == INVALID and append(lib, qo=None) == INVALID
    assert append(lib, v=heads(V, H=3)) == INVALID
    assert append(lib, qo=heads(K)) == INVALID                       # over k
    size = 8 * 2 * 2080
    assert append(lib, kv=K - size + 16) == INVALID                  # the last record ends inside k
    assert passes(lib, append(lib, kv=K - size))
    assert append(lib, kv=TAB - size + 16) == INVALID and append(lib, kv=POS) == INVALID
    assert append(lib, r=rope(rot=24)) == UNSUPPORTED
    assert append(lib, T=0) == OK


def read(lib, kv=KV, tab=TAB, ids=IDS, pos=POS, k=OUT, v=OUT + 0x100000, T=16, S=2, Hkv=2, d=64, bs=16, mb=4, nb=8):  # noqa: F811
    return lib.kv8_read_paged(kv, tab, ids, pos, k, v, T, S, Hkv, d, bs, mb, nb, None)


def test_read_refusals(lib):  # noqa: F811
    assert passes(lib, read(lib))
    assert read(lib, d=32) == UNSUPPORTED and read(lib, bs=8) == UNSUPPORTED
    assert read(lib, Hkv=0) == INVALID and read(lib, T=-1) == INVALID
    assert read(lib, k=None) == INVALID and read(lib, v=OUT + 8) == INVALID
    assert read(lib, v=OUT + 16) == INVALID                          # k and v overlap
    assert read(lib, k=KV + 2080) == INVALID and read(lib, v=IDS) == INVALID
    assert read(lib, T=0) == OK


def test_binding_refuses_append_and_read(no_library_calls):  # noqa: F811
    T, S, Hq, Hkv, d = 6, 2, 4, 2, 64
    rec = attn.kv8_record_bytes(d)
    base = dict(q=dev((T, Hq, d), BF), k=dev((T, Hkv, d), BF), v=dev((T, Hkv, d), BF), kv_cache=dev((9, Hkv, rec), U8),
                block_table=dev((S, 4), I32), seq_ids=dev((T,), I32), positions=dev((T,), I32),
                inv_freq=dev((32,), F32), q_out=dev((T, Hq, d), BF))
    for bad, match in [(dict(v=dev((T, Hkv + 1, d), BF)), "same shape"), (dict(seq_ids=dev((T + 1,), I32)), "seq_ids must have"),
                       (dict(positions=dev((T,), torch.int64)), "positions must be torch.int32"),
                       (dict(block_table=dev((S,), I32)), "block_table must be"), (dict(q=None), "q_out without q"),
                       (dict(inv_freq=None, rope_positions=dev((T,), I32)), "need inv_freq"),
                       (dict(kv_cache=dev((9, Hkv, rec + 16), U8)), "kv_cache must be"),
                       (dict(kv_cache=dev((9, Hkv, rec), torch.int8)), "kv_cache must be torch.uint8"),
                       (dict(kv_cache=dev((9, 3, rec), U8)), "k's heads"),
                       (dict(kv_cache=torch.zeros((9, Hkv, rec), dtype=U8)), "kv_cache must be a CUDA tensor")]:
        with pytest.raises(ValueError, match=match):
            attn.kv8_append_paged(**(base | bad))
    r = {n: base[n] for n in ("kv_cache", "block_table", "seq_ids", "positions")}
    r.update(d=d, k=dev((T, Hkv, d), BF), v=dev((T, Hkv, d), BF))
    for bad, match in [(dict(d=128), "kv_cache must be"), (dict(k=dev((T, Hkv, 128), BF)), "k must have shape"),
                       (dict(seq_ids=dev((T, 1), I32)), "seq_ids must be"), (dict(d=48), "8-bit cache has d")]:
        with pytest.raises(ValueError, match=match):
            attn.kv8_read_paged(**(r | bad))


O, LSE, WS = 0x8000000, 0x9000000, 0xA000000


def attend(lib, N=None, S=2, Hq=12, Hkv=2, d=128, bs=16, mb=4, nb=8, scale=0.1, q=Q, kv=KV, tab=TAB, lens=IDS, o=O,  # noqa: F811
           lse=LSE, ws=WS, ws_bytes=None):
    if N is None:
        need = lib.attn_decode_paged_kv8_workspace_size(S, Hq, Hkv, d)
        f, n = lib.attn_decode_paged_kv8, ()
    else:
        need = lib.attn_prefill_paged_kv8_workspace_size(S, Hq, Hkv, N, d)
        f, n = lib.attn_prefill_paged_kv8, (N,)
    return f(q, kv, tab, lens, S, Hq, Hkv, *n, d, bs, mb, nb, scale, o, lse, ws, need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("N", [None, 1, 4, 300])
def test_attention_refusals(lib, N):  # noqa: F811
    def call(**kw):
        return attend(lib, N, **kw)

    assert passes(lib, call()) and passes(lib, call(lse=None)) and passes(lib, call(d=64, Hq=7, Hkv=7))
    assert call(d=80) == UNSUPPORTED and call(bs=8) == UNSUPPORTED and call(mb=1 << 27) == UNSUPPORTED
    assert call(Hq=13) == INVALID and call(S=-1) == INVALID and call(nb=0) == INVALID and call(Hkv=0) == INVALID
    assert call(scale=0.0) == INVALID and call(scale=float("nan")) == INVALID and call(scale=float("inf")) == INVALID
    for x in (dict(q=None), dict(kv=None), dict(tab=None), dict(lens=None), dict(o=None), dict(q=Q + 8), dict(kv=KV + 4),
              dict(o=O + 2), dict(tab=TAB + 1), dict(lens=IDS + 2), dict(lse=LSE + 2)):
        assert call(**x) == INVALID, x
    assert call(nb=1 << 30) == UNSUPPORTED and call(S=1 << 24, Hq=1 << 8, Hkv=1 << 8) == UNSUPPORTED
    assert call(S=0) == OK
    # Outputs over what is read, or each other.
    for at in (Q, KV + 256, TAB, IDS):
        assert call(o=at) == INVALID and "o overlaps" in lib.attn_last_error().decode()
        assert call(lse=at) == INVALID and "lse overlaps" in lib.attn_last_error().decode()
    assert call(lse=O + 64) == INVALID
    cache = 8 * 2 * 4128
    assert call(kv=O - cache + 16) == INVALID and passes(lib, call(kv=O - cache))
    assert call(ws=None) == INVALID and call(ws=WS + 8) == INVALID and call(ws_bytes=64) == WORKSPACE
    assert call(ws=Q) == INVALID and call(o=WS) == INVALID and call(lse=WS + 64) == INVALID


def test_prefill_of_its_own(lib):  # noqa: F811
    assert attend(lib, -1) == INVALID and attend(lib, 0) == OK
    assert attend(lib, 1 << 30) == UNSUPPORTED and attend(lib, 1 << 20, S=1 << 10) == UNSUPPORTED
    # More than 16 query heads to a KV head: the prefill's alone.
    assert attend(lib, None, Hq=34) == UNSUPPORTED and passes(lib, attend(lib, 1, Hq=34))
    # More blocks in all passes than 31 bits count: tiles.
    wide = dict(S=1000, Hq=32, Hkv=8, d=64, mb=1 << 17, nb=1 << 20, q=0x10000000000, o=0x20000000000, lse=None,
                kv=0x30000000000, tab=0x40000000000)
    assert passes(lib, attend(lib, 20, **wide)) and passes(lib, attend(lib, 20, ws=None, ws_bytes=0, **wide))
    assert attend(lib, 8, ws=None, ws_bytes=0, **wide) == INVALID
    assert attend(lib, 20, **(wide | dict(S=1 << 12))) == UNSUPPORTED
    # Many rows in all go in tiles, without a workspace.
    assert passes(lib, attend(lib, 2000, S=4, o=0x40000000, lse=None, ws=None, ws_bytes=0))


def test_workspace_sizes(lib):  # noqa: F811
    decode, prefill = lib.attn_decode_paged_kv8_workspace_size, lib.attn_prefill_paged_kv8_workspace_size
    for d, passes in ((64, {16: 1, 17: 1, 24: 1, 25: 2, 32: 2, 64: 4, 71: 3, 240: 10}),
                      (128, {8: 1, 16: 1, 17: 2, 32: 2, 47: 3, 160: 10})):
        for group in (1, 6, 16):
            assert decode(5, 2 * group, 2, d) == decode(500, 2 * group, 2, d) == 256 * 8 + 512 * group * (d + 2) * 4
            assert prefill(5, 2 * group, 2, 1, d) == decode(5, 2 * group, 2, d)
        # Groups of as equal sizes as can be.
        for rows, groups in passes.items():
            assert prefill(1, 1, 1, rows, d) == 256 * 8 + 512 * -(-rows // groups) * (d + 2) * 4
    for bad in ((0, 12, 2, 128), (2, 12, 5, 128), (2, 0, 2, 128), (2, 12, 2, 0)):
        assert decode(*bad) == 0 and prefill(*bad[:3], 4, bad[3]) == 0
    assert prefill(2, 12, 2, 0, 128) == 0 and prefill(2, 12, 2, 1 << 30, 128) == 0
    # Tiles: d = 128: more than 3 passes for each CTA of a wave of 152.
    for S, waves in ((1, 1), (40, 1), (76, 1), (77, 2)):
        last = 3 * 152 * waves // (2 * S) * 16               # rows of a KV head
        if last <= 256:
            assert prefill(S, 2, 2, last, 128) > 0 and prefill(S, 2, 2, last + 1, 128) == 0


def test_binding_refuses_attention(no_library_calls):  # noqa: F811
    S, Hq, Hkv, d, N = 2, 4, 2, 64, 3
    rec = attn.kv8_record_bytes(d)
    for f, shape in ((attn.attn_decode_paged_kv8, (S, Hq, d)), (attn.attn_prefill_paged_kv8, (S, Hq, N, d))):
        base = dict(q=dev(shape, BF), kv_cache=dev((9, Hkv, rec), U8), block_table=dev((S, 4), I32), seq_lens=dev((S,), I32),
                    o=dev(shape, BF), lse=dev(shape[:-1], F32))
        for bad, match in [(dict(q=dev(shape, F32)), "q must be torch.bfloat16"), (dict(q=dev((S, d), BF)), r"q must be \[S"),
                           (dict(kv_cache=dev((9, Hkv, rec - 16), U8)), "kv_cache must be"),
                           (dict(kv_cache=dev((9, Hkv, rec), torch.int8)), "kv_cache must be torch.uint8"),
                           (dict(block_table=dev((S + 1, 4), I32)), "block_table must be"),
                           (dict(block_table=dev((S, 4), torch.int64)), "block_table must be torch.int32"),
                           (dict(seq_lens=dev((S + 1,), I32)), "seq_lens must have"),
                           (dict(o=dev(shape, F32)), "o must be torch.bfloat16"),
                           (dict(o=dev(shape[:-1] + (d + 1,), BF)), "o must have"),
                           (dict(lse=dev(shape, F32)), "lse must have"),
                           (dict(seq_lens=torch.zeros(S, dtype=I32)), "seq_lens must be a CUDA tensor")]:
            with pytest.raises(ValueError, match=match):
                f(**(base | bad))
