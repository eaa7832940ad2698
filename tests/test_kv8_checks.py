"""The 8-bit cache's entry points refuse bad arguments on the host before any
device is touched, and the binding before the library.  CPU."""

import ctypes

import pytest
import torch

import exact_attention_47_gb300 as attn
from exact_attention_47_gb300 import _binding
from test_rope_kv4_checks import (BF, F32, I32, INVALID, K, OK, Q, QO, U8, UNSUPPORTED, dev, heads, lib,  # noqa: F401
                                  no_library_calls, passes, ref, rope)

V, TAB, IDS, POS, KV, OUT = 0x5000000, 0x6000000, 0x6100000, 0x6200000, 0x20000000, 0x7000000


def test_exported_and_sized(lib):  # noqa: F811
    for n in ("kv8_record_bytes", "kv8_append_paged", "kv8_read_paged"):
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
