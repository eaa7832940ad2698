"""The 8-bit cache's calls both ways, through csrc/fast_calls.cpp and the Python
one: the same bytes, the Python way's errors, a failed launch reported once.
Streams, threads and memory of their own."""

import ctypes
import threading

import pytest
import torch

import exact_attention_47_gb300 as attn
import workloads
from exact_attention_47_gb300 import _binding
from test_gpu_fast_calls import both, fast_only  # noqa: F401
from test_gpu_kv8_attention import case
from test_gpu_rope import map_case, randn, views

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def on_gpu(*args, **kw):
    return tuple(t.to(DEV) for t in case(*args, **kw))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [False, True])
def test_append_read(fast_only, d, queries):  # noqa: F811
    Hq, Hkv = 6, 2
    table, ids, pos, nb, x, q, k, v = map_case([0, 21], [5, 40], Hq, Hkv, d, 3, padding=1)
    q, k, v = views(x.to(DEV), Hq, Hkv, d)
    table, ids, pos = (t.to(DEV) for t in (table, ids, pos))
    f = workloads.rope_inv_freq(d).to(DEV)
    axis = [p % 2 for p in range(d // 2)]
    q = q if queries else None
    out = torch.zeros(x.shape[0], Hq, d, dtype=BF, device=DEV) if queries else None   # padding rows stay zero
    for rot in (dict(), dict(inv_freq=f, rope_positions=pos), dict(
            inv_freq=f, rope_positions=torch.stack([pos, pos + 3]), pair_axis=axis, interleaved=True)):
        kv = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2).to(DEV)
        kv = both(fast_only, lambda s, c: attn.kv8_append_paged(q, k, v, c, table, ids, pos, q_out=out, stream=s, **rot),
                  kv)[-1]
        T = 45
        both(fast_only, lambda s: attn.kv8_read_paged(kv, table, ids[:T], pos[:T], d, stream=s))
        mine = [torch.empty(T, Hkv, d, dtype=BF, device=DEV) for _ in range(2)]
        assert attn.kv8_read_paged(kv, table, ids[:T], pos[:T], d, *mine)[0] is mine[0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [None, 3, 300])
def test_attention(fast_only, d, N):  # noqa: F811
    lens = [1, 0, 300, 77] * (1 if N != 300 else 8)
    Hq, Hkv = 8, 2
    args = on_gpu(lens, Hq, Hkv, d, seed=5, N=N)
    call = attn.attn_decode_paged_kv8 if N is None else attn.attn_prefill_paged_kv8
    size = (attn.attn_decode_paged_kv8_workspace_size(len(lens), Hq, Hkv, d) if N is None
            else attn.attn_prefill_paged_kv8_workspace_size(len(lens), Hq, Hkv, N, d))
    assert (size == 0) == (N == 300)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(scale=0.3), dict(return_lse=False), dict(workspace=ws)):
        both(fast_only, lambda s: call(*args, stream=s, **kw))
    o, lse = torch.empty_like(args[0]), torch.empty(args[0].shape[:-1], device=DEV)
    got = call(*args, o=o, lse=lse, return_lse=False)
    assert got[0] is o and got[1] is lse


def test_nothing_to_do(fast_only):  # noqa: F811
    d, Hkv = 64, 2
    kv = torch.full((3, Hkv, attn.kv8_record_bytes(d)), 0x5A, dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 3, dtype=torch.int32, device=DEV)
    x = torch.zeros(0, Hkv, d, dtype=BF, device=DEV)
    for long_way in (False, True):
        fast_only.long_way = long_way
        attn.kv8_append_paged(None, x, x, kv, table, none, none)
        assert attn.kv8_read_paged(kv, table, none, none, d)[0].shape == (0, Hkv, d)
        o, lse = attn.attn_decode_paged_kv8(torch.zeros(0, 4, d, dtype=BF, device=DEV), kv, table[:0], none)
        assert o.shape == (0, 4, d) and lse.shape == (0, 4)
        o, lse = attn.attn_prefill_paged_kv8(torch.zeros(1, 4, 0, d, dtype=BF, device=DEV), kv, table, none.new_zeros(1))
        assert o.shape == (1, 4, 0, d) and lse.shape == (1, 4, 0)
    torch.cuda.synchronize()
    assert torch.all(kv == 0x5A) and attn.device_status() == 0


def test_errors_take_the_long_way():
    d = 64
    q, rec, table, lens = on_gpu([40, 3], 4, 2, d, seed=6)
    many = torch.zeros(2, 4, 3, d, dtype=BF, device=DEV)
    for call, x in ((attn.attn_decode_paged_kv8, q), (attn.attn_prefill_paged_kv8, many)):
        with pytest.raises(ValueError, match="q must be torch.bfloat16"):
            call(x.float(), rec, table, lens)
        with pytest.raises(ValueError, match="contiguous"):
            call(x.transpose(0, 1).contiguous().transpose(0, 1), rec, table, lens)
        with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
            call(x, rec, table.cpu(), lens)
        with pytest.raises(ValueError, match="workspace has 16 bytes"):
            call(x, rec, table, lens, workspace=rec.new_empty(16))
        with pytest.raises(attn.AttnError, match=call.__name__ + " failed"):
            call(x[:, :3].contiguous(), rec, table, lens)             # 3 heads over 2
        with pytest.raises(attn.AttnError, match=call.__name__ + " failed"):
            call(x, rec, table, lens, scale=-1.0)
        one, two = call(x, rec, table, lens, scale=1), call(x, rec, table, lens, scale=1.0)   # an integer scale
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    with pytest.raises(ValueError, match="seq_ids must have shape|positions must have shape"):
        attn.kv8_read_paged(rec, table, lens[:1], lens, d)
    x = randn(2, 5, 2, d).to(DEV)
    ids, pos = torch.zeros(5, dtype=torch.int32, device=DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="positions must be torch.int32"):
        attn.kv8_append_paged(None, x, x, rec, table, ids, pos.long())
    with pytest.raises(attn.AttnError, match="kv8_append_paged failed"):
        attn.kv8_append_paged(x, x, x, rec, table, ids, pos, q_out=x)      # the queries' output over the keys


@pytest.mark.parametrize("status", [3, 4])
def test_a_call_whose_launch_failed_is_not_made_again(status):
    fast, lib = _binding._fast(), attn.load_library()
    made, keep = [], []

    def stub(name):
        restype, argtypes = _binding._SIGS[name]
        if restype is ctypes.c_size_t:
            return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
        f = ctypes.CFUNCTYPE(restype, *argtypes)(lambda *a: made.append(name) or status)
        keep.append(f)
        return ctypes.cast(f, ctypes.c_void_p).value

    d = 64
    q, rec, tab, lens = on_gpu([40, 3], 4, 2, d, seed=6)
    table, ids, pos, nb, x, _, _, _ = map_case([0], [5], 4, 2, d, 3)
    table, ids, pos, x = (t.to(DEV) for t in (table, ids, pos, x))
    kv = torch.zeros(nb, 2, attn.kv8_record_bytes(d), dtype=torch.uint8, device=DEV)
    cases = {"kv8_append_paged": lambda: attn.kv8_append_paged(*views(x, 4, 2, d), kv, table, ids, pos),
             "kv8_read_paged": lambda: attn.kv8_read_paged(kv, table, ids, pos, d),
             "attn_decode_paged_kv8": lambda: attn.attn_decode_paged_kv8(q, rec, tab, lens),
             "attn_prefill_paged_kv8": lambda: attn.attn_prefill_paged_kv8(q[:, :, None], rec, tab, lens)}
    for call in cases.values():                              # (sizes that are kept by the binding)
        call()
    try:
        fast.bind8(*(stub(n) for n in _binding._FAST_KV8))
        for name, call in cases.items():
            del made[:]
            with pytest.raises(attn.AttnError, match=name + " failed") as e:
                call()
            assert e.value.status == status and made == [name]
    finally:
        fast.bind8(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _binding._FAST_KV8))
    for call in cases.values():
        call()
    torch.cuda.synchronize()
    assert attn.device_status() == 0


@pytest.mark.parametrize("N", [None, 2, 150])
def test_threads_on_streams_of_their_own(N):
    d = 128
    cases = [on_gpu([500 + 100 * i, 60] * (1 if N != 150 else 8), 4, 2, d, seed=i, N=N) for i in range(4)]
    call = attn.attn_decode_paged_kv8 if N is None else attn.attn_prefill_paged_kv8
    want = [call(*c) for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    o, lse = call(*cases[i])
                    if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                        bad.append(i)
        except Exception as e:                               # (a thread's would be a warning)
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad and attn.device_status() == 0


@pytest.mark.parametrize("name", ["fwd", "decode", "decode8", "passes8", "tiles8"])
def test_the_first_call_of_a_thread(name):
    """A thread that has made no CUDA call has no context bound to it."""
    d = 64
    q, rec, table, lens = on_gpu([40, 3] * 8, 4, 2, d, seed=6)
    one = torch.zeros(1, 2, 40, d, dtype=BF, device=DEV)
    bf = torch.zeros(rec.shape[0], 2, 16, d, dtype=BF, device=DEV)
    few, many = (torch.zeros(16, 4, n, d, dtype=BF, device=DEV) for n in (2, 300))
    assert attn.attn_prefill_paged_kv8_workspace_size(16, 4, 2, 300, d) == 0
    call = dict(fwd=lambda: attn.attn_fwd(one, one, one), decode=lambda: attn.attn_decode_paged(q, bf, bf, table, lens),
                decode8=lambda: attn.attn_decode_paged_kv8(q, rec, table, lens),
                passes8=lambda: attn.attn_prefill_paged_kv8(few, rec, table, lens),
                tiles8=lambda: attn.attn_prefill_paged_kv8(many, rec, table, lens))[name]
    want = call()
    torch.cuda.synchronize()
    got = []

    def work():
        try:
            got.append(call())
        except Exception as e:
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert isinstance(got[0], tuple), got[0]
    assert torch.equal(torch.nan_to_num(got[0][0]), torch.nan_to_num(want[0])) and attn.device_status() == 0


def test_what_a_call_on_a_given_stream_allocates_is_that_streams():
    d, S, Hq = 128, 64, 8
    q, rec, table, lens = on_gpu([40] * S, Hq, 2, d, seed=8)
    want = attn.attn_decode_paged_kv8(q, rec, table, lens)[0]
    wide = attn.attn_prefill_paged_kv8(q[:, :, None], rec, table, lens)[0]
    side = torch.cuda.Stream()
    for name, call, ref in (("decode", lambda: attn.attn_decode_paged_kv8(q, rec, table, lens, stream=side)[0], want),
                            ("prefill", lambda: attn.attn_prefill_paged_kv8(q[:, :, None], rec, table, lens,
                                                                            stream=side)[0], wide)):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = [torch.empty_like(ref) for _ in range(8)]
        torch.cuda._sleep(20_000_000)
        for h in held:
            h.fill_(7.0)
        del held, h
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, ref), name
