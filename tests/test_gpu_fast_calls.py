"""Both ways of making a rotary, append or 4-bit-cache call give the same
bytes: the usual case through csrc/fast_calls.cpp, and the Python one.  Errors
are the Python way's."""

import threading

import pytest
import torch

import exact_attention_47_gb300 as attn
import workloads
from exact_attention_47_gb300 import _binding
from test_gpu_kv4 import decode_case
from test_gpu_rope import map_case, randn, views

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


class Nothing:
    """Stands in for the module of the fast calls: nothing is the usual case."""

    def __getattr__(self, name):
        return lambda *args: None


@pytest.fixture
def fast_only(monkeypatch):
    """Fails where a call takes the Python way, unless `long_way` is set: then
    it has to."""
    real_call, real_fast = _binding._call, _binding._fast

    def call(func, device, *args):
        assert call.long_way, "%s took the long way" % func
        return real_call(func, device, *args)

    call.long_way = False
    monkeypatch.setattr(_binding, "_call", call)
    monkeypatch.setattr(_binding, "_fast", lambda: Nothing() if call.long_way else real_fast())
    return call


def both(flag, f, *caches):
    """f() by both ways and, the fast one, on a stream given, each on its own
    copy of the caches."""
    got = []
    for long_way, stream in ((False, None), (True, None), (False, torch.cuda.Stream()), (True, torch.cuda.Stream())):
        flag.long_way = long_way
        mine = [c.clone() for c in caches]
        torch.cuda.synchronize()
        out = f(stream, *mine)
        torch.cuda.synchronize()
        got.append([x for x in (out if isinstance(out, tuple) else (out,)) if x is not None] + mine)
    flag.long_way = False
    assert attn.device_status() == 0
    for other in got[1:]:
        assert len(got[0]) == len(other)
        for a, b in zip(got[0], other):
            assert a.shape == b.shape and a.dtype == b.dtype and a.stride() == b.stride()
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    return got[0]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("axis", [None, list, tuple, bytes])
def test_rope(fast_only, axis, back):
    B, N, d = 2, 37, 64
    x = randn(1, B, N, 6 * d).to(DEV)
    q = x[..., :4 * d].view(B, N, 4, d).transpose(1, 2)
    k = x[..., 4 * d:].view(B, N, 2, d).transpose(1, 2)
    f = workloads.rope_inv_freq(d).to(DEV)
    pos = torch.arange(3 * B * N, dtype=torch.int32, device=DEV).view(3, B, N)
    call = attn.rope_bwd if back else attn.rope_fwd
    pairs = None if axis is None else axis(p % 3 for p in range(d // 2))
    for p in ((pos, pos[:, 0]) if pairs else (pos[0], pos[0, 0])):
        both(fast_only, lambda s: call(q, k, p, f, pairs, stream=s))
        both(fast_only, lambda s: call(q, None, p, f, pairs, True, stream=s))
    out = [torch.empty(B, N, 6, d, dtype=BF, device=DEV)[:, :, i:j].transpose(1, 2) for i, j in ((0, 4), (4, 6))]
    got = call(q, k, p, f, pairs, False, *out)
    assert got[0] is out[0] and got[1] is out[1]


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("queries", [False, True])
def test_append_read(fast_only, group, queries):
    Hq, Hkv, d = 6, 2, 128
    table, ids, pos, nb, x, q, k, v = map_case([0, 21], [5, 40], Hq, Hkv, d, 3, padding=1)
    q, k, v = views(x.to(DEV), Hq, Hkv, d)
    table, ids, pos = (t.to(DEV) for t in (table, ids, pos))
    f = workloads.rope_inv_freq(d).to(DEV)
    axis = [p % 2 for p in range(d // 2)]
    q = q if queries else None
    out = torch.zeros(x.shape[0], Hq, d, dtype=BF, device=DEV) if queries else None   # padding rows stay zero
    for rot in (dict(), dict(inv_freq=f, rope_positions=pos), dict(
            inv_freq=f, rope_positions=torch.stack([pos, pos + 3]), pair_axis=axis, interleaved=True)):
        rot["q_out"] = out
        if group:
            kv = workloads.kv4_cache(nb, Hkv, attn.kv4_record_bytes(d, group), d, group, seed=2).to(DEV)
            kv = both(fast_only, lambda s, c: attn.rope_append_paged_kv4(q, k, v, c, table, ids, pos, group, stream=s, **rot),
                      kv)[-1]
            T = 45
            both(fast_only, lambda s: attn.kv4_read_paged(kv, table, ids[:T], pos[:T], d, group, stream=s))
            mine = [torch.empty(T, Hkv, d, dtype=BF, device=DEV) for _ in range(2)]
            assert attn.kv4_read_paged(kv, table, ids[:T], pos[:T], d, group, *mine)[0] is mine[0]
        else:
            cache = torch.zeros(nb, Hkv, 16, d, dtype=BF, device=DEV)
            both(fast_only, lambda s, a, b: attn.rope_append_paged(q, k, v, a, b, table, ids, pos, stream=s, **rot),
                 cache, cache)


@pytest.mark.parametrize("d,group", [(64, 32), (128, 64)])
def test_decode(fast_only, d, group):
    case = decode_case([1, 0, 300, 77], 8, 2, d, group, seed=5)
    q, rec, table, lens = (t.to(DEV) for t in case[:4])
    ws = torch.zeros(attn.attn_decode_paged_kv4_workspace_size(4, 8, 2, d), dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(scale=0.3), dict(return_lse=False), dict(workspace=ws)):
        both(fast_only, lambda s: attn.attn_decode_paged_kv4(q, rec, table, lens, group, stream=s, **kw))
    o, lse = torch.empty_like(q), torch.empty(4, 8, device=DEV)
    got = attn.attn_decode_paged_kv4(q, rec, table, lens, group, o=o, lse=lse, return_lse=False)
    assert got[0] is o and got[1] is lse


def test_errors_and_unusual_calls_take_the_long_way():
    d, group = 64, 32
    q, rec, table, lens = (t.to(DEV) for t in decode_case([40, 3], 4, 2, d, group, seed=6)[:4])
    with pytest.raises(ValueError, match="q must be torch.bfloat16"):
        attn.attn_decode_paged_kv4(q.float(), rec, table, lens, group)
    with pytest.raises(ValueError, match="block_table must be a CUDA tensor"):
        attn.attn_decode_paged_kv4(q, rec, table.cpu(), lens, group)
    with pytest.raises(ValueError, match="workspace has 16 bytes"):
        attn.attn_decode_paged_kv4(q, rec, table, lens, group, workspace=rec.new_empty(16))
    with pytest.raises(attn.AttnError, match="attn_decode_paged_kv4 failed"):
        attn.attn_decode_paged_kv4(q[:, :3].contiguous(), rec, table, lens, group)   # 3 heads over 2
    with pytest.raises(ValueError, match="seq_ids must have shape|positions must have shape"):
        attn.kv4_read_paged(rec, table, lens[:1], lens, d, group)
    x = randn(2, 1, 4, 5, d).to(DEV)
    f, pos = workloads.rope_inv_freq(d).to(DEV), torch.arange(5, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="positions must be torch.int32"):
        attn.rope_fwd(x, None, pos.long(), f)
    with pytest.raises(attn.AttnError, match="rope_fwd failed"):
        attn.rope_fwd(x, None, pos, f, pair_axis=None, q_out=x[:, :1].expand(1, 4, 5, d))   # overlapping rows
    one = attn.attn_decode_paged_kv4(q, rec, table, lens, group, scale=1)          # an integer scale
    two = attn.attn_decode_paged_kv4(q, rec, table, lens, group, scale=1.0)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_threads_on_streams_of_their_own():
    d, group = 128, 32
    cases = [tuple(t.to(DEV) for t in decode_case([500 + 100 * i, 60], 4, 2, d, group, seed=i)[:4]) for i in range(4)]
    want = [attn.attn_decode_paged_kv4(q, rec, table, lens, group) for q, rec, table, lens in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        q, rec, table, lens = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                o, lse = attn.attn_decode_paged_kv4(q, rec, table, lens, group)
                if not (torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad and attn.device_status() == 0


def test_what_a_call_on_a_given_stream_allocates_is_that_streams():
    """Memory freed on the current stream, where writes to it are still to
    come, is not handed to a call on another stream."""
    d, group, S, Hq = 128, 32, 64, 8
    q, rec, table, lens = (t.to(DEV) for t in decode_case([40] * S, Hq, 2, d, group, seed=8)[:4])
    want = attn.attn_decode_paged_kv4(q, rec, table, lens, group)[0]
    x = randn(5, 1, Hq, S, d).to(DEV)
    f, pos = workloads.rope_inv_freq(d).to(DEV), torch.arange(S, dtype=torch.int32, device=DEV)
    turned = attn.rope_fwd(x, None, pos, f)[0]
    side = torch.cuda.Stream()
    for name, call, ref in (("decode", lambda: attn.attn_decode_paged_kv4(q, rec, table, lens, group, stream=side)[0], want),
                            ("rope", lambda: attn.rope_fwd(x, None, pos, f, stream=side)[0], turned)):
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


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        device = torch.device("cuda", 1)

    x = randn(5, 1, 2, 8, 64).to(DEV)
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        attn.rope_fwd(x, None, torch.arange(8, dtype=torch.int32, device=DEV), workloads.rope_inv_freq(64).to(DEV),
                      stream=Elsewhere())
