"""A launch that the CUDA runtime refuses is reported by its own call, and by
no other.

The refused launch is one into a stream whose capture has been invalidated (by
waiting for the stream while it is captured): an error of the host alone, after
which the stream is as it was."""

import contextlib
import ctypes

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


@contextlib.contextmanager
def invalid_capture():
    """A stream in which every launch is refused; afterwards an ordinary one."""
    cudart = ctypes.CDLL("libcudart.so.13")
    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    torch.cuda.synchronize()
    assert cudart.cudaStreamBeginCapture(handle, 2) == 0                        # relaxed: this stream only
    assert cudart.cudaStreamSynchronize(handle) == 900                          # not permitted: invalidates the capture
    try:
        yield stream
    finally:
        assert cudart.cudaStreamEndCapture(handle, ctypes.byref(graph)) == 901  # invalidated
        cudart.cudaGetLastError()                                               # torch's runtime keeps none of it
        stream.synchronize()


def fail_once():
    x = randn(1, 1, 2, 40, 64).to(DEV)
    f, pos = workloads.rope_inv_freq(64).to(DEV), torch.arange(40, dtype=torch.int32, device=DEV)
    out = torch.zeros_like(x)
    torch.cuda.synchronize()
    with invalid_capture() as stream:
        with pytest.raises(attn.AttnError, match="rope_fwd launch failed"):
            attn.rope_fwd(x, None, pos, f, q_out=out, stream=stream)
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_an_in_place_rotation_after_a_refused_launch_turns_once():
    x = randn(2, 2, 3, 50, 128).to(DEV)
    f, pos = workloads.rope_inv_freq(128).to(DEV), torch.arange(50, dtype=torch.int32, device=DEV) + 3
    want, _ = attn.rope_fwd(x, None, pos, f)
    fail_once()
    got, _ = attn.rope_fwd(x, None, pos, f, q_out=x)
    assert got is x and torch.equal(x, want)


def calls():
    B, H, N, d = 1, 2, 40, 64
    q, k, v = (randn(s, B, H, N, d).to(DEV) for s in (3, 4, 5))
    kc, vc = (torch.zeros(3, H, 16, d, dtype=BF, device=DEV) for _ in range(2))
    table = torch.arange(3, dtype=torch.int32, device=DEV)[None]
    ctx, lens = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((1,), 40, dtype=torch.int32, device=DEV)
    x, w = randn(6, 32, 64).to(DEV), torch.ones(64, dtype=BF, device=DEV)
    return dict(
        fwd=lambda: attn.attn_fwd(q, k, v), prefill_paged=lambda: attn.attn_prefill_paged(q, k, v, kc, vc, table, ctx),
        decode=lambda: attn.attn_decode_paged(q[:, :, 0].contiguous(), kc, vc, table, lens),
        add_rmsnorm=lambda: attn.fused_add_rmsnorm(x, x.clone(), w),
        exp2=lambda: attn.selftest_exp2_poly(torch.zeros(8, device=DEV)))


@pytest.mark.parametrize("name", ["fwd", "prefill_paged", "decode", "add_rmsnorm", "exp2"])
def test_other_calls_do_not_report_it(name):
    call = calls()[name]
    call()
    fail_once()
    call()
    torch.cuda.synchronize()
    assert attn.device_status() == 0


@pytest.mark.parametrize("status", [3, 4])
def test_a_call_whose_launch_failed_is_not_made_again(status):
    """The entry points that the fast calls pass on to, replaced by ones that
    count: one call each, and its status raised.  (What is refused before a
    launch goes to the Python way, and is raised there.)"""
    fast, lib = _binding._fast(), attn.load_library()
    made = []
    keep = []

    def stub(name):
        restype, argtypes = _binding._SIGS[name]
        if restype is ctypes.c_size_t:
            return ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
        f = ctypes.CFUNCTYPE(restype, *argtypes)(lambda *a: made.append(name) or status)
        keep.append(f)
        return ctypes.cast(f, ctypes.c_void_p).value

    d, group = 64, 32
    q, rec, tab, lens = (t.to(DEV) for t in decode_case([40, 3], 4, 2, d, group, seed=6)[:4])
    table, ids, pos, nb, x, _, _, _ = map_case([0], [5], 4, 2, d, 3)
    table, ids, pos, x = (t.to(DEV) for t in (table, ids, pos, x))
    kv = torch.zeros(nb, 2, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
    kc, vc = (torch.zeros(nb, 2, 16, d, dtype=BF, device=DEV) for _ in range(2))
    f = workloads.rope_inv_freq(d).to(DEV)
    y = randn(7, 1, 2, 9, d).to(DEV)
    at = torch.arange(9, dtype=torch.int32, device=DEV)
    attn.attn_decode_paged_kv4(q, rec, tab, lens, group)     # (sizes that are kept by the binding)
    cases = {"rope_fwd": lambda: attn.rope_fwd(y, None, at, f, q_out=y),
             "rope_bwd": lambda: attn.rope_bwd(y, None, at, f, dq=y),
             "rope_append_paged": lambda: attn.rope_append_paged(*views(x, 4, 2, d), kc, vc, table, ids, pos, f),
             "rope_append_paged_kv4": lambda: attn.rope_append_paged_kv4(*views(x, 4, 2, d), kv, table, ids, pos, group, f),
             "kv4_read_paged": lambda: attn.kv4_read_paged(kv, table, ids, pos, d, group),
             "attn_decode_paged_kv4": lambda: attn.attn_decode_paged_kv4(q, rec, tab, lens, group)}
    before = y.clone()
    try:
        fast.bind(*(stub(n) for n in _binding._FAST))
        for name, call in cases.items():
            del made[:]
            with pytest.raises(attn.AttnError, match=name + " failed") as e:
                call()
            assert e.value.status == status and made == [name]
    finally:
        fast.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _binding._FAST))
    torch.cuda.synchronize()
    assert torch.equal(y, before)
