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
from test_gpu_rope import randn

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
