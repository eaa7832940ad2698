"""Rotations into views that share a buffer with other views of the call: the
same bytes as into memory of their own, and the rest of the buffer as it was."""

import pytest
import torch

import exact_attention_47_gb300 as attn
import workloads
from test_gpu_rope import map_case, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def parts(x, how, B, N, H, d):
    """q, k and v as [B, H, N, d] views of one buffer."""
    if how == "by head":                           # every head's q, k and v beside each other
        y = x.view(B, N, H, 3, d)
        return [y[..., i, :].transpose(1, 2) for i in range(3)]
    if how == "merged":
        y = x.view(B, N, 3 * H, d)
        return [y[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in range(3)]
    y = x.view(B, 3 * H, N, d)                     # head-major
    return [y[:, i * H:(i + 1) * H] for i in range(3)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("B,N", [(4, 1), (2, 37), (1, 200)])
@pytest.mark.parametrize("how", ["by head", "merged", "head-major"])
def test_in_place_and_into_parts_of_one_buffer(how, B, N, back):
    H, d = 3, 64
    x = randn(31, B, N, 3 * H * d).to(DEV)
    f, pos = workloads.rope_inv_freq(d).to(DEV), torch.arange(N, dtype=torch.int32, device=DEV) + 5
    call = attn.rope_bwd if back else attn.rope_fwd
    q, k, v = parts(x, how, B, N, H, d)
    want_q, want_k = call(q, k, pos, f)
    want_v = v.clone()
    y = torch.zeros_like(x)
    yq, yk, yv = parts(y, how, B, N, H, d)
    call(q, k, pos, f, None, False, yq, yk)        # from one buffer into another
    call(q, k, pos, f, None, False, q, k)          # in place
    torch.cuda.synchronize()
    for a, b, c in ((yq, yk, yv), (q, k, v)):
        assert torch.equal(a, want_q) and torch.equal(b, want_k)
    assert torch.all(yv == 0) and torch.equal(v, want_v)


@pytest.mark.parametrize("group", [None, 32])
def test_append_of_parts_interleaved_by_head(group):
    H, d = 3, 64
    table, ids, pos, nb, _, _, _, _ = map_case([0, 21], [5, 40], H, H, d, 3, padding=1)
    x = randn(33, ids.numel(), 3 * H * d).to(DEV)
    table, ids, pos = (t.to(DEV) for t in (table, ids, pos))
    f = workloads.rope_inv_freq(d).to(DEV)
    y = x.view(-1, H, 3, d)
    q, k, v = (y[:, :, i] for i in range(3))
    outs = []
    for own in (True, False):
        if group is None:
            caches = [torch.zeros(nb, H, 16, d, dtype=BF, device=DEV) for _ in range(2)]
            call, more = attn.rope_append_paged, ()
        else:
            caches = [torch.zeros(nb, H, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)]
            call, more = attn.rope_append_paged_kv4, (group,)
        out = call(q, k, v, *caches, table, ids, pos, *more, f, q_out=q.clone() if own else q)
        outs.append([out.clone()] + caches)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.equal(y[:, :, 1:], randn(33, ids.numel(), 3 * H * d).to(DEV).view(-1, H, 3, d)[:, :, 1:])
