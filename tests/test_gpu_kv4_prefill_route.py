"""A prompt chunk over a 4-bit cache by the calls there are: cached rows read
back, put into a bf16 pool of blocks, and the chunk attending to that; its own
keys and values go into the 4-bit cache as well, which a decode step then
attends to."""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import oracle
import workloads
from parity import assert_attn_close, to64
from test_gpu_kv4 import check_decode
from test_gpu_rope import randn, views

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("d,group,Hq,Hkv,ctx,new", [(128, 32, 12, 2, [45, 0, 300], 70), (64, 64, 8, 8, [16, 129], 33)])
def test_a_chunk_attends_to_a_4_bit_prefix(d, group, Hq, Hkv, ctx, new):
    S, f = len(ctx), workloads.rope_inv_freq(d).to(DEV)
    lens = [n + new + 1 for n in ctx]
    table, ids, pos, nb = workloads.token_map([0] * S, lens, seed=5)
    kv = torch.zeros(nb, Hkv, attn.kv4_record_bytes(d, group), dtype=torch.uint8, device=DEV)
    old = torch.cat([torch.arange(n) < c for n, c in zip(lens, ctx)])
    T, tab = int(old.sum()), table.to(DEV)
    oi, op = ids[old].to(DEV), pos[old].to(DEV)
    x = randn(251, T, (Hq + 2 * Hkv) * d).to(DEV)
    attn.rope_append_paged_kv4(*views(x, Hq, Hkv, d), kv, tab, oi, op, group, inv_freq=f)
    # the prefix into a bf16 pool with a table of its own
    table2, _, _, nb2 = workloads.token_map([0] * S, [n - 1 for n in lens], seed=6)
    tab2 = table2.to(DEV)
    kc, vc = (torch.zeros(nb2, Hkv, 16, d, dtype=BF, device=DEV) for _ in range(2))
    rk, rv = attn.kv4_read_paged(kv, tab, oi, op, d, group)
    attn.rope_append_paged(None, rk, rv, kc, vc, tab2, oi, op)
    before = [to64(c) for c in (kc, vc)]
    # the chunk: rotated to the attention's layout, and appended to the 4-bit cache
    y = randn(252, S * new, (Hq + 2 * Hkv) * d).to(DEV)
    at = torch.cat([torch.arange(c, c + new) for c in ctx]).int().to(DEV)
    seqs = torch.arange(S, dtype=torch.int32, device=DEV)
    q, k, v = (t.view(S, new, -1, d).transpose(1, 2) for t in views(y, Hq, Hkv, d))
    qr, kr = attn.rope_fwd(q, k, at.view(S, new), f)
    vr = v.contiguous()
    ctx_lens = torch.tensor(ctx, dtype=torch.int32)
    scale = d ** -0.5
    o, lse = attn.attn_prefill_paged(qr, kr, vr, kc, vc, tab2, ctx_lens.to(DEV), scale=scale)
    attn.rope_append_paged_kv4(*views(y, Hq, Hkv, d), kv, tab, seqs.repeat_interleave(new), at, group, inv_freq=f)
    torch.cuda.synchronize()
    assert attn.device_status() == 0
    ro, rl, ck, cv = oracle.prefill_paged(to64(qr), to64(kr), to64(vr), *before, table2.numpy(), ctx_lens.numpy(), scale, 16)
    assert_attn_close(o, lse, ro, rl, what="chunk over a read-back prefix")
    assert np.array_equal(to64(kc), ck) and np.array_equal(to64(vc), cv)
    # the next token
    z = views(randn(253, S, (Hq + 2 * Hkv) * d).to(DEV), Hq, Hkv, d)
    last = ctx_lens + new
    q4 = attn.rope_append_paged_kv4(*z, kv, tab, seqs, last.to(DEV), group, inv_freq=f)
    o4, l4 = attn.attn_decode_paged_kv4(q4, kv, tab, (last + 1).to(DEV), group)
    torch.cuda.synchronize()
    check_decode(o4, l4, q4.cpu(), kv.cpu(), table, last + 1, scale, d, group, "after the chunk")
