"""Attention over the 8-bit cache where it can go wrong at the edges of what it
accepts, against the fp64 oracle, held to the values that the call may use."""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import oracle
from kv8_bounds import compare_live
from test_gpu_kv8_attention import DECODES, PREFILLS, case, decode, prefill, ways

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("lens,Hq,Hkv,d", DECODES)
def test_decode_beside_large_garbage(lens, Hq, Hkv, d):
    """Slots past the ends and unused blocks hold the largest numbers."""
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=len(lens) + Hq, garbage=0x7E)
    o, lse = decode(q, cache, table, sl)
    ref = oracle.decode_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d)
    assert attn.device_status() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,N,d", PREFILLS)
def test_prefill_beside_large_garbage(lens, Hq, Hkv, N, d):
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N, garbage=0x7E)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)
    assert attn.device_status() == 0


def flag(cache, table, b, p, h, kind, d):
    """A NaN in the key (kind 0) or value of head h of sequence b's token p."""
    rec = cache[table[b, p // 16].long(), h]
    rec[(16 * kind + p % 16) * d + p % d] = 0x7F
    word = rec[32 * d + 8: 32 * d + 12].view(torch.int32)
    word |= 1 << (16 * kind + p % 16) if 16 * kind + p % 16 < 31 else -2 ** 31


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,N", [(2, 2, 300), (3, 1, 200), (2, 1, 520)])
def test_flagged_tokens_where_the_query_tiles_end_apart(Hq, Hkv, N, d):
    """The two query tiles of 128 rows that a CTA works on see different numbers of
    key tiles.  Flags in the last key tile that the first sees, in its last key, just
    behind, in the second's last one, and in none."""
    first = 100 + 127                                # last key of the first query tile: of key tile 1 of 128
    flagged = [200, first, first + 1, 255, 256, 99 + min(N, 256), None, 100 + N - 1, 0]
    lens = [100 + N] * len(flagged)
    q, cache, table, sl = case(lens, Hq, Hkv, d, seed=N, N=N)
    for b, p in enumerate(flagged):
        if p is not None:
            flag(cache, table, b, p, b % Hkv, b % 2, d)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    for times in ways(len(lens), Hq, Hkv, N, d):
        o, lse = prefill([x.to(DEV) for x in (q, cache, table, sl)], times)
        compare_live(o, lse, ref, cache.numpy(), table.numpy(), lens, d, what="%d times" % times)
    assert attn.device_status() == 0
