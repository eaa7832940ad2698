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
