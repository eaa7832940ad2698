"""Appends to the 8-bit cache whose rows leave positions out: all rows of a block
share its scales and its fresh start, whatever lies between their slots.  The
records are the oracle's byte for byte (no rotation: the quantiser's steps are exact
products with powers of two and one rounding)."""

import numpy as np
import pytest
import torch

import exact_attention_47_gb300 as attn
import workloads
from test_gpu_kv8 import append_both
from test_gpu_rope import randn

pytestmark = pytest.mark.gpu


def rows(S, span, keep, seed, most_ctx=40):
    """Table, seq_ids, positions of a part of `span` positions of each sequence, from
    any slot on."""
    gen = np.random.default_rng(seed)
    picks = []
    for b in range(S):
        ctx = int(gen.integers(0, most_ctx))
        at = ctx + np.flatnonzero(gen.random(span) < keep)
        picks.append(at if len(at) else np.array([ctx]))
    width = -(-(most_ctx + span) // 16)
    table = torch.from_numpy(gen.permutation(S * width).astype(np.int32).reshape(S, width))
    ids = torch.from_numpy(np.repeat(np.arange(S), [len(p) for p in picks]).astype(np.int32))
    return table, ids, torch.from_numpy(np.concatenate(picks).astype(np.int32)), S * width


@pytest.mark.parametrize("S,span,keep,Hkv,d", [(1, 16, 0.5, 1, 64), (3, 40, 0.5, 2, 128), (40, 30, 0.6, 3, 64),
                                               (4, 2000, 0.9, 2, 128), (700, 25, 0.3, 1, 128), (3, 3000, 0.1, 5, 64)])
def test_rows_that_leave_positions_out(S, span, keep, Hkv, d):
    table, ids, pos, nb = rows(S, span, keep, seed=S + span)
    T = len(pos)
    gen = torch.Generator().manual_seed(T)
    size = torch.exp2(torch.randint(-6, 7, (T, Hkv, 1), generator=gen).float()).to(torch.bfloat16)
    k, v = randn(T, T, Hkv, d) * size, randn(T + 1, T, Hkv, d) * size.flip(0)
    k[T // 2, 0, 3] = float("inf")
    cache = workloads.kv8_cache(nb, Hkv, attn.kv8_record_bytes(d), d, seed=2)
    got, want = append_both(cache, k, v, table, ids, pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0


@pytest.mark.parametrize("slots", [[0, 15], [0, 2, 4], [1, 3], [5, 14, 15], [0], [15], list(range(0, 16, 3))])
def test_two_blocks_with_the_same_slots(slots):
    """The last slot of one block is followed by the first of the next one's."""
    d, Hkv = 64, 2
    pos = torch.tensor(slots + [16 + s for s in slots], dtype=torch.int32)
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    x = randn(7, len(pos), Hkv, d)
    x[-1] *= 512
    cache = workloads.kv8_cache(3, Hkv, attn.kv8_record_bytes(d), d, seed=3)
    got, want = append_both(cache, x, x.flip(0), table, torch.zeros_like(pos), pos, d)
    assert np.array_equal(got, want) and attn.device_status() == 0
