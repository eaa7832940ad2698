"""The bound that attention over an 8-bit cache is held to is of the size of what
the call may use, whatever lies beside it, and a value from beside it breaks it.
CPU."""

import numpy as np
import pytest
import torch

import oracle
from kv8_bounds import compare_live, live_top
from test_gpu_kv8_attention import PREFILLS, case


def answer(c, garbage):
    lens, Hq, Hkv, N, d = c
    q, cache, table, _ = case(lens, Hq, Hkv, d, seed=N, N=N, garbage=garbage)
    ref = oracle.prefill_paged_kv8(q.double().numpy(), cache.numpy(), table.numpy(), lens, d ** -0.5, d)
    return cache.numpy(), table.numpy(), ref


SMALL = [c for c in PREFILLS if sum(c[0]) * c[1] * c[3] < 200000]


@pytest.mark.parametrize("garbage", [0xFF, 0x7E])
@pytest.mark.parametrize("c", SMALL)
def test_the_bound_is_of_the_values_size(c, garbage):
    lens, Hq, Hkv, N, d = c
    cache, table, ref = answer(c, garbage)
    top = live_top(cache, table, lens, d)
    assert np.all(top < 16)
    o = torch.from_numpy(np.nan_to_num(ref[0])).to(torch.bfloat16)
    o[torch.from_numpy(np.isnan(ref[1]))] = float("nan")
    compare_live(o, torch.from_numpy(ref[1]).float(), ref, cache, table, lens, d)


def test_a_value_past_the_end_breaks_it():
    """1 / 16 of a token behind the last one, in one row of one head."""
    lens, Hq, Hkv, N, d = [3, 0, 40, 7], 12, 2, 4, 128
    cache, table, (o, lse) = answer((lens, Hq, Hkv, N, d), 0x7E)
    behind = oracle.kv8_unpack(cache, d)[1][table[2, 40 // 16], 1, 40 % 16]
    assert np.all(behind != 0)
    wrong = o.copy()
    wrong[2, 11, 3] += behind / 16
    args = [torch.from_numpy(x).to(t) for x, t in ((wrong, torch.bfloat16), (lse, torch.float32))]
    with pytest.raises(AssertionError, match="o at"):
        compare_live(*args, (o, lse), cache, table, lens, d)
