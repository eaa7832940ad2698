"""attn_set_decode_max_ctas bounds the decode over a 4-bit cache too."""

import pytest
import torch

import exact_attention_47_gb300 as attn
from test_gpu_kv4 import DEV, check_decode, decode_case, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctas", [1, 2, 7, 64])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", [([9000, 0, 33, 700], 6, 1, 128, 64), ([300] * 40, 32, 2, 64, 32),
                                                 ([17, 5000, 1], 8, 2, 128, 32), ([2] * 1500, 2, 2, 64, 64)])
def test_results_and_workspace_of_few_ctas(lens, Hq, Hkv, d, group, ctas):
    """Results against the oracle; of the workspace (counters of 256 CTAs, then
    their partial results in order) only what these CTAs have is written."""
    case = decode_case(lens, Hq, Hkv, d, group, seed=231)
    G = Hq // Hkv
    ws = torch.full((attn.attn_decode_paged_kv4_workspace_size(len(lens), Hq, Hkv, d),), 0xA5, dtype=torch.uint8, device=DEV)
    try:
        attn.set_decode_max_ctas(ctas)
        o, lse = run(*case, group, 0.09, workspace=ws)
        again, _ = run(*case, group, 0.09, workspace=ws)
    finally:
        attn.set_decode_max_ctas(0)
    check_decode(o, lse, *case, 0.09, d, group, "%d CTAs" % ctas)
    assert torch.equal(o, again)
    counters, rest = ws[:256 * 8].view(256, 8), ws[256 * 8:]
    parts = rest[:2 * 256 * G * d * 4].view(2 * 256, G * d * 4)
    sums = rest[2 * 256 * G * d * 4:].view(2 * 256, G * 8)
    for t, n in ((counters, ctas), (parts, 2 * ctas), (sums, 2 * ctas)):
        assert torch.all(t[n:] == 0xA5)


def test_the_bound_is_seen_in_the_workspace():
    """Without it a run of 9000 tokens is split over many CTAs."""
    case = decode_case([9000], 6, 1, 128, 64, seed=231)
    ws = torch.full((attn.attn_decode_paged_kv4_workspace_size(1, 6, 1, 128),), 0xA5, dtype=torch.uint8, device=DEV)
    run(*case, 64, 0.09, workspace=ws)
    assert not torch.all(ws[256 * 8 + 4 * 6 * 128 * 4:][:2 * 6 * 128 * 4] == 0xA5)


def test_many_queries_with_one_cta():
    """64 MB of queries: what one CTA asks for ahead is bounded."""
    S, Hq, Hkv, d, group = 4096, 64, 4, 128, 64
    case = decode_case([1, 2, 0, 3] * (S // 4), Hq, Hkv, d, group, seed=239)
    try:
        attn.set_decode_max_ctas(1)
        o, lse = run(*case, group, 0.09)
    finally:
        attn.set_decode_max_ctas(0)
    want, want_lse = run(*case, group, 0.09)
    assert torch.equal(lse, want_lse) and torch.equal(o, want)
