"""Decode over a 4-bit cache whose values are poisoned or of very different
size: a group of V is its own columns' business alone.

Bounds are those of test_gpu_kv4, with a group's own largest value in place of
the pool's: a numerator's product with a V scale is rounded to 11 bits, so a
group's columns are off by at most 2^-11 of 15 scales, under 2^-10 of its
largest |V| (products under 2^-19 of a numerator of 1 with the group's largest
scale add 2^-30 of that each), before the bf16 rounding of O."""

import numpy as np
import pytest
import torch

import oracle
from parity import to64
from test_gpu_kv4 import decode_case, run

pytestmark = pytest.mark.gpu


def v_words(rec, d, group):
    """The parameter words of V, [num_blocks, Hkv, slot, group], as a view."""
    n = 16 * (d // group)
    return rec[..., 16 * d:].view(torch.int32)[..., n:].unflatten(-1, (16, d // group))


def check_groups(o, lse, q, rec, table, lens, scale, d, group, skip=None):
    """O, every group within its own bound, and LSE against the oracle.
    ``skip`` [S, Hq, d]: elements left out."""
    ro, rl = oracle.decode_paged_kv4(to64(q), rec.numpy(), table.numpy(), lens.numpy(), scale, d, group)
    _, v = oracle.kv4_unpack(rec.numpy(), d, group)
    S, Hq = q.shape[:2]
    Hkv = rec.shape[1]
    lim = np.zeros_like(ro)
    for b in range(S):
        at = np.arange(int(lens[b]))
        if not len(at):
            continue
        mine = np.abs(v[table.numpy()[b][at // 16], :, at % 16])                 # [tokens, Hkv, d]
        top = mine.reshape(len(at), Hkv, d // group, group).max((0, 3))
        lim[b] = np.repeat(np.repeat(top, group, -1), Hq // Hkv, 0) * 2.0 ** -10
    lim = lim + 2.0 ** -8 * np.abs(ro)
    err = np.abs(to64(o) - ro)
    ok = err <= lim
    if skip is not None:
        ok |= skip
    assert ok.all(), "O off by %.3g of its bound at %s" % (
        np.nanmax(np.where(ok, 0, err / np.maximum(lim, 1e-300))), np.argwhere(~ok)[0])
    fin = np.isfinite(rl)
    assert np.array_equal(to64(lse)[~fin], rl[~fin])
    assert np.all(np.abs(to64(lse)[fin] - rl[fin]) <= 2.0 ** -16 * np.maximum(1.0, np.abs(rl[fin])))


# Few warps to a run, a run over several CTAs, many runs a CTA.
SHAPES = [([200, 40], 8, 2, 128, 32), ([9000, 0, 33], 6, 1, 128, 64), ([4100, 100], 32, 2, 64, 32),
          ([700] * 90, 4, 2, 64, 64), ([3000, 2900], 16, 1, 128, 32)]


@pytest.mark.parametrize("word", [0x7FC07FC0, 0x7F803F80])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", SHAPES)
def test_a_poisoned_value_group_shows_in_its_columns_only(lens, Hq, Hkv, d, group, word):
    """A group that stands for NaN (or has an infinite scale), at the first, a
    middle or the last token of a sequence."""
    scale, h, G = 0.09, Hkv - 1, Hq // Hkv
    for t in (0, lens[0] // 3, lens[0] - 1):
        q, rec, table, n = decode_case(lens, Hq, Hkv, d, group, seed=211)
        g = (d // group) // 2
        bad = rec.clone()
        v_words(bad, d, group)[int(table[0, t // 16]), h, t % 16, g] = word
        o, lse = run(q, bad, table, n, group, scale)
        skip = np.zeros(tuple(o.shape), bool)
        skip[0, h * G:(h + 1) * G, g * group:(g + 1) * group] = True
        check_groups(o, lse, q, rec, table, n, scale, d, group, skip)
        assert not np.isfinite(to64(o)[skip]).any()


def test_every_value_group_poisoned_leaves_the_lse():
    q, rec, table, n = decode_case([300, 50], 8, 2, 128, 32, seed=213)
    bad = rec.clone()
    v_words(bad, 128, 32)[...] = 0x7FC07FC0
    o, lse = run(q, bad, table, n, 32, 0.09)
    check_groups(o, lse, q, rec, table, n, 0.09, 128, 32, np.ones(tuple(o.shape), bool))
    assert torch.isnan(o.float()).all()


def scaled_words(rec, d, group, powers):
    """The cache with V groups times 2^powers ([group], or anything that
    broadcasts against [num_blocks, Hkv, slot, group])."""
    rec = rec.clone()
    w = v_words(rec, d, group)
    pair = w.contiguous().view(torch.bfloat16).unflatten(-1, (d // group, 2)).double()
    pair = (pair * 2.0 ** torch.as_tensor(powers, dtype=torch.float64)[..., None]).to(torch.bfloat16)
    w.copy_(pair.flatten(-2).contiguous().view(torch.int32))
    return rec


@pytest.mark.parametrize("powers", [(0, -28), (-24, 20), (100, 0), (-60, -100), (40, -40)])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", SHAPES)
def test_value_groups_of_very_different_size(lens, Hq, Hkv, d, group, powers):
    q, rec, table, n = decode_case(lens, Hq, Hkv, d, group, seed=221)
    groups = d // group
    rec = scaled_words(rec, d, group, (powers * groups)[:groups])
    o, lse = run(q, rec, table, n, group, 0.09)
    check_groups(o, lse, q, rec, table, n, 0.09, d, group)


@pytest.mark.parametrize("step", [12, 40])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", SHAPES)
def test_value_sizes_that_change_along_a_run(lens, Hq, Hkv, d, group, step):
    """Values grow along the run in even groups and shrink in odd ones, and
    the sharp softmax of large scores looks at one place or another."""
    q, rec, table, n = decode_case(lens, Hq, Hkv, d, group, seed=223)
    powers = torch.zeros(rec.shape[0], Hkv, 16, d // group)
    for b, L in enumerate(lens):
        for j in range(0, L, 16):
            powers[int(table[b, j // 16])] = ((4 * j // L - 2) * step / 2 * (-1.0) ** torch.arange(d // group)).round()
    rec = scaled_words(rec, d, group, powers)
    for scale in (0.02, 2.0):
        o, lse = run(q, rec, table, n, group, scale)
        check_groups(o, lse, q, rec, table, n, scale, d, group)


@pytest.mark.parametrize("low", [1e30, -3e25, 1e-30])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", SHAPES)
def test_constant_value_groups_of_any_size(lens, Hq, Hkv, d, group, low):
    """Every V group is constant (scale 0, as the append writes it): O is a
    mean of what they hold."""
    q, rec, table, n = decode_case(lens, Hq, Hkv, d, group, seed=227)
    w = v_words(rec, d, group)
    mins = (low * (1 + torch.rand(w.shape, generator=torch.Generator().manual_seed(1)))).to(torch.bfloat16)
    w.copy_(mins.view(torch.int16).int() & 0xFFFF)
    o, lse = run(q, rec, table, n, group, 0.09)
    check_groups(o, lse, q, rec, table, n, 0.09, d, group)


@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e-10])
def test_queries_of_zero_and_tiny_scales_weigh_all_tokens_alike(scale):
    q, rec, table, n = decode_case([5, 300, 17, 16], 12, 2, 128, 32, seed=241)
    q[:, ::3] = 0
    q[:, 1::3] *= 2.0 ** -100
    o, lse = run(q, rec, table, n, 32, scale)
    check_groups(o, lse, q, rec, table, n, scale, 128, 32)


def test_one_sequence_of_131072_tokens():
    q, rec, table, n = decode_case([131072, 100000], 8, 1, 128, 64, seed=243)
    o, lse = run(q, rec, table, n, 64, 0.09)
    check_groups(o, lse, q, rec, table, n, 0.09, 128, 64)


@pytest.mark.parametrize("quiet", [0.0, 2.0 ** -126, 2.0 ** -110])
@pytest.mark.parametrize("lens,Hq,Hkv,d,group", SHAPES)
def test_scales_of_next_to_nothing_before_ordinary_ones(lens, Hq, Hkv, d, group, quiet):
    """Tokens whose V groups are constant (or hardly vary) come first, or lie
    between others."""
    q, rec, table, n = decode_case(lens, Hq, Hkv, d, group, seed=233)
    low = int(torch.tensor(quiet).to(torch.bfloat16).view(torch.int16)) << 16
    for part in (lambda j, L: j < L // 2, lambda j, L: j // 64 % 2 == 0):
        mine = rec.clone()
        w = v_words(mine, d, group)
        for b, L in enumerate(lens):
            for j in range(L):
                if part(j, L):
                    at = w[int(table[b, j // 16]), :, j % 16]
                    at.copy_((at & 0xFFFF) | low)
        o, lse = run(q, mine, table, n, group, 0.09)
        check_groups(o, lse, q, mine, table, n, 0.09, d, group)
