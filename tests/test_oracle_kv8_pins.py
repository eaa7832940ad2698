"""The 8-bit cache's reference, pinned to torch's own e4m3 conversion, brute
force over the codes, closed forms and invariants; mutants are caught.  CPU."""

import numpy as np
import pytest
import torch

import oracle
import workloads

D = 64


def record(n=1, H=1):
    return np.zeros((n, H, oracle.kv8_record_bytes(D)), np.uint8)


def test_code_values_are_torchs():
    v = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.kv8_code_values(), v, equal_nan=True)


def test_codes_are_the_nearest_and_torchs():
    gen = np.random.default_rng(1)
    x = np.concatenate([gen.standard_normal(20000) * 2.0 ** gen.integers(-12, 9, 20000), [0.0, -0.0, 448, -448, 1e-30, 460]])
    x = np.clip(x, -448, 448)
    c = oracle.kv8_codes(x)
    want = torch.tensor(x, dtype=torch.float64).to(torch.float32)
    exact = want.double().numpy() == x
    assert np.array_equal(c[exact], want.to(torch.float8_e4m3fn).view(torch.uint8).numpy()[exact])
    vals = oracle.kv8_code_values()
    finite = vals[~np.isnan(vals)]
    best = np.abs(x[:500, None] - finite[None]).min(-1)
    assert np.array_equal(np.abs(vals[c[:500]] - x[:500]), best)


def test_half_way_goes_to_the_even_code():
    vals = oracle.kv8_code_values()[:127]
    mid = (vals[1:] + vals[:-1]) / 2
    c = oracle.kv8_codes(mid)
    assert np.all(c % 2 == 0) and np.all(np.abs(c - np.arange(126) - 0.5) == 0.5)
    assert np.array_equal(oracle.kv8_codes(-mid[1:]), c[1:] + 128)


def test_scale_is_the_smallest_power_of_two():
    gen = np.random.default_rng(2)
    for _ in range(300):
        x = gen.standard_normal(5) * 2.0 ** gen.integers(-40, 40)
        s = oracle.kv8_scale(x)
        assert np.abs(x).max() <= 448 * s and np.abs(x).max() > 448 * s / 2
    assert oracle.kv8_scale([448.0]) == 1.0 and oracle.kv8_scale([448.0 * (1 + 1e-15)]) == 2.0
    assert oracle.kv8_scale([0.0]) == 2.0 ** -64 and oracle.kv8_scale([1e38]) == 2.0 ** 64
    assert oracle.kv8_scale([np.nan, np.inf, 448.0]) == 1.0


def test_append_stores_what_is_read_back():
    gen = np.random.default_rng(3)
    k, v = gen.standard_normal((2, 40, 2, D))
    table = np.array([[2, 0, 1]])
    c = oracle.kv8_append(record(3, 2), k, v, table, [0] * 40, range(40), D)
    rk, rv, flags = oracle.kv8_unpack(c, D)
    assert not flags.any()
    for got, x in ((rk, k), (rv, v)):
        rows = np.stack([got[table[0, t // 16], :, t % 16] for t in range(40)])
        top = np.stack([np.abs(x[t // 16 * 16: t // 16 * 16 + 16]).max((0, 2)) for t in range(40)])[..., None]
        assert np.all(np.abs(rows - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * top / 224))
        assert np.array_equal(torch.tensor(rows).to(torch.bfloat16).double().numpy(), rows)
    assert np.all(rk[1, :, 8:] == 0)                # slots not written of a block begun


def test_token_by_token_equals_at_once_where_nothing_is_subnormal():
    """Growth of a scale is exact unless a code becomes subnormal."""
    gen = np.random.default_rng(4)
    x = (1 + gen.random((16, 1, D))) * np.where(gen.random((16, 1, D)) < 0.5, -1, 1) * 2.0 ** np.arange(16)[:, None, None] / 512
    table = np.array([[0]])
    at_once = oracle.kv8_append(record(), x, x, table, [0] * 16, range(16), D)
    step = record()
    for t in range(16):
        oracle.kv8_append(step, x[t: t + 1], x[t: t + 1], table, [0], [t], D)
    small = np.abs(oracle.kv8_unpack(at_once, D)[0]) < 2.0 ** -6 * oracle.kv8_scale(x)
    a, b = oracle.kv8_unpack(at_once, D)[0], oracle.kv8_unpack(step, D)[0]
    assert np.array_equal(a[~small], b[~small]) and small.any()
    assert np.all(np.abs(a - b) <= 2.0 ** -9 * oracle.kv8_scale(x))


def test_what_is_not_finite_is_flagged_and_alone():
    x = np.ones((3, 1, D))
    x[1, 0, 5], x[2, 0, 0] = np.nan, -np.inf
    c = oracle.kv8_append(record(), x, np.ones_like(x), np.array([[0]]), [0] * 3, [0, 1, 2], D)
    k, v, flags = oracle.kv8_unpack(c, D)
    assert flags[0, 0].tolist() == [False, True, True] + [False] * 13
    assert np.isnan(k[0, 0, 1, 5]) and np.isnan(k[0, 0, 2, 0]) and np.isnan(k).sum() == 2 and not np.isnan(v).any()
    assert k[0, 0, 0, 0] == 1.0
    oracle.kv8_append(c, x[:1], x[:1], np.array([[0]]), [0], [1], D)
    assert oracle.kv8_unpack(c, D)[2][0, 0].tolist() == [False, False, True] + [False] * 13


def test_attention_over_it_is_attention():
    Hq, Hkv, N = 4, 2, 5
    table, ids, pos, nb = workloads.token_map([0, 0, 0], [3, 20, 0], seed=5)
    cache = workloads.kv8_cache(nb, Hkv, oracle.kv8_record_bytes(D), D, seed=6).numpy()
    k, v, _ = oracle.kv8_unpack(cache, D)
    q = np.random.default_rng(7).standard_normal((3, Hq, N, D))
    o, lse = oracle.prefill_paged_kv8(q, cache, table.numpy(), [3, 20, 0], 0.1, D)
    for b, L in ((0, 3), (1, 20)):
        keys = np.stack([k[table[b, j // 16], :, j % 16] for j in range(L)], 1)
        vals = np.stack([v[table[b, j // 16], :, j % 16] for j in range(L)], 1)
        for i in range(N):
            n = L - N + i + 1
            if n <= 0:
                assert np.all(o[b, :, i] == 0) and np.all(lse[b, :, i] == -np.inf)
                continue
            ro, rl = oracle.attention(q[b][None, :, i: i + 1], keys[None, :, :n], vals[None, :, :n], 0.1, False)
            assert np.allclose(o[b, :, i], ro[0, :, 0], atol=1e-12) and np.allclose(lse[b, :, i], rl[0, :, 0], atol=1e-12)
    assert np.all(o[2] == 0)
    od, ld = oracle.decode_paged_kv8(q[:, :, -1], cache, table.numpy(), [3, 20, 0], 0.1, D)
    assert np.allclose(od, o[:, :, -1], atol=1e-13) and np.allclose(ld, lse[:, :, -1], atol=1e-13)


@pytest.mark.parametrize("mutant", ["truncate", "scale_up", "no_regrow", "kinds_swapped"])
def test_mutants_are_caught(mutant, monkeypatch):
    """Each of these breaks one of the tests above."""
    import oracle.kv8 as m
    codes, scale = m.kv8_codes, m.kv8_scale
    if mutant == "truncate":
        monkeypatch.setattr(oracle, "kv8_codes", lambda x: np.where(np.abs(m.kv8_code_values()[codes(x)]) > np.abs(x),
                                                                    codes(x) - 1, codes(x)))
        failing = [test_half_way_goes_to_the_even_code]
    elif mutant == "scale_up":
        monkeypatch.setattr(oracle, "kv8_scale", lambda x: 2 * scale(x))
        failing = [test_scale_is_the_smallest_power_of_two]
    elif mutant == "no_regrow":
        monkeypatch.setattr(m, "kv8_scale", lambda x: scale(np.asarray(x)[:1]))
        failing = [test_token_by_token_equals_at_once_where_nothing_is_subnormal, test_append_stores_what_is_read_back]
    else:
        monkeypatch.setattr(oracle, "kv8_append", lambda c, k, v, *a: m.kv8_append(c, v, k, *a))
        failing = [test_append_stores_what_is_read_back]
    with pytest.raises(AssertionError):
        for t in failing:
            t()
