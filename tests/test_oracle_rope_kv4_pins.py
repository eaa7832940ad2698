"""Pins of the rotary-position and 4-bit-cache oracles (CPU): complex
multiplication, invariants of a rotation, finite differences, the cell layout
as a permutation, rounding bounds, and a round trip through a record."""

import numpy as np
import pytest
import torch

import oracle


def _freq(rot):
    return (10000.0 ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 64))
    pos = np.array([0, 1, 7, 1000003, -4])
    f = _freq(32)
    y = oracle.rope_rotate(x, pos, f, interleaved=interleaved)
    head = x[..., :32]
    z = head[..., 0::2] + 1j * head[..., 1::2] if interleaved else head[..., :16] + 1j * head[..., 16:]
    z = z * np.exp(1j * pos[:, None] * f.astype(np.float64))
    want = np.stack([z.real, z.imag], -1).reshape(2, 5, 32) if interleaved else np.concatenate([z.real, z.imag], -1)
    np.testing.assert_allclose(y[..., :32], want, rtol=0, atol=1e-9)
    assert np.array_equal(y[..., 32:], x[..., 32:])


def test_rotation_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 64)), rng.standard_normal((1, 64))
    f = _freq(64)

    def dot(a, b):
        return float((oracle.rope_rotate(q, [a], f) * oracle.rope_rotate(k, [b], f)).sum())

    assert abs(dot(12, 5) - dot(1012, 1005)) < 1e-9
    assert abs(np.linalg.norm(oracle.rope_rotate(q, [99], f)) - np.linalg.norm(q)) < 1e-12


def test_axes_select_positions():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 64))
    pos = np.array([[1, 2, 3], [10, 20, 30], [7, 7, 9]])
    axis = [0] * 8 + [1] * 12 + [2] * 12
    f = _freq(64)
    y = oracle.rope_rotate(x, pos, f, pair_axis=axis)
    for p in (0, 7, 8, 19, 20, 31):
        one = oracle.rope_rotate(x, pos[axis[p]], f)
        np.testing.assert_array_equal(y[:, [p, p + 32]], one[:, [p, p + 32]])


def test_inverse_is_the_gradient():
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((2, 32)), rng.standard_normal((2, 32))
    f, pos = _freq(32), np.array([3, 17])
    back = oracle.rope_rotate(g, pos, f, inverse=True)
    eps = 1e-6
    for i in (0, 5, 16, 31):
        d = np.zeros_like(x)
        d[:, i] = eps
        num = ((oracle.rope_rotate(x + d, pos, f) - oracle.rope_rotate(x - d, pos, f)) * g).sum(-1) / (2 * eps)
        np.testing.assert_allclose(back[:, i], num, atol=1e-8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [0, 1])
def test_cells_are_a_permutation(kind, d):
    assert sorted(oracle.kv4_cell(kind, e, d) for e in range(d)) == list(range(d))


@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64)])
def test_quantiser_bounds_and_record_round_trip(d, group):
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((16, d)) * np.exp(rng.standard_normal((16, 1)))).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    x[3, :group] = 2.5                          # a constant group
    x[4] = 0.0
    codes, words = oracle.kv4_quantise(x, group)
    vals = oracle.kv4_values(codes, words, group)
    scale = np.repeat((words >> 16 << 16).astype(np.uint32).view(np.float32).astype(np.float64), group, -1)
    low = np.abs(np.repeat((words << 16).astype(np.uint32).view(np.float32).astype(np.float64), group, -1))
    # Half a step, plus the roundings of min and of 15 scales to bf16 (2^-8 each).
    assert np.all(np.abs(vals - x) <= scale / 2 + 2.0 ** -8 * (low + 15 * scale) + 1e-12)
    assert np.array_equal(vals[3, :group], x[3, :group]) and np.all(vals[4] == 0)
    # torch's bf16 conversion rounds alike
    t = torch.from_numpy(x).unflatten(-1, (-1, group)).amin(-1).to(torch.bfloat16)
    assert np.array_equal(t.view(torch.int16).numpy().astype(np.uint16), (words & 0xFFFF).astype(np.uint16))
    rec = rng.integers(0, 256, (1, 1, oracle.kv4_record_bytes(d, group))).astype(np.uint8)
    other, _ = oracle.kv4_quantise(-x, group)
    for s in range(16):
        oracle.kv4_store(rec[0, 0], 0, s, codes[s], words[s], d, group)
        oracle.kv4_store(rec[0, 0], 1, s, other[s], words[s], d, group)
    k, v = oracle.kv4_unpack(rec, d, group)
    assert np.array_equal(k[0, 0], vals)
    assert np.array_equal(v[0, 0], oracle.kv4_values(other, words, group))


def test_decode_over_a_cache_is_the_softmax_of_its_values():
    rng = np.random.default_rng(5)
    d, group = 64, 32
    cache = rng.integers(0, 256, (3, 2, oracle.kv4_record_bytes(d, group))).astype(np.uint8)
    # parameters: scale 0.25, min -2
    words = np.full((3, 2, 2 * 16 * 2), (0x3E80 << 16) | 0xC000, dtype="<u4")
    cache[..., 16 * d:] = words.view(np.uint8).reshape(3, 2, -1)
    q = rng.standard_normal((1, 4, d))
    o, lse = oracle.decode_paged_kv4(q, cache, np.array([[2, 0]]), [21], 0.125, d, group)
    k, v = oracle.kv4_unpack(cache, d, group)
    for h in range(4):
        kk = np.concatenate([k[2, h // 2], k[0, h // 2, :5]])
        vv = np.concatenate([v[2, h // 2], v[0, h // 2, :5]])
        s = kk @ q[0, h] * 0.125
        p = np.exp(s - s.max())
        np.testing.assert_allclose(o[0, h], p @ vv / p.sum(), atol=1e-12)
        np.testing.assert_allclose(lse[0, h], s.max() + np.log(p.sum()), atol=1e-12)
