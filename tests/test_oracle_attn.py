"""Pins of the attention oracle: worked cases, brute force, invariants (CPU only)."""
import math

import numpy as np
import pytest

from oracle import attn_oracle as ao


def test_rotation_by_hand():
    # two pairs, f = (1, 0.01); position 3 turns (1, 0) of pair 0 to (cos 3, sin 3)
    f, m = ao.rope_freqs(4, base=10000.0)
    assert m == 1.0 and np.allclose(f, [1.0, 0.01], rtol=1e-15)
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 7.0]]])
    half = ao.rotate(x, [3], f, layout="half")[0, 0]
    assert np.allclose(half, [math.cos(3), -2 * math.sin(.03), math.sin(3), 2 * math.cos(.03), 7.0], atol=1e-15)
    inter = ao.rotate(x, [3], f, layout="interleaved")[0, 0]
    assert np.allclose(inter, [math.cos(3), math.sin(3), -2 * math.sin(.03), 2 * math.cos(.03), 7.0], atol=1e-15)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scores_depend_on_distance_alone(layout):
    rng = np.random.default_rng(1)
    f, _ = ao.rope_freqs(32, base=1e4)
    q, k = rng.normal(size=(1, 1, 32)), rng.normal(size=(1, 1, 32))
    dot = [np.sum(ao.rotate(q, [p + 5], f, layout=layout) * ao.rotate(k, [p], f, layout=layout)) for p in (0, 17, 4000)]
    assert np.allclose(dot, dot[0], atol=1e-10)


def test_scaled_frequencies():
    f, _ = ao.rope_freqs(16, base=1e6)
    lin, m = ao.rope_freqs(16, base=1e6, scaling="linear", factor=4)
    assert m == 1.0 and np.allclose(lin, f / 4)
    parts, m = ao.rope_freqs(16, base=1e6, scaling="parts", factor=4, original_len=4096, slow=1, fast=32)
    assert m == pytest.approx(1 + 0.1 * math.log(4))
    turns = 4096 * f / (2 * math.pi)
    assert np.array_equal(parts[turns >= 32], f[turns >= 32])
    assert np.allclose(parts[turns <= 1], f[turns <= 1] / 4)
    assert np.all(parts <= f) and np.all(parts >= f / 4)


def test_e4m3_values_by_hand():
    assert list(ao.e4m3_values([0x00, 0x01, 0x07, 0x08, 0x38, 0x7E, 0xB9])) == [0, 2 ** -9, 7 * 2 ** -9, 2 ** -6, 1, 448, -1.125]


def test_attention_brute_force():
    rng = np.random.default_rng(2)
    n, L, heads, group, D = 3, 5, 4, 2, 6
    q, k, v = rng.normal(size=(n, heads, D)), rng.normal(size=(L, 2, D)), rng.normal(size=(L, 2, D))
    o, a = ao.attend(q, k, v, 0.3, group)
    for i in range(n):
        for h in range(heads):
            w = [math.exp(0.3 * sum(q[i, h, d] * k[j, h // 2, d] for d in range(D))) for j in range(L - n + i + 1)]
            for d in range(D):
                ref = sum(wj * v[j, h // 2, d] for j, wj in enumerate(w)) / sum(w)
                assert abs(o[i, h, d] - ref) < 1e-12
                assert a[i, h, d] >= abs(o[i, h, d]) - 1e-12


def test_rows_without_keys_are_zero():
    q = np.ones((3, 1, 4))
    k = v = np.ones((1, 1, 4))
    o, _ = ao.attend(q, k, v, 1.0, 1)
    assert not o[:2].any() and np.array_equal(o[2, 0], np.ones(4))


def test_one_key_gives_its_value():
    rng = np.random.default_rng(3)
    v = rng.normal(size=(1, 1, 4))
    o, _ = ao.attend(rng.normal(size=(1, 2, 4)), rng.normal(size=(1, 1, 4)), v, 1.0, 2)
    assert np.allclose(o[0, 0], v[0, 0]) and np.allclose(o[0, 1], v[0, 0])
