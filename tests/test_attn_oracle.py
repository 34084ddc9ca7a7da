"""Pins of the attention oracle: rotations that preserve what a rotation has
to preserve, frequencies by hand, paging by hand, attention by hand."""
import math

import numpy as np
import pytest

from oracle import attn_oracle as A


def test_frequencies_by_hand():
    f = A.frequencies(16, theta=10000.0)
    assert f[0] == 1.0 and abs(f[4] - 0.01) < 1e-17
    assert np.array_equal(A.frequencies(16, scaling="linear", factor=4.0), f / 4.0)
    # turns over 8192 positions: f = 1 makes 1303.8 (kept), the slowest 8192 * 10^-3.5 / 2 pi = 0.412 (divided)
    g = A.frequencies(16, scaling="by_parts", factor=8.0)
    assert g[0] == f[0] and abs(g[7] - f[7] / 8.0) < 1e-18
    # f = 10^-3 makes 1.3038 turns: w = 0.10127
    w = (8.192 / (2 * math.pi) - 1.0) / 3.0
    assert abs(g[6] - 1e-3 * ((1 - w) / 8 + w)) < 1e-15


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_norms_and_relative_positions(layout):
    rng = np.random.default_rng(0)
    f = A.frequencies(32)
    q, k = rng.normal(size=(1, 1, 48)), rng.normal(size=(1, 1, 48))
    dots = []
    for p in (0, 5, 100000):
        a, _ = A.rotate(q, np.array([p + 7]), f, layout)
        b, _ = A.rotate(k, np.array([p]), f, layout)
        assert abs(np.sum(a * a) - np.sum(q * q)) < 1e-9
        assert np.array_equal(a[..., 32:], q[..., 32:])
        dots.append(np.sum(a * b))
    assert max(dots) - min(dots) < 1e-8
    zero, _ = A.rotate(q, np.array([0]), f, layout)
    assert np.array_equal(zero, q)


def test_rotation_by_hand():
    f = np.array([math.pi / 2, math.pi])  # quarter and half turns
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    y, mag = A.rotate(x, np.array([1]), f, "half")          # pairs (1, 3), (2, 4)
    assert np.allclose(y, [[[-3.0, -2.0, 1.0, -4.0]]], atol=1e-15) and np.allclose(mag, [[[4.0, 6.0, 4.0, 6.0]]])
    y, _ = A.rotate(x, np.array([1]), f, "interleaved")     # pairs (1, 2), (3, 4)
    assert np.allclose(y, [[[-2.0, 1.0, -3.0, -4.0]]], atol=1e-15)


def test_norm_by_hand():
    y = A.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, np.array([[3.0, 8.0]]) / math.sqrt(12.5), atol=1e-15)


def test_append_and_gather_by_hand():
    cK, cV = np.zeros((3, 1, 2, 1)), np.zeros((3, 1, 2, 1))
    k = np.arange(1.0, 7.0).reshape(6, 1, 1)
    # sequence 0: 3 rows at positions 1..3; sequence 1: none; sequence 2: 2 rows, the first before position 0;
    # row 5 lies behind the last sequence
    cu, kv = [0, 3, 3, 5], [4, 9, 1]
    table = np.array([[2, 0], [7, 7], [1, -1]])
    done = A.append(cK, cV, k, 10 * k, cu, kv, table)
    assert done == [(0, 2, 1), (1, 0, 0), (2, 0, 1), (4, 1, 0)]
    assert cK[:, 0, :, 0].tolist() == [[2.0, 3.0], [5.0, 0.0], [0.0, 1.0]]
    assert np.array_equal(cV, 10 * cK)
    assert A.gather(cK, table[0], 3)[:, 0, 0].tolist() == [0.0, 1.0, 2.0]
    assert A.gather(cK, table[1], 1)[:, 0, 0].tolist() == [0.0]  # a page outside the cache


def test_attention_by_hand():
    # two keys whose scores differ by ln 3: weights 1/4 and 3/4
    cK = np.zeros((1, 1, 4, 1))
    cV = np.zeros((1, 1, 4, 1))
    cK[0, 0, :, 0] = [0.0, math.log(3.0), np.nan, np.nan]
    cV[0, 0, :, 0] = [8.0, 4.0, np.nan, np.nan]
    q = np.ones((3, 1, 1))
    o, tol, written = A.attention(q, cK, cV, [0, 2, 3], [2, 0], np.array([[0], [0]]), scale=1.0)
    assert np.allclose(o[:, 0, 0], [8.0, 5.0, 0.0]) and written.tolist() == [True] * 3
    assert np.all(tol[:2] > 0) and np.all(tol[:2] < 0.1)


def test_grouped_heads_share_keys():
    rng = np.random.default_rng(1)
    cK, cV = rng.normal(size=(2, 2, 4, 8)), rng.normal(size=(2, 2, 4, 8))
    q = rng.normal(size=(3, 4, 8))
    table = np.array([[1, 0]])
    o, _, _ = A.attention(q, cK, cV, [0, 3], [7], table)
    for h in range(4):
        p, _, _ = A.attention(q[:, h:h + 1], cK[:, h // 2:h // 2 + 1], cV[:, h // 2:h // 2 + 1], [0, 3], [7], table)
        assert np.allclose(o[:, h], p[:, 0])
    # a direct sum for one row
    keys = np.concatenate([cK[1, 0], cK[0, 0]])[:6]
    vals = np.concatenate([cV[1, 0], cV[0, 0]])[:6]
    w = np.exp(keys @ q[1, 0] / math.sqrt(8))
    assert np.allclose(o[1, 0], (w[:, None] * vals).sum(0) / w.sum())
