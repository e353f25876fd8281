"""Pins of oracle.decode against something other than itself: exact rationals
for codes and products, torch's bf16 rounding, scipy's logsumexp with a sort of
every continuation for the selection, an explicit loop for the reordering."""
from fractions import Fraction

import numpy as np
import pytest
import torch
from scipy.special import logsumexp

from oracle import decode


def test_bf16_round_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(5000).astype(np.float32) * np.float32(10.0) ** rng.integers(-30, 30, 5000),
                        np.array([0.0, -0.0, np.inf, -np.inf, 3.4e38, 1e-40], dtype=np.float32)]).astype(np.float32)
    want = torch.from_numpy(x).bfloat16().float().numpy()
    assert np.array_equal(decode.bf16_round(x), want)


def _nearest_even(f: Fraction) -> int:
    return round(f)   # Python rounds a Fraction half to even


@pytest.mark.parametrize("seed", [0, 1])
def test_codes_are_the_rounded_exact_quotients(seed):
    rng = np.random.default_rng(seed)
    u = decode.bf16_round(rng.standard_normal((20, 37)).astype(np.float32))
    u[3] = 0
    u[4] = np.arange(37)          # many quotients in the middle between two codes
    u[4, -1] = 254
    codes, scales = decode.quantize(u)
    for i in range(20):
        top = max(abs(Fraction(float(v))) for v in u[i])
        for j in range(37):
            want = 0 if top == 0 else _nearest_even(127 * Fraction(float(u[i, j])) / top)
            assert codes[i, j] == want
        assert scales[i] == pytest.approx(float(top / 127), rel=1e-15)
    u[5, 2] = np.nan
    u[6, 0] = -np.inf
    codes, scales = decode.quantize(u)
    assert np.isnan(scales[[5, 6]]).all() and (codes[[5, 6]] == 0).all() and np.isfinite(scales[7:]).all()


def test_norm_against_its_formula():
    rng = np.random.default_rng(2)
    x, r = rng.standard_normal((2, 9, 64)).astype(np.float32)
    g = (1 + 0.1 * rng.standard_normal(64)).astype(np.float32)
    codes, scales, h = decode.rms_norm(x, g, 1e-6, residual=r)
    assert np.array_equal(h, x + r)
    y = h.astype(np.float64) / np.sqrt(np.mean(h.astype(np.float64) ** 2, axis=1, keepdims=True) + 1e-6) * g
    assert np.abs(codes * scales[:, None] - y).max() <= 0.5 * scales.max() * (1 + 1e-9)
    assert np.abs(scales - np.abs(y).max(1) / 127).max() < 1e-14


def test_product_sums_are_exact():
    rng = np.random.default_rng(3)
    q = rng.integers(-128, 128, (4, 48)).astype(np.int8)
    w = rng.integers(-128, 128, (5, 48)).astype(np.int8)
    one = decode.product(q, np.ones(4, np.float32), w, np.ones(5, np.float32))
    for i in range(4):
        for j in range(5):
            assert one[i, j] == sum(int(a) * int(b) for a, b in zip(q[i], w[j]))


def test_selection_against_a_sort_of_everything():
    rng = np.random.default_rng(4)
    B, K, V, n = 3, 4, 50, 7
    logits = np.round(rng.standard_normal((B * K, V)) * 2, 1)      # equal logits
    logits[rng.random((B * K, V)) < 0.1] = -np.inf
    logits[5] = logits[4]                                          # equal rows: ties across beams
    scores = -rng.random((B, K))
    scores[1, 1] = scores[1, 0]
    scores[2, 3] = -np.inf
    finished = np.zeros((B, K), dtype=bool)
    finished[0, 2] = True
    s, p, t, _ = decode.beam_select(logits, scores, n, finished, pad_token=9)
    for b in range(B):
        every = []
        for k in range(K):
            if scores[b, k] == -np.inf:
                continue
            if finished[b, k]:
                every.append((-scores[b, k], k, 9))
                continue
            z = logsumexp(logits[b * K + k])
            every += [(-(scores[b, k] + (logits[b * K + k, v] - z)), k, v) for v in range(V)
                      if logits[b * K + k, v] > -np.inf]
        every = sorted((round(a, 9), k, v) for a, k, v in every)[:n]
        assert [(k, v) for _, k, v in every] == list(zip(p[b], t[b]))
        assert np.allclose([-a for a, _, _ in every], s[b], atol=1e-8)


def test_selection_with_little_to_choose_from():
    logits = np.full((2, 5), -np.inf)
    logits[0, 3] = 1.0
    logits[1] = [np.nan, 2.0, -np.inf, 0.0, np.nan]
    s, p, t, _ = decode.beam_select(logits, np.zeros((1, 2)), 4)
    assert p[0].tolist() == [0, 1, 1, -1] and t[0].tolist() == [3, 1, 3, -1]
    assert s[0, 0] == 0 and s[0, 1] == pytest.approx(2 - np.log(np.exp(2) + 1)) and s[0, 3] == -np.inf
    logits[1, 2] = np.inf
    assert decode.beam_select(logits, np.zeros((1, 2)), 4)[1][0].tolist() == [0, -1, -1, -1]


def test_reordering():
    state = np.arange(2 * 6 * 3).reshape(2, 6, 3)
    parents = np.array([[2, 2, 0], [-1, 1, 7]])
    out = decode.beam_reorder(state, parents, 1)
    assert np.array_equal(out[:, 0], state[:, 2]) and np.array_equal(out[:, 1], state[:, 2])
    assert np.array_equal(out[:, 2], state[:, 0]) and np.array_equal(out[:, 3:], state[:, 3:])
