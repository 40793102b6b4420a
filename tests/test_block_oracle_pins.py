"""Pins of the block operators' oracle: brute force, differences, all 8-bit values."""

import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as ref


def _draw(seed, *shapes):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in shapes]


def _quotient(f, x, e=1e-6):
    out = np.empty_like(x)
    for i in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += e
        lo[i] -= e
        out[i] = (f(hi) - f(lo)) / (2 * e)
    return out


@pytest.mark.parametrize("kind", [None, "relu2", "gelu"])
def test_activation_by_hand(kind):
    z = np.array([-40.0, -3.0, -0.25, 0.0, 0.5, 2.0, 40.0])
    want = []
    for v in z:
        if kind == "relu2":
            want.append(max(v, 0.0) ** 2)
        elif kind == "gelu":
            want.append(0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))))
        else:
            want.append(v)
    np.testing.assert_allclose(ref.act(z, kind), want, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("kind", [None, "relu2", "gelu"])
def test_linear_gradients_are_difference_quotients(kind):
    x, w, b, r, dy = _draw(1, (3, 5), (4, 5), (4,), (3, 4), (3, 4))
    y, z = ref.linear(x, w, b, kind, r)
    for i in range(3):
        for j in range(4):
            s = b[j] + sum(x[i, k] * w[j, k] for k in range(5))
            assert abs(s - z[i, j]) < 1e-12
    dx, dw, db = ref.linear_backward(dy, x, w, kind, z)
    for got, f, at in [(dx, lambda v: ref.linear(v, w, b, kind, r), x),
                       (dw, lambda v: ref.linear(x, v, b, kind, r), w),
                       (db, lambda v: ref.linear(x, w, v, kind, r), b)]:
        np.testing.assert_allclose(got, _quotient(lambda v: np.sum(dy * f(v)[0]), at), rtol=1e-6,
                                   atol=1e-7)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("with_res", [True, False])
def test_rms_norm_gradients_are_difference_quotients(weighted, with_res):
    x, w, r, dy, dr = _draw(2, (3, 8), (8,), (3, 8), (3, 8), (3, 8))
    w, r, dr = w if weighted else None, r if with_res else None, dr if with_res else None
    eps = 1e-2
    y, h = ref.rms_norm(x, w, r, eps)
    for i in range(3):
        ms = sum(float(v) ** 2 for v in h[i]) / 8
        for j in range(8):
            want = h[i, j] / math.sqrt(ms + eps) * (1 if w is None else w[j])
            assert abs(y[i, j] - want) < 1e-12

    def loss(x, w):
        y, h = ref.rms_norm(x, w, r, eps)
        return np.sum(dy * y) + (np.sum(dr * h) if with_res else 0.0)

    dx, dw = ref.rms_norm_backward(dy, h, w, dr, eps)
    np.testing.assert_allclose(dx, _quotient(lambda v: loss(v, w), x), rtol=1e-6, atol=1e-7)
    if weighted:
        np.testing.assert_allclose(dw, _quotient(lambda v: loss(x, v), w), rtol=1e-6, atol=1e-7)


def test_e4m3_takes_every_value_to_itself_and_rounds_as_the_type():
    values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    values = values[np.isfinite(values)]
    assert np.array_equal(ref.e4m3(values), values) and values.max() == ref.E4M3_MAX
    v = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.05, 0.05, 4001)])
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    got = ref.e4m3(torch.from_numpy(v).float().double().numpy())
    assert np.array_equal(got, want)


def test_scales_are_least_powers_of_two():
    y = np.array([[448.0, 0, 449.0, 1, 0, 0, 2.0 ** -140, 0], [7.0, -7.1, 3.5, 0, np.inf, 1, 0, 0]])
    s = ref.group_scales(y, 2)
    assert s[0].tolist() == [1.0, 2.0, 1.0, 2.0 ** -126]
    assert s[1, 0] == 2.0 ** -5 and s[1, 1] == 2.0 ** -7 and np.isnan(s[1, 2]) and s[1, 3] == 1.0
    for i in range(2):
        for g in range(4):
            top = np.abs(y[i, 2 * g:2 * g + 2]).max()
            if np.isfinite(top) and top > 2.0 ** -120:
                assert top <= 448 * s[i, g] and top > 448 * s[i, g] / 2
    assert ref.group_scales(y[:1], 0).shape == (1, 1)
    assert ref.spread(s, 8, 2)[0, 3] == s[0, 1]


def test_embedding_gradient_is_the_difference_quotient():
    table, dy = _draw(3, (5, 4), (7, 4))
    ids = np.array([3, 0, 3, 4, -1, 3, 5])
    y = ref.embedding(ids, table, 2.0)
    assert np.isnan(y[[4, 6]]).all() and np.array_equal(y[0], 2 * table[3])
    good = np.array([0, 1, 2, 3, 5])
    want = _quotient(lambda t: np.sum(dy[good] * ref.embedding(ids[good], t, 2.0)), table)
    np.testing.assert_allclose(ref.embedding_backward(dy, ids, 5, 2.0), want, rtol=1e-6, atol=1e-7)


def test_clip_factor():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    assert ref.grad_norm(g) == 5.0
    assert ref.clip_factor(5.0, 10.0) == 1.0
    assert abs(ref.clip_factor(5.0, 1.0, 0.0) - 0.2) < 1e-15
