"""Pins of the attention-path oracle: brute-force loops, differences, invariants."""

import math

import numpy as np
import pytest

from oracle import attention_oracle as ref


def _draw(seed, *shapes):
    r = np.random.default_rng(seed)
    return [r.standard_normal(s) for s in shapes]


def _tables(length, rot):
    ang = np.arange(length)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / max(rot, 1))[None, :]
    return np.cos(ang), np.sin(ang)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 8])
def test_norm_rope_brute_force(interleaved, rot):
    t, h, d, eps = 3, 2, 8, 1e-3
    x, w = _draw(0, (t, h, d), (d,))
    cos, sin = _tables(10, rot)
    pos = np.array([4, 0, 9])
    y = ref.norm_rope(x, w, cos, sin, pos, eps=eps, interleaved=interleaved)
    for i in range(t):
        for j in range(h):
            ms = sum(float(e) ** 2 for e in x[i, j]) / d
            n = [x[i, j, e] / math.sqrt(ms + eps) * w[e] for e in range(d)]
            want = list(n)
            for p in range(rot // 2):
                a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
                c, s = cos[pos[i], p], sin[pos[i], p]
                # the pair as a complex number times e^(i angle)
                z = complex(n[a], n[b]) * complex(c, s)
                want[a], want[b] = z.real, z.imag
            np.testing.assert_allclose(y[i, j], want, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("norm,weighted,interleaved", [(True, True, False), (True, False, True),
                                                       (False, False, True)])
def test_norm_rope_gradient_is_the_difference_quotient(norm, weighted, interleaved):
    t, h, d, rot = 2, 2, 8, 4
    x, dy, w = _draw(1, (t, h, d), (t, h, d), (d,))
    w = w if weighted else None
    cos, sin = _tables(t, rot)
    kw = dict(norm=norm, eps=1e-2, interleaved=interleaved)
    pos = np.arange(t)
    dx, dw = ref.norm_rope_backward(dy, x, w, cos, sin, pos, **kw)

    def loss(x, w):
        return np.sum(dy * ref.norm_rope(x, w, cos, sin, pos, **kw))

    e = 1e-6
    for idx in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[idx] += e
        lo[idx] -= e
        assert abs((loss(hi, w) - loss(lo, w)) / (2 * e) - dx[idx]) < 1e-7
    for i in range(d if weighted else 0):
        hi, lo = w.copy(), w.copy()
        hi[i] += e
        lo[i] -= e
        assert abs((loss(x, hi) - loss(x, lo)) / (2 * e) - dw[i]) < 1e-7


CU = [0, 3, 3, 4, 9]      # lengths 3, 0, 1, 5, then two tokens past the end


def test_attention_brute_force():
    t, hq, hk, d = 11, 4, 2, 5
    q, k, v = _draw(2, (t, hq, d), (t, hk, d), (t, hk, d))
    out, lse = ref.attention(q, k, v, CU, scale=0.7)
    start = [0, 0, 0, 3, 4, 4, 4, 4, 4]
    for h in range(hq):
        for i in range(t):
            if i >= CU[-1]:
                assert lse[h, i] == -np.inf and np.all(out[i, h] == 0)
                continue
            js = range(start[i], i + 1)
            e = [math.exp(0.7 * float(q[i, h] @ k[j, h // 2])) for j in js]
            assert abs(lse[h, i] - math.log(sum(e))) < 1e-12
            want = sum(x * v[j, h // 2] for x, j in zip(e, js)) / sum(e)
            np.testing.assert_allclose(out[i, h], want, rtol=1e-12, atol=1e-14)


def test_attention_gradient_is_the_difference_quotient():
    t, hq, hk, d = 11, 4, 2, 3
    q, k, v, do = _draw(3, (t, hq, d), (t, hk, d), (t, hk, d), (t, hq, d))
    out, lse = ref.attention(q, k, v, CU)
    grads = ref.attention_backward(do, q, k, v, out, lse, CU)
    e = 1e-6
    for n, g in enumerate(grads):
        assert g.shape == (q, k, v)[n].shape
        for idx in np.ndindex(g.shape):
            hi, lo = [q, k, v], [q, k, v]
            hi[n], lo[n] = hi[n].copy(), lo[n].copy()
            hi[n][idx] += e
            lo[n][idx] -= e
            d_loss = np.sum(do * (ref.attention(*hi, CU)[0] - ref.attention(*lo, CU)[0])) / (2 * e)
            assert abs(d_loss - g[idx]) < 1e-7
    for g in grads:
        assert np.all(g[CU[-1]:] == 0)


def test_non_finite_values_stay_in_their_sequence_and_after_their_token():
    t, h, d = 9, 1, 4
    q, k, v, do = _draw(4, *[(t, h, d)] * 4)
    v[6, 0, 1] = np.inf
    k[2, 0, 0] = np.nan
    out, lse = ref.attention(q, k, v, CU)
    bad = ~np.isfinite(out[:, 0]).all(axis=1)
    assert list(np.nonzero(bad)[0]) == [2, 6, 7, 8]
    assert np.isfinite(lse[0, [0, 1, 3, 4, 5, 6, 7, 8]]).all() and np.isnan(lse[0, 2])
    dq, dk, dv = ref.attention_backward(do, q, k, v, out, lse, CU)
    # queries 6..8 see v_6; a key is reached by the queries at or after it in its sequence
    assert np.isfinite(dq[[0, 1, 3, 4, 5]]).all()
    assert np.isfinite(dv[[3]]).all() and np.isfinite(dk[[3]]).all()
    assert np.isfinite(dv[4:]).all()          # the weights themselves are finite there
