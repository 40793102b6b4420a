"""GPU parity of the norm + rotation of query and key heads with the float64 oracle.

Bounds are element by element.  The kernels work in fp32 (unit roundoff 2^-24): a result is a
handful of products and sums of its pair's members, so its error is at most kF32 = 2^-20 times
the sum of the magnitudes that enter it (16 roundings); the mean of squares and the mean of G h
are sums of at most 256 terms over 8 + 5 additions, which kF32 covers too.  bf16 outputs add
their own rounding, kBf16 = 2^-8 of the result.  The weights' gradients sum over tokens and
heads: a thread's chain here is under 500 additions, so 2^-15 of the sum of magnitudes.
"""

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import attention_oracle as ref

pytestmark = pytest.mark.gpu

kF32, kBf16, kSum = 2.0 ** -20, 2.0 ** -8, 2.0 ** -15
EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def _draw(seed, t, hq, hk, d, rot, dtype, *, fused=True, table=None, weights=True):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, (hq + 2 * hk) * d, generator=gen).to(dtype).cuda()
    if not fused:
        x = x.clone()
    q = x[:, :hq * d].unflatten(1, (hq, d))
    k = x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    table = table or t
    cos, sin = muon.rope_tables(table, rot, base=100.0)
    w = [(1 + 0.3 * torch.randn(d, generator=gen)).cuda() if weights else None for _ in range(2)]
    dy = [torch.randn(t, h, d, generator=gen).to(dtype).cuda() for h in (hq, hk)]
    pos = torch.randint(0, table, (t,), generator=gen, dtype=torch.int32).cuda()
    return q, k, cos, sin, w, dy, pos


def _within(got, want, bound, what):
    err = np.abs(f64(got) - want)
    assert np.all(err <= bound + 1e-30), (what, float((err - bound).max()))


def _check(q, k, cos, sin, w, dy, pos, *, norm=True, interleaved=False, stream=None):
    kw = dict(q_weight=w[0], k_weight=w[1], positions=pos, norm=norm, eps=EPS,
              interleaved=interleaved, stream=stream)
    y = muon.qk_norm_rope(q, k, cos, sin, **kw)
    dx = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **kw)
    torch.cuda.synchronize()
    c, s = f64(cos), f64(sin)
    p = np.arange(q.shape[0]) if pos is None else pos.cpu().numpy()
    okw = dict(norm=norm, eps=EPS, interleaved=interleaved)
    u = kBf16 if q.dtype == torch.bfloat16 else 0.0
    for n, x in enumerate((q, k)):
        if x.shape[1] == 0:
            continue
        X, W, G = f64(x), None if w[n] is None else f64(w[n]), f64(dy[n])
        want = ref.norm_rope(X, W, c, s, p, **okw)
        a, b = ref.pairs(2 * c.shape[1], interleaved)
        mag = np.abs(ref.norm_rope(X, W, np.zeros_like(c), np.zeros_like(c), p, **okw))
        n_ = np.abs(ref.norm_rope(X, W, np.ones_like(c), np.zeros_like(c), p, **okw))
        mag[..., a], mag[..., b] = n_[..., a] + n_[..., b], n_[..., a] + n_[..., b]
        _within(y[n], want, u * np.abs(want) + kF32 * (1 + u) * mag, "y")
        dwant, dw = ref.norm_rope_backward(G, X, W, c, s, p, **okw)
        # magnitudes: the rotated gradient, and r (|G| + |h| mean |G h|)
        g = np.abs(G).copy()
        g[..., a], g[..., b] = g[..., a] + g[..., b], g[..., a] + g[..., b]
        mag = g
        if norm:
            r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True) + EPS)
            h = np.abs(X) * r
            gw = g if W is None else g * np.abs(W)
            mag = r * (gw + h * np.mean(gw * h, -1, keepdims=True))
        _within(dx[n], dwant, u * np.abs(dwant) + kF32 * (1 + u) * mag, "dx")
        if w[n] is None:
            assert dx[2 + n] is None
        else:
            _within(dx[2 + n], dw, kSum * np.sum(g * h, axis=(0, 1)), "dw")
    return y, dx


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,rot", [
    (1, 1, 1, 8, 8), (33, 8, 4, 64, 64), (129, 5, 5, 80, 80), (257, 9, 3, 96, 64),
    (130, 4, 1, 128, 8), (65, 3, 1, 256, 256), (40, 2, 1, 24, 16), (700, 33, 8, 128, 128)])
def test_parity(t, hq, hk, d, rot, interleaved, dtype):
    _check(*_draw(t + d, t, hq, hk, d, rot, dtype), interleaved=interleaved)


@pytest.mark.parametrize("norm,weights,rot,with_pos", [
    (False, False, 64, True), (True, False, 64, False), (True, True, 0, False),
    (False, False, 0, True)])
def test_options(norm, weights, rot, with_pos):
    q, k, cos, sin, w, dy, pos = _draw(7, 77, 6, 2, 64, rot, torch.bfloat16, weights=weights)
    _check(q, k, cos, sin, w, dy, pos if with_pos else None, norm=norm)


def test_one_weight_only_and_one_side_only():
    q, k, cos, sin, w, dy, pos = _draw(8, 50, 4, 2, 64, 64, torch.float32)
    _check(q, k, cos, sin, [w[0], None], dy, pos)
    _check(q, k, cos, sin, [None, w[1]], dy, pos)
    _check(q, k[:, :0], cos, sin, [w[0], None], [dy[0], dy[1][:, :0]], pos)


def test_in_place_and_strided_outputs():
    q, k, cos, sin, w, dy, pos = _draw(9, 120, 8, 4, 64, 64, torch.bfloat16)
    kw = dict(q_weight=w[0], k_weight=w[1], positions=pos)
    y = muon.qk_norm_rope(q, k, cos, sin, **kw)
    dx = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **kw)
    fused = torch.full((120, 16 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    vq, vk = fused[:, :512].unflatten(1, (8, 64)), fused[:, 512:768].unflatten(1, (4, 64))
    muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, dq=vq, dk=vk, **kw)
    assert torch.equal(vq, dx[0]) and torch.equal(vk, dx[1])
    assert torch.all(fused[:, 768:] == 7.0)
    out = muon.qk_norm_rope(q, k, cos, sin, q_out=q, k_out=k, **kw)
    assert out[0] is q and torch.equal(q, y[0]) and torch.equal(k, y[1])


def test_repeated_calls_give_equal_bits():
    a = _draw(10, 5000, 8, 4, 64, 64, torch.bfloat16)
    q, k, cos, sin, w, dy, pos = a
    kw = dict(q_weight=w[0], k_weight=w[1], positions=pos)
    first = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **kw)
    for _ in range(3):
        again = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **kw)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_many_tokens_weight_gradient():
    # more tokens than resident warps: every block and both levels of the sum take part
    _check(*_draw(11, 20011, 3, 1, 64, 64, torch.float32))


def test_gradient_is_the_difference_quotient_of_the_forward_kernel():
    q, k, cos, sin, w, dy, pos = _draw(12, 24, 4, 2, 64, 48, torch.float32)
    kw = dict(positions=pos, eps=1e-2)
    grads = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, q_weight=w[0], k_weight=w[1],
                                       **kw)
    gen = torch.Generator().manual_seed(1)
    dirs = [torch.randn(x.shape, generator=gen).cuda() for x in (q, k, w[0], w[1])]

    def loss(step):
        x = [a + step * b for a, b in zip((q, k, w[0], w[1]), dirs)]
        y = muon.qk_norm_rope(x[0], x[1], cos, sin, q_weight=x[2], k_weight=x[3], **kw)
        return sum((f64(a) * f64(b)).sum() for a, b in zip(y, dy))

    h = 2.0 ** -8
    quotient = (loss(h) - loss(-h)) / (2 * h)
    want = sum((f64(a) * f64(b)).sum() for a, b in zip(grads, dirs))
    # rounding: 2^-22 a term, 9216 terms of size ~1 added at random, over 2 h; truncation
    # h^2 / 6 times a third derivative of about 10 a term, added at random
    assert abs(quotient - want) <= 2.0 ** -22 * 96 / (2 * h) * 4 + h * h / 6 * 10 * 96


def test_position_outside_the_tables_gives_nan_there_only():
    q, k, cos, sin, w, dy, pos = _draw(13, 20, 4, 2, 64, 32, torch.bfloat16)
    pos[3], pos[11] = 20, -1
    bad = torch.zeros(20, dtype=torch.bool, device="cuda")
    bad[[3, 11]] = True
    y = muon.qk_norm_rope(q, k, cos, sin, positions=pos)
    dx = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, positions=pos)
    for x in (*y, *dx[:2]):
        assert torch.isnan(x[bad]).all() and torch.isfinite(x[~bad]).all()


def test_non_finite_heads_stay_alone():
    q, k, cos, sin, w, dy, pos = _draw(14, 20, 4, 2, 64, 32, torch.float32, fused=False)
    q[5, 1, 40], k[7, 0, 3] = float("inf"), float("nan")
    y = muon.qk_norm_rope(q, k, cos, sin, positions=pos)
    ok = torch.ones(20, 4, dtype=torch.bool, device="cuda")
    ok[5, 1] = False
    assert torch.isfinite(y[0][ok]).all() and not torch.isfinite(y[0][5, 1]).all()
    assert not torch.isfinite(y[1][7, 0]).any()
    # without a norm, an unrotated element passes as it is
    y = muon.qk_norm_rope(q, k, cos, sin, positions=pos, norm=False)
    assert torch.isinf(y[0][5, 1, 40]) and torch.isfinite(y[0][5, 1]).sum() == 63


def test_zero_tokens():
    q, k, cos, sin, w, dy, pos = _draw(15, 4, 4, 2, 64, 64, torch.bfloat16)
    e = dict(q_weight=w[0], k_weight=w[1], positions=pos[:0])
    before = muon.kernel_launch_count()
    y = muon.qk_norm_rope(q[:0], k[:0], cos, sin, **e)
    dx = muon.qk_norm_rope_backward(dy[0][:0], dy[1][:0], q[:0], k[:0], cos, sin, **e)
    assert y[0].shape == (0, 4, 64) and dx[1].shape == (0, 2, 64)
    assert torch.count_nonzero(dx[2]) == 0 and torch.count_nonzero(dx[3]) == 0
    assert muon.kernel_launch_count() == before


def test_another_stream_and_explicit_workspace():
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    _check(*_draw(16, 300, 8, 4, 64, 64, torch.bfloat16), stream=st)
    q, k, cos, sin, w, dy, pos = _draw(16, 300, 8, 4, 64, 64, torch.bfloat16)
    ws = muon.Workspace(muon.norm_rope_workspace_bytes(64))
    muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, q_weight=w[0], workspace=ws)
    assert muon.workspace_status(ws) == 0
    assert torch.count_nonzero(ws.tensor[:256]) == 0      # tickets return to zero


def test_refusals():
    q, k, cos, sin, w, dy, pos = _draw(17, 20, 4, 2, 64, 64, torch.bfloat16)
    for bad, exc in [((q.half(), k.half(), cos, sin), TypeError), ((q, k.float(), cos, sin), TypeError),
                     ((q[:5], k, cos, sin), ValueError), ((q, k, cos.double(), sin), TypeError),
                     ((q, k, cos, sin[:3]), ValueError), ((q[0], k, cos, sin), ValueError),
                     ((q.transpose(1, 2), k, cos, sin), ValueError)]:
        with pytest.raises(exc):
            muon.qk_norm_rope(*bad)
    with pytest.raises(ValueError):
        muon.qk_norm_rope(q, k, cos, sin, norm=False, q_weight=w[0])
    with pytest.raises(TypeError):
        muon.qk_norm_rope(q, k, cos, sin, positions=pos.long())
    with pytest.raises(muon.MuonError):                    # fewer table rows than tokens
        muon.qk_norm_rope(q, k, cos[:10], sin[:10])
    with pytest.raises(muon.MuonError):                    # rows of the output overlap
        muon.qk_norm_rope(q, k, cos, sin, q_out=torch.empty_like(q[:1]).expand_as(q))
    with pytest.raises(muon.MuonError):                    # not 16-byte aligned
        muon.qk_norm_rope(torch.empty(20 * 256 + 1, dtype=q.dtype, device="cuda")[1:].view(
            20, 4, 64), k, cos, sin)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hk,d,rot", [(2, 1, 24, 16), (1, 1, 80, 80), (3, 1, 96, 64),
                                         (2, 2, 40, 8), (1, 1, 200, 200)])
def test_position_outside_the_tables_with_lanes_past_the_head(hq, hk, d, rot, interleaved, dtype):
    # d / 8 is no power of two: some lanes of a row hold none of its elements
    t = 150
    q, k, cos, sin, w, dy, pos = _draw(18 + d, t, hq, hk, d, rot, dtype)
    bad = torch.zeros(t, dtype=torch.bool, device="cuda")
    bad[[0, 3, 11, 64, 149]] = True
    p = torch.where(bad, torch.tensor(t, dtype=torch.int32, device="cuda"), pos)
    kw = dict(q_weight=w[0], k_weight=w[1], interleaved=interleaved)
    y = muon.qk_norm_rope(q, k, cos, sin, positions=p, **kw)
    dx = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, positions=p, **kw)
    good = muon.qk_norm_rope(q, k, cos, sin, positions=pos, **kw)
    good += muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, positions=pos, **kw)[:2]
    for x, want in zip((*y, *dx[:2]), good):
        assert torch.isnan(x[bad]).all() and torch.equal(x[~bad], want[~bad])


def test_outputs_over_other_inputs_are_refused():
    q, k, cos, sin, w, dy, pos = _draw(20, 50, 4, 4, 64, 64, torch.bfloat16)
    kw = dict(q_weight=w[0], k_weight=w[1], positions=pos)
    want = muon.qk_norm_rope(q, k, cos, sin, **kw)
    dwant = muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **kw)
    before = [x.clone() for x in (q, k, *dy)]
    spare = torch.empty(51, 8, 64, dtype=q.dtype, device="cuda")
    for bad in (dict(q_out=k), dict(k_out=q), dict(q_out=spare[:50, :4], k_out=spare[1:, 3:7])):
        with pytest.raises(muon.MuonError):
            muon.qk_norm_rope(q, k, cos, sin, **bad, **kw)
    for bad in (dict(dq=k), dict(dk=q), dict(dq=dy[1]), dict(dk=dy[0]),
                dict(dq=spare[:50, :4], dk=spare[1:, 3:7])):
        with pytest.raises(muon.MuonError):
            muon.qk_norm_rope_backward(dy[0], dy[1], q, k, cos, sin, **bad, **kw)
    with pytest.raises(muon.MuonError):                    # rows of its own input, a token on
        muon.qk_norm_rope(spare[:50, :4], k, cos, sin, q_out=spare[1:, :4], **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((q, k, *dy), before))
    # over the gradients of the outputs, and over the inputs
    g = [x.clone() for x in dy]
    got = muon.qk_norm_rope_backward(*g, q, k, cos, sin, dq=g[0], dk=g[1], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, dwant))
    x = [q.clone(), k.clone()]
    got = muon.qk_norm_rope_backward(*dy, *x, cos, sin, dq=x[0], dk=x[1], **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, dwant))
    got = muon.qk_norm_rope(q, k, cos, sin, q_out=q, k_out=k, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
