"""GPU parity of the RMS norm with the residual's addition, its 8-bit form and its gradients, with
the float64 oracle.

Bounds are element by element.  The kernels work in fp32: the sum of squares of up to 16384 values
is a chain of at most 32 additions a thread and 5 + 16 across threads, the other steps a handful
of roundings, so kF32 = 2^-18 of the magnitudes covers a result (64 roundings of 2^-24).  bf16
outputs add their rounding, kBf16 = 2^-8.  The weight's gradient sums over tokens: chains of
under 500 additions here, 2^-15 of the sum of magnitudes.  In 8 bits the values are compared with
the oracle's scales where these are the same, half a step of e4m3 (2^-4 of the value, and 2^-10 of
the scale below 2^-6 of it) away from y.
"""

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import block_oracle as ref

pytestmark = pytest.mark.gpu

kF32, kBf16, kSum = 2.0 ** -18, 2.0 ** -8, 2.0 ** -15
EPS = 1e-6
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def _draw(seed, t, d, dtype, *, weight=True, pad=0):
    gen = torch.Generator().manual_seed(seed)

    def mat(std=1.0):
        x = torch.full((t, d + 2 * pad), float("nan"), dtype=dtype)
        x[:, pad:pad + d] = (std * torch.randn(t, d, generator=gen)).to(dtype)
        return x.to(DEV)[:, pad:pad + d]

    x, r, dy, dr = mat(), mat(3.0), mat(), mat()
    w = (1 + 0.3 * torch.randn(d, generator=gen)).to(DEV) if weight else None
    return x, r, dy, dr, w


def _within(got, want, bound, what):
    err = np.abs(f64(got) - want) - bound - 1e-30
    assert np.all(err <= 0), (what, float(err.max()))


def _check(x, r, dy, dr, w, *, eps=EPS, stream=None):
    u = kBf16 if x.dtype == torch.bfloat16 else 0.0
    X, G, W = f64(x), f64(dy), None if w is None else f64(w)
    R, D = (None if v is None else f64(v) for v in (r, dr))
    y, h = muon.rms_norm(x, w, residual=r, eps=eps, stream=stream)
    dx, dw = muon.rms_norm_backward(dy, h, w, dresidual=dr, eps=eps, stream=stream)
    torch.cuda.synchronize()
    want, wh = ref.rms_norm(X, W, R, eps)
    mag, _ = ref.rms_norm(np.abs(X), None if W is None else np.abs(W),
                          None if R is None else np.abs(R), eps)
    # (x and residual may cancel: h is off by 2^-24 of |x| + |residual|)
    s = np.abs(X) + (0 if R is None else np.abs(R))
    rms = np.sqrt(np.mean(wh * wh, axis=1, keepdims=True) + eps)
    e = kF32 * (np.abs(want) + s / rms * (1 if W is None else np.abs(W)))
    _within(y, want, e + u * (np.abs(want) + e), "y")
    if R is None:
        assert h is x
    else:
        _within(h, wh, 2.0 ** -24 * s + u * np.abs(wh) * (1 + 2.0 ** -23), "h")
    H = f64(h)
    dwant, wdw = ref.rms_norm_backward(G, H, W, D, eps)
    inv = 1 / np.sqrt(np.mean(H * H, axis=1, keepdims=True) + eps)
    n, gw = np.abs(H) * inv, np.abs(G) * (1 if W is None else np.abs(W))
    m = inv * (gw + n * np.mean(gw * n, axis=1, keepdims=True)) + (0 if D is None else np.abs(D))
    _within(dx, dwant, kF32 * m + u * (np.abs(dwant) + kF32 * m), "dx")
    if w is None:
        assert dw is None
    else:
        _within(dw, wdw, kSum * np.sum(np.abs(G) * n, axis=0), "dw")
    return y, h, dx, dw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,d", [(1, 8), (33, 64), (5, 256), (257, 264), (33, 512), (100, 520),
                                 (77, 1024), (65, 1032), (40, 2048), (33, 2056), (20, 4104),
                                 (9, 8192), (7, 8200), (5, 16384)])
def test_parity(t, d, dtype):
    _check(*_draw(t + d, t, d, dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [72, 512, 1096, 4096, 16376])
@pytest.mark.parametrize("with_r,with_d,with_w", [(False, False, True), (True, False, False),
                                                  (False, True, False)])
def test_options(d, dtype, with_r, with_d, with_w):
    x, r, dy, dr, w = _draw(3, 50, d, dtype, weight=with_w)
    _check(x, r if with_r else None, dy, dr if with_d else None, w)


def test_strided_rows_and_eps():
    _check(*_draw(4, 70, 200, torch.bfloat16, pad=8), eps=0.5)
    _check(*_draw(5, 70, 200, torch.float32, pad=4), eps=0.0)


def test_more_tokens_than_resident_rows():
    _check(*_draw(6, 20011, 64, torch.bfloat16))
    _check(*_draw(7, 5000, 520, torch.float32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("t,d", [(1, 8), (33, 64), (65, 200), (40, 512), (33, 1000), (20, 1032),
                                 (30, 4096), (9, 8200), (3, 16384)])
def test_eight_bits(t, d, group, dtype):
    x, r, _, _, w = _draw(t + d + group, t, d, dtype)
    q, s, h = muon.rms_norm_fp8(x, w, residual=r, eps=EPS, group=group)
    y, h2 = muon.rms_norm(x.float(), w, residual=r.float(), eps=EPS)
    torch.cuda.synchronize()
    assert q.dtype == torch.float8_e4m3fn and s.shape == (t, 1 if group == 0 else -(-d // 128))
    assert torch.equal(h, h2.to(dtype))
    # y in fp32, as the kernel has it before the scales: same steps, same bits
    Y, S, Q = f64(y), f64(s), f64(q.float())
    assert np.array_equal(S, ref.group_scales(Y, group))
    at = ref.spread(S, d, group)
    assert np.array_equal(Q, ref.e4m3(Y / at))
    want, _ = ref.rms_norm(f64(x), f64(w), f64(r), EPS)
    err = np.abs(Q * at - want)
    assert np.all(err <= (2.0 ** -4 + 2.0 ** -12) * np.abs(want) + 2.0 ** -10 * at + 1e-4)


@pytest.mark.parametrize("group", [0, 128])
def test_eight_bits_of_zeros_and_of_what_is_not_finite(group):
    x = torch.randn(6, 264, generator=torch.Generator().manual_seed(8)).to(DEV)
    x[1] = 0.0
    x[2, 130] = float("nan")
    x[3, 5] = float("inf")
    x[4] = 0.0
    x[4, 7] = 1e-3
    q, s, _ = muon.rms_norm_fp8(x, eps=0.5, group=group)
    v = q.float()
    assert torch.all(s[1] == 1.0) and torch.all(v[1] == 0.0)
    # a NaN makes the whole row's norm one; an Inf's own group
    assert torch.isnan(s[2]).all() and torch.isnan(v[2]).all()
    assert torch.isnan(s[3, 0]) and torch.isnan(v[3, :128]).all()
    if group:
        assert torch.all(s[3, 1:] == 1.0) and torch.all(v[3, 128:] == 0.0)
        assert torch.all(s[4, 1:] == 1.0)
    for i in (0, 5):
        assert torch.isfinite(s[i]).all() and torch.isfinite(v[i]).all()
    top = (v[4] * s[4, 0]).abs().max()
    assert 224 * s[4, 0] < top <= 448 * s[4, 0]


def test_outputs_in_place():
    for t, d in ((50, 512), (20, 4104)):
        x, r, dy, dr, w = _draw(9, t, d, torch.bfloat16)
        y, h = muon.rms_norm(x, w, residual=r)
        dx, dw = muon.rms_norm_backward(dy, h, w, dresidual=dr)
        for out, total in ((0, 1), (1, 0), (None, 1), (0, None)):
            c = [x.clone(), r.clone()]
            got = muon.rms_norm(c[0], w, residual=c[1], out=None if out is None else c[out],
                                residual_out=None if total is None else c[total])
            assert torch.equal(got[0], y) and torch.equal(got[1], h)
            assert (out is None or got[0] is c[out]) and (total is None or got[1] is c[total])
        for over in range(3):
            c = [dy.clone(), h.clone(), dr.clone()]
            got = muon.rms_norm_backward(c[0], c[1], w, dresidual=c[2], dx=c[over])
            assert got[0] is c[over] and torch.equal(got[0], dx) and torch.equal(got[1], dw)
        c = x.clone()
        assert torch.equal(muon.rms_norm(c, w, out=c)[0], muon.rms_norm(x, w)[0])


def test_outputs_given_leave_their_padding():
    x, r, dy, dr, w = _draw(10, 33, 200, torch.bfloat16)
    wide = torch.full((33, 632), 7.0, dtype=torch.bfloat16, device=DEV)
    y, h = muon.rms_norm(x, w, residual=r, out=wide[:, 8:208], residual_out=wide[:, 216:416])
    dx, _ = muon.rms_norm_backward(dy, h, w, dx=wide[:, 424:624])
    wy, wh = muon.rms_norm(x, w, residual=r)
    assert torch.equal(y, wy) and torch.equal(h, wh)
    assert torch.equal(dx, muon.rms_norm_backward(dy, wh, w)[0])
    for c in (slice(0, 8), slice(208, 216), slice(416, 424), slice(624, 632)):
        assert torch.all(wide[:, c] == 7.0)
    q = torch.zeros(33, 216, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    got = muon.rms_norm_fp8(x, w, residual=r, out=q[:, :200])
    assert torch.equal(got[0].float(), muon.rms_norm_fp8(x, w, residual=r)[0].float())
    assert torch.count_nonzero(q.view(torch.uint8)[:, 200:]) == 0


def test_a_row_that_is_not_finite_stays_alone():
    x, r, dy, dr, w = _draw(11, 40, 520, torch.bfloat16)
    x[7, 3], dy[9, 100] = float("nan"), float("inf")
    y, h = muon.rms_norm(x, w, residual=r)
    dx, dw = muon.rms_norm_backward(dy, h, w, dresidual=dr)
    rows = torch.ones(40, dtype=torch.bool, device=DEV)
    rows[7] = False
    assert torch.isnan(y[7]).all() and torch.isfinite(y[rows]).all()
    assert torch.isnan(h[7]).sum() == 1
    rows[9] = False
    assert torch.isfinite(dx[rows]).all() and torch.isnan(dx[7]).all()


def test_gradient_is_the_difference_quotient_of_the_forward_kernel():
    x, r, dy, dr, w = _draw(12, 24, 72, torch.float32)
    dx, dw = muon.rms_norm_backward(dy, muon.rms_norm(x, w, residual=r, eps=1e-2)[1], w,
                                    dresidual=dr, eps=1e-2)
    gen = torch.Generator().manual_seed(1)
    dirs = [torch.randn(v.shape, generator=gen).to(DEV) for v in (x, w)]

    def loss(step):
        y, h = muon.rms_norm(x + step * dirs[0], w + step * dirs[1], residual=r, eps=1e-2)
        return (f64(y) * f64(dy)).sum() + (f64(h) * f64(dr)).sum()

    h = 2.0 ** -8
    quotient = (loss(h) - loss(-h)) / (2 * h)
    want = (f64(dx) * f64(dirs[0])).sum() + (f64(dw) * f64(dirs[1])).sum()
    # rounding: 2^-21 a term (values up to about 8), 3456 terms added at random, over 2 h;
    # truncation h^2 / 6 times a third derivative of about 10 a term, added at random
    assert abs(quotient - want) <= 2.0 ** -21 * 60 * 4 / (2 * h) + h * h / 6 * 10 * 60


def test_repeated_captured_streams_and_status():
    x, r, dy, dr, w = _draw(13, 3000, 520, torch.bfloat16)
    y, h = muon.rms_norm(x, w, residual=r)
    want = muon.rms_norm_backward(dy, h, w, dresidual=dr)
    for _ in range(3):
        got = muon.rms_norm_backward(dy, h, w, dresidual=dr)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append((*muon.rms_norm(x, w, residual=r),
                         *muon.rms_norm_backward(dy, h, w, dresidual=dr)))
        graphs.append(g)
    for i in (1, 0):
        for v in outs[i]:
            v.fill_(3.0)
        graphs[i].replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, (y, h, *want)))
    _check(*_draw(14, 300, 64, torch.bfloat16), stream=stream)
    ws = muon.Workspace(muon.rms_norm_workspace_bytes(520))
    muon.selftest_wait_timeout(ws, limit_us=1000)
    dx = torch.full_like(x, 3.0)
    muon.rms_norm_backward(dy, h, w, dx=dx, workspace=ws)
    assert muon.workspace_status(ws, clear=True) == 4 and torch.all(dx == 3.0)
    muon.rms_norm_backward(dy, h, w, dresidual=dr, dx=dx, workspace=ws)
    assert muon.workspace_status(ws) == 0 and torch.equal(dx, want[0])


def test_zero_tokens():
    x, r, dy, dr, w = _draw(15, 3, 64, torch.bfloat16)
    before = muon.kernel_launch_count()
    y, h = muon.rms_norm(x[:0], w, residual=r[:0])
    q, s, _ = muon.rms_norm_fp8(x[:0], w)
    dx, dw = muon.rms_norm_backward(dy[:0], x[:0], w)
    assert y.shape == h.shape == q.shape == dx.shape == (0, 64) and s.shape == (0, 1)
    assert torch.count_nonzero(dw) == 0 and muon.kernel_launch_count() == before


def test_refusals():
    x, r, dy, dr, w = _draw(16, 20, 64, torch.bfloat16)
    for args, kw, exc in [((x.half(),), {}, TypeError), ((x[0],), {}, ValueError),
                          ((x, w.bfloat16()), {}, TypeError), ((x, w[:32]), {}, ValueError),
                          ((x.t(),), {}, ValueError), ((x,), dict(residual=r.float()), TypeError),
                          ((x,), dict(residual=r[:5]), ValueError),
                          ((x,), dict(residual_out=r), ValueError),
                          ((x,), dict(out=r.float()), TypeError)]:
        with pytest.raises(exc):
            muon.rms_norm(*args, **kw)
        if "out" not in kw:
            with pytest.raises(exc):
                muon.rms_norm_fp8(*args, **kw)
    with pytest.raises(ValueError):
        muon.rms_norm_fp8(x, group=64)
    with pytest.raises(TypeError):
        muon.rms_norm_fp8(x, out=torch.empty_like(x))
    for bad in (dict(out=r, residual_out=r), dict(out=x, residual_out=x)):
        with pytest.raises(muon.MuonError):
            muon.rms_norm(x, w, residual=r, **bad)
    with pytest.raises(muon.MuonError):                 # dim is no multiple of 8
        muon.rms_norm(x[:, :60])
    with pytest.raises(muon.MuonError):                 # not 16-byte aligned
        muon.rms_norm(torch.empty(20 * 64 + 1, dtype=x.dtype, device=DEV)[1:].view(20, 64))
    with pytest.raises(muon.MuonError):                 # rows over other rows of the input
        muon.rms_norm(x[:10], w, out=x[1:11])
    for v in (x, w, r):
        v.requires_grad_(True)
        with pytest.raises(ValueError, match="rms_norm_backward"):
            muon.rms_norm(x, w, residual=r)
        with pytest.raises(ValueError):
            muon.rms_norm_fp8(x, w, residual=r)
        v.requires_grad_(False)


def _spread(x, empty=False):
    """x in rows so far apart that the last ones begin past 2^31 elements."""
    rows, cols = x.shape
    stride = ((1 << 31) // (rows - 2) // 8 + 1) * 8
    buf = torch.empty((rows - 1) * stride + (cols + 7) // 8 * 8, dtype=x.dtype, device=DEV)
    view = buf.as_strided((rows, cols), (stride, 1))
    assert (rows - 1) * stride > 1 << 31
    view.fill_(3.0) if empty else view.copy_(x)
    return view


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_offsets_past_32_bits(dtype):
    gen = torch.Generator().manual_seed(43)
    x, r, dy = (torch.randn(50, 1024, generator=gen).to(dtype).to(DEV) for _ in range(3))
    w = torch.randn(1024, generator=gen).to(DEV)
    y, h = muon.rms_norm(x, w, residual=r)
    dx, dw = muon.rms_norm_backward(dy, h, w, dresidual=r)
    q, s, _ = muon.rms_norm_fp8(x, w, residual=r)
    X, R, DY = (_spread(v) for v in (x, r, dy))
    Y, H, DX = (_spread(x, True) for _ in range(3))
    muon.rms_norm(X, w, residual=R, out=Y, residual_out=H)
    assert torch.equal(Y, y) and torch.equal(H, h)
    got = muon.rms_norm_backward(DY, H, w, dresidual=R, dx=DX)
    assert torch.equal(DX, dx) and torch.equal(got[1], dw)
    Q = _spread(q.view(torch.uint8), True).view(torch.float8_e4m3fn)
    _, S, _ = muon.rms_norm_fp8(X, w, residual=R, out=Q, residual_out=H)
    assert torch.equal(Q.view(torch.uint8), q.view(torch.uint8)) and torch.equal(S, s)


# magnitudes of rows whose squares leave fp32's range, between ordinary ones (the residual is three
# times x: the largest sums stay below 2^128)
MAGNITUDES = [1.0, 1e20, 1e-24, 1e37, 1e-12, 1e-36, 1e15, 1.0, 1e19, 1e-20]


def _check_far(x, r, dy, dr, w, eps):
    """As _check, but a residual's y may be that of h as stored: rounded, it moves an element and the
    row's norm by kBf16 of themselves each."""
    u = kBf16 if x.dtype == torch.bfloat16 else 0.0
    X, R, W = (None if v is None else f64(v) for v in (x, r, w))
    y, h = muon.rms_norm(x, w, residual=r, eps=eps)
    want, wh = ref.rms_norm(X, W, R, eps)
    s = np.abs(X) + (0 if R is None else np.abs(R))
    rms = np.sqrt(np.mean(wh * wh, axis=1, keepdims=True) + eps)
    e = kF32 * (np.abs(want) + s / rms * (1 if W is None else np.abs(W)))
    e = e + (0.0 if R is None else 2 * u * np.abs(want))
    _within(y, want, e + u * (np.abs(want) + e), "y")
    _within(h, wh, 2.0 ** -24 * s + u * np.abs(wh) * (1 + 2.0 ** -23), "h")
    # from h on there is no difference
    _check(h, None, dy, dr, w, eps=eps)
    # ... nor by where the outputs are
    for out in (0, 1):
        c = [x.clone(), None if r is None else r.clone()]
        total = None if r is None else c[1 - out]
        got = muon.rms_norm(c[0], w, residual=c[1], eps=eps, out=c[out], residual_out=total)
        assert torch.equal(got[0], y) and (r is None or torch.equal(got[1], h))
        if r is None:
            break


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
@pytest.mark.parametrize("d", [64, 264, 520, 2048, 4104, 16384])
def test_rows_of_any_magnitude(d, eps, dtype):
    x, r, dy, dr, w = _draw(44 + d, 30, d, torch.float32)
    m = torch.tensor(MAGNITUDES * 3, device=DEV)[:, None]
    x, r, dy, dr = (v.to(dtype) for v in (m * x, m * r, m * dy, dr))
    _check_far(x, r, dy, dr, w, eps)
    _check_far(x, None, dy, None, None, eps)
    # one large element in a row of small ones
    x[:, d // 2] = 1e25
    _check_far(x, None, dy, dr, w, eps)
    u = 2 * kBf16 if dtype == torch.bfloat16 else 0.0
    for res in (None, r):
        for group in (0, 128):
            q, s, _ = muon.rms_norm_fp8(x, w, residual=res, eps=eps, group=group)
            want, _ = ref.rms_norm(f64(x), f64(w), None if res is None else f64(res), eps)
            at = ref.spread(f64(s), d, group)
            err = np.abs(f64(q.float()) * at - want)
            off = (0.0 if res is None else u) + 2.0 ** -12
            assert np.all(err <= (2.0 ** -4 * (1 + off) + off) * np.abs(want) + 2.0 ** -10 * at)
            top = np.abs(want[:, :128 if group else d]).max(axis=1)
            assert np.all(top <= 448 * (1 + off) * at[:, 0])
            # (2^-126 is the least scale, and a y below fp32's least value is 0, with scale 1)
            assert np.all((top > 224 * (1 - off) * at[:, 0]) | (top < 2.0 ** -117))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_any_magnitude_leave_the_others_as_they_are(dtype):
    # a team's later rows, by the loop or after it: the same bits
    x, r, dy, dr, w = _draw(46, 20000, 264, dtype)
    far = torch.arange(20000, device=DEV) % 97 == 5
    for res in (None, r):
        y, h = muon.rms_norm(x, w, residual=res)
        dx, _ = muon.rms_norm_backward(dy, h, w, dresidual=dr)
        q, s, _ = muon.rms_norm_fp8(x, w, residual=res)
        X = x.clone()
        X[far] *= 1e22
        Y, H = muon.rms_norm(X, w, residual=res)
        DX, _ = muon.rms_norm_backward(dy, H, w, dresidual=dr)
        Q, S, _ = muon.rms_norm_fp8(X, w, residual=res)
        for a, b in ((y, Y), (h, H), (dx, DX), (s, S), (q.view(torch.uint8), Q.view(torch.uint8))):
            assert torch.equal(a[~far], b[~far])
        want, _ = ref.rms_norm(f64(X[far]), f64(w))
        assert np.all(np.abs(f64(Y[far]) - want) <= 3 * 2.0 ** -8 * np.abs(want) + 1e-12)


def test_rows_that_are_not_finite_or_zero_without_eps():
    x, _, dy, _, _ = _draw(45, 8, 520, torch.float32)
    x[1], x[2], x[5] = 0.0, 1e25 * x[2], 1e-30 * x[5]
    x[3, 7], x[4, 9] = float("inf"), float("nan")
    y, _ = muon.rms_norm(x, eps=0.0)
    dx, _ = muon.rms_norm_backward(dy, x, eps=0.0)
    assert torch.isnan(y[[1, 4]]).all() and torch.isnan(dx[[1, 4]]).all()   # 0 / 0
    assert torch.isnan(y[3, 7]) and torch.count_nonzero(y[3]) == 1
    rest = [0, 2, 5, 6, 7]
    want, _ = ref.rms_norm(f64(x)[rest], eps=0.0)
    _within(y[rest], want, kF32 * np.abs(want), "y")
    assert torch.isfinite(dx[rest]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 520, 4104])
def test_rows_of_any_magnitude_in_place(d, dtype):
    x, r, dy, dr, w = _draw(47, 3000, d, torch.float32)
    m = torch.ones(3000, 1, device=DEV)
    m[::7], m[3::50] = 1e22, 1e-24
    x, r, dy, dr = (v.to(dtype) for v in (m * x, m * r, m * dy, dr))
    y, h = muon.rms_norm(x, w, residual=r, eps=0.0)
    dx, dw = muon.rms_norm_backward(dy, h, w, dresidual=dr, eps=0.0)
    q, s, _ = muon.rms_norm_fp8(x, w, residual=r, eps=0.0)
    assert torch.isfinite(y).all() and torch.isfinite(dx).all()
    for over in range(3):
        c = [dy.clone(), h.clone(), dr.clone()]
        got = muon.rms_norm_backward(c[0], c[1], w, dresidual=c[2], eps=0.0, dx=c[over])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    for over in range(2):
        c = [x.clone(), r.clone()]
        got = muon.rms_norm_fp8(c[0], w, residual=c[1], eps=0.0, residual_out=c[over])
        assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8))
        assert torch.equal(got[1], s) and torch.equal(got[2], h)
    assert all(torch.equal(a, b) for a, b in zip(
        muon.rms_norm_backward(dy, h, w, dresidual=dr, eps=0.0), (dx, dw)))   # the same bits again


@pytest.mark.parametrize("d", [64, 1024])
def test_a_sum_of_squares_that_leaves_the_range_by_its_rounding(d):
    # In units of u = 2^122 (d = 64): 63 elements of (1 - 0.55 2^-8)^2 u and one of 1.34 u are past 64 u =
    # 2^128; stored, the 63 are (1 - 2^-8)^2 u, and the sum is below it.  (d = 1024: u = 2^118.)
    scale = 2.0 ** (61 if d == 64 else 59)
    x = torch.full((5, d), (1 - 2.0 ** -8) * scale).bfloat16()
    r = torch.full((5, d), 0.45 * 2.0 ** -8 * scale).bfloat16()
    x[:, ::64], r[:, ::64] = 1.15625 * scale, 0.0
    wide, stored = x.double() + r.double(), (x.float() + r.float()).bfloat16().double()
    assert torch.all(wide.square().sum(1) > 2.0 ** 128)
    assert torch.all(stored.square().sum(1) < 2.0 ** 128)
    x, r = x.to(DEV), r.to(DEV)
    y, h = muon.rms_norm(x, residual=r)
    assert torch.equal(h.double().cpu(), stored)
    want, _ = ref.rms_norm(f64(x), None, f64(r))
    assert np.all(np.abs(f64(y) - want) <= 3 * kBf16 * np.abs(want))
    for group in (0, 128):
        q, s, _ = muon.rms_norm_fp8(x, residual=r, group=group)
        values = f64(q.float()) * ref.spread(f64(s), d, group)
        assert np.all(np.abs(values - want) <= (2.0 ** -4 + 3 * kBf16) * np.abs(want))


@pytest.mark.parametrize("with_r", [False, True])
def test_rows_at_the_ends_of_the_range_do_not_go_by_their_neighbours(with_r):
    t, d = 20000, 264
    x, r, _, _, w = _draw(48, t, d, torch.float32)
    k = torch.arange(t, device=DEV) % 60
    m = torch.exp2(torch.where(k < 30, -22 + k / 6, 54 + (k - 30) / 6).double())[:, None]
    x, r = ((m * v.double() / 4).bfloat16() for v in (x, r))
    r = r if with_r else None
    far = torch.arange(t, device=DEV) % 97 == 5
    X = x.clone()
    X[far] = 1e25
    for group in (None, 0, 128):
        def call(v):
            if group is None:
                y, h = muon.rms_norm(v, w, residual=r, eps=0.0)
                return y.view(torch.int16), h
            q, s, h = muon.rms_norm_fp8(v, w, residual=r, eps=0.0, group=group)
            return q.view(torch.uint8), s, h
        for a, b in zip(call(x), call(X)):
            assert torch.equal(a[~far], b[~far])
    y, _ = muon.rms_norm(x, w, residual=r, eps=0.0)
    want, _ = ref.rms_norm(f64(x), f64(w), None if r is None else f64(r), 0.0)
    s = np.abs(f64(x)) + (0 if r is None else np.abs(f64(r)))
    total = f64(x) + (0 if r is None else f64(r))
    rms = np.sqrt(np.mean(total ** 2, axis=1, keepdims=True))
    e = kF32 * (np.abs(want) + s / rms * np.abs(f64(w))) + (2 * kBf16 * np.abs(want) if with_r else 0)
    _within(y, want, e + kBf16 * (np.abs(want) + e), "y")
