"""GPU parity of the product with a weight matrix, and its gradients, with the float64 oracle.

Bounds are element by element.  Products of bf16 values are exact in fp32; a sum of K of them
in fp32, in any order and even with truncated additions, is off by at most K 2^-23 times the sum
of magnitudes.  Bias, activation and residual add a few roundings of fp32 (kF32 = 2^-20 of the
magnitudes, which covers the hardware's powers of two and reciprocals, 2^-22 each).  Every result
adds its rounding to bf16, kBf16 = 2^-8.  The activation's slope is at most 1.13 (GELU) or twice
the argument (relu^2).  The gradients go by preact as stored, which the oracle takes too, and by
dz rounded to bf16.
"""

import threading

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import block_oracle as ref

pytestmark = pytest.mark.gpu

kF32, kBf16, kAdd = 2.0 ** -20, 2.0 ** -8, 2.0 ** -23
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def _matrix(gen, rows, cols, std=1.0, pad=None):
    """Rows padded with NaN to a multiple of 8 (or by `pad` columns on both sides)."""
    left = 0 if pad is None else pad
    width = left + (cols + 7) // 8 * 8 + left
    x = torch.full((rows, width), float("nan"), dtype=torch.bfloat16)
    x[:, left:left + cols] = (std * torch.randn(rows, cols, generator=gen)).bfloat16()
    return x.to(DEV)[:, left:left + cols]


def _draw(seed, t, k, n, *, bias=True, residual=True, pad=None):
    gen = torch.Generator().manual_seed(seed)
    x, w = _matrix(gen, t, k, pad=pad), _matrix(gen, n, k, k ** -0.5, pad=pad)
    b = torch.randn(n, generator=gen).bfloat16().to(DEV) if bias else None
    r = _matrix(gen, t, n, pad=pad) if residual else None
    return x, w, b, r, _matrix(gen, t, n, pad=pad)


def _within(got, want, bound, what):
    err = np.abs(f64(got) - want) - bound - 1e-30
    assert np.all(err <= 0), (what, float(err.max()), np.argwhere(err > 0)[:4].tolist())


def _check_forward(x, w, b, r, kind, y, z):
    X, W = f64(x), f64(w)
    B, R = (None if v is None else f64(v) for v in (b, r))
    want, wz = ref.linear(X, W, B, kind, R)
    mag = np.abs(X) @ np.abs(W).T + (0 if B is None else np.abs(B))
    ez = (X.shape[1] * kAdd + kF32) * mag
    if z is not None:
        _within(z, wz, ez + kBf16 * (np.abs(wz) + ez), "preact")
    a = ref.act(wz, kind)
    lip = 1.13 if kind == "gelu" else 2 * np.abs(wz) + ez if kind == "relu2" else 1.0
    e = lip * ez + kF32 * (np.abs(a) + np.abs(wz) + (0 if R is None else np.abs(R)))
    _within(y, want, e + kBf16 * (np.abs(want) + e), "out")


def _check_backward(dy, x, w, kind, z, bias, grads):
    G, X, W = f64(dy), f64(x), f64(w)
    Z = None if z is None else f64(z)
    want = ref.linear_backward(G, X, W, kind, Z)
    dz = np.abs(G * (1.0 if kind is None else ref.slope(Z, kind)))
    # the slope in fp32: 2^-18 of |dout| (terms of up to 1.2 each in GELU's)
    e32 = 0.0 if kind is None else 2.0 ** -18 * np.abs(G) * (1 + (np.abs(Z) if kind == "relu2" else 0))
    e = e32 + (0.0 if kind is None else kBf16 * (dz + e32))
    t, n = G.shape
    for got, full, off, mag, terms in [
            (grads[0], want[0], e @ np.abs(W) if kind else 0.0, (dz + e) @ np.abs(W), n),
            (grads[1], want[1], e.T @ np.abs(X) if kind else 0.0, (dz + e).T @ np.abs(X), t)]:
        bound = off + terms * kAdd * mag
        _within(got, full, bound + kBf16 * (np.abs(full) + bound), "dx or dw")
    if bias:
        off = np.sum(e32 + t * 2.0 ** -24 * (dz + e32), axis=0)
        _within(grads[2], want[2], off + kBf16 * (np.abs(want[2]) + off), "dbias")
    else:
        assert grads[2] is None


def _check(seed, t, k, n, *, kind=None, bias=True, residual=True, pad=None):
    x, w, b, r, dy = _draw(seed, t, k, n, bias=bias, residual=residual, pad=pad)
    y = muon.linear(x, w, bias=b, activation=kind, residual=r, save_preact=kind is not None)
    y, z = y if kind else (y, None)
    grads = muon.linear_backward(dy, x, w, bias=bias, activation=kind, preact=z)
    torch.cuda.synchronize()
    _check_forward(x, w, b, r, kind, y, z)
    _check_backward(dy, x, w, kind, z, bias, grads)
    assert muon.workspace_status(None) == 0


# one token to several tiles; widths of one tile, past it, and no multiple of 8; few and many
# blocks of the contraction, so that products are split and not
@pytest.mark.parametrize("t,k,n", [
    (1, 8, 8), (1, 13, 9), (2, 520, 1000), (3, 64, 64), (4, 200, 513), (5, 13, 9), (9, 64, 64),
    (17, 512, 512), (63, 72, 136), (128, 256, 256), (129, 257, 255), (256, 64, 512),
    (257, 130, 77), (300, 520, 1000), (1003, 96, 40), (40, 2056, 24)])
@pytest.mark.parametrize("kind", [None, "relu2", "gelu"])
def test_parity(t, k, n, kind):
    _check(t + k + n, t, k, n, kind=kind)


@pytest.mark.parametrize("t", [3, 200])
@pytest.mark.parametrize("kind,bias,residual", [
    (None, False, False), (None, True, False), (None, False, True), ("relu2", False, False),
    ("relu2", True, False), ("gelu", False, True)])
def test_options(t, kind, bias, residual):
    _check(7, t, 264, 328, kind=kind, bias=bias, residual=residual)


@pytest.mark.parametrize("t,k,n", [(4000, 128, 520), (30, 4096, 640), (2600, 1032, 1544)])
def test_more_tiles_than_pairs_and_long_contractions(t, k, n):
    _check(11, t, k, n, kind="relu2")


@pytest.mark.parametrize("t", [2, 150])
def test_columns_of_wider_tensors(t):
    _check(12, t, 72, 136, kind="gelu", pad=16)


def test_outputs_given_and_their_padding():
    x, w, b, r, dy = _draw(13, 270, 130, 77)
    want, wz = muon.linear(x, w, bias=b, activation="gelu", residual=r, save_preact=True)
    wg = muon.linear_backward(dy, x, w, activation="gelu", preact=wz)

    def room(rows, cols):
        width = (cols + 40) // 8 * 8
        return torch.full((rows, width), 7.0, dtype=torch.bfloat16, device=DEV)[:, 16:16 + cols]

    y, z, dx, dw = (room(*s) for s in ((270, 77), (270, 77), (270, 130), (77, 130)))
    out = muon.linear(x, w, bias=b, activation="gelu", residual=r, preact=z, out=y)
    assert out[0] is y and out[1] is z and torch.equal(y, want) and torch.equal(z, wz)
    got = muon.linear_backward(dy, x, w, activation="gelu", preact=z, dx=dx, dweight=dw)
    assert got[0] is dx and torch.equal(dx, wg[0]) and torch.equal(dw, wg[1])
    for v in (y, z, dx, dw):
        base = v._base
        rest = torch.ones_like(base, dtype=torch.bool)
        rest[:, 16:16 + v.shape[1]] = False
        assert torch.all(base[rest] == 7.0)


@pytest.mark.parametrize("t,k", [(2, 512), (200, 64), (40, 4096)])
def test_out_may_be_the_residual(t, k):
    x, w, b, r, dy = _draw(14, t, k, 264)
    want, wz = muon.linear(x, w, bias=b, activation="relu2", residual=r, save_preact=True)
    for save in (False, True):
        c = r.clone()
        out = muon.linear(x, w, bias=b, activation="relu2", residual=c, out=c, save_preact=save)
        assert torch.equal(c, want) and (not save or torch.equal(out[1], wz))


@pytest.mark.parametrize("t,k,n", [(3, 4096, 1000), (33, 4096, 264), (1003, 520, 1000)])
def test_repeated_calls_give_equal_bits(t, k, n):
    x, w, b, r, dy = _draw(15, t, k, n)

    def call():
        y, z = muon.linear(x, w, bias=b, activation="gelu", residual=r, save_preact=True)
        return (y, z, *muon.linear_backward(dy, x, w, bias=True, activation="gelu", preact=z))

    first = call()
    for _ in range(4):
        assert all(torch.equal(a, c) for a, c in zip(first, call()))


def test_gradients_are_difference_quotients_of_the_forward():
    # loss = sum dout y, y's slope along random directions; fp32 differences of bf16 outputs are
    # too coarse, so the oracle's forward in 64 bits is differenced at the same inputs
    x, w, b, r, dy = _draw(16, 20, 40, 24)
    _, z = muon.linear(x, w, bias=b, activation="gelu", save_preact=True)
    dx, dw, db = muon.linear_backward(dy, x, w, bias=True, activation="gelu", preact=z)
    X, W, B, G = (f64(v) for v in (x, w, b, dy))
    rng = np.random.default_rng(0)
    for at, grad in ((0, dx), (1, dw), (2, db)):
        d = rng.standard_normal((X, W, B)[at].shape)

        def loss(s):
            a = [X, W, B]
            a[at] = a[at] + s * d
            return np.sum(G * ref.linear(*a, "gelu")[0])

        quotient = (loss(1e-5) - loss(-1e-5)) / 2e-5
        # roundings to bf16 of z, dz and the gradient: 3 x 2^-8 of the magnitudes, at most
        # (GELU's second derivative is below 1.2, so z's rounding moves a slope by 1.2 2^-8 |z|)
        mag = np.sum(np.abs(f64(grad) * d))
        dz = np.abs(G) * (1.13 + 1.2 * np.abs(f64(z)))
        reach = (lambda: np.abs(d) @ np.abs(W).T, lambda: np.abs(X) @ np.abs(d).T,
                 lambda: np.abs(d)[None, :])[at]()
        assert abs(quotient - np.sum(f64(grad) * d)) <= kBf16 * (mag + 2 * np.sum(dz * reach))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("t", [4, 300])
def test_values_that_are_not_finite_stay_in_their_rows(t, value):
    x, w, b, r, dy = _draw(17, t, 136, 200)
    x[2, 5] = value
    y, z = muon.linear(x, w, bias=b, activation="relu2", residual=r, save_preact=True)
    rows = torch.arange(t, device=DEV) != 2
    assert torch.isfinite(y[rows]).all() and not torch.isfinite(z[2]).any()
    with np.errstate(all="ignore"):
        want, wz = ref.linear(f64(x), f64(w), f64(b), "relu2", f64(r))
    assert np.array_equal(np.isnan(f64(y[2])), np.isnan(want[2]))
    x[2, 5] = 0.0
    dy[2, 7] = value
    dx, dw, _ = muon.linear_backward(dy, x, w)
    assert torch.isfinite(dx[rows]).all() and not torch.isfinite(dx[2]).any()
    cols = torch.arange(200, device=DEV) != 7
    assert torch.isfinite(dw[cols]).all()


@pytest.mark.parametrize("t", [4, 40])
def test_activations_at_the_ends_of_the_type(t):
    # z takes given values: x = e_0, w[:, 0] = values
    values = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 1e10, -1e10, 1e30, -1e30, 3e38, -3e38,
              float("inf"), float("-inf"), float("nan"), 0.5]
    x = torch.zeros(t, 16, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1.0
    w = torch.zeros(16, 16, dtype=torch.bfloat16, device=DEV)
    w[:, 0] = torch.tensor(values).bfloat16()
    x[:, 1:] = 0.0
    dy = torch.ones(t, 16, dtype=torch.bfloat16, device=DEV)
    for kind in ("relu2", "gelu"):
        y, z = muon.linear(x, w, activation=kind, save_preact=True)
        Z = f64(w[:, 0])
        assert np.array_equal(f64(z[0]), Z, equal_nan=True)
        with np.errstate(all="ignore"):
            want = f64(torch.from_numpy(ref.act(Z, kind)).float().bfloat16())
        got = f64(y[0])
        assert np.array_equal(np.isnan(got), np.isnan(want)), kind
        fin = np.isfinite(want)
        assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
        # tiny results may be flushed to 0
        assert np.all(np.abs(got[fin] - want[fin]) <= 2 * kBf16 * np.abs(want[fin]) + 1e-37)
        _, _, db = muon.linear_backward(dy, x, w, bias=True, activation=kind, preact=z)
        s = f64(db) / t
        finite = np.abs(Z) <= 1e30
        zs = np.clip(Z[finite], -40, 40) if kind == "gelu" else Z[finite]
        slope = ref.slope(zs, kind)
        assert np.all(np.abs(s[finite] - slope) <= 2 * kBf16 * np.abs(slope) + 2.0 ** -17)
        assert np.isnan(s[14])


def test_zero_tokens():
    x, w, b, r, dy = _draw(18, 4, 130, 77)
    before = muon.kernel_launch_count()
    y, z = muon.linear(x[:0], w, bias=b, activation="gelu", residual=r[:0], save_preact=True)
    assert y.shape == z.shape == (0, 77)
    dx, dw, db = muon.linear_backward(dy[:0], x[:0], w, bias=True, activation="gelu", preact=z)
    assert dx.shape == (0, 130) and torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0
    assert dw.shape == (77, 130) and muon.kernel_launch_count() == before


@pytest.mark.parametrize("t,k", [(3, 512), (1003, 520), (40, 4096)])
def test_captured_and_replayed_beside_eager_calls(t, k):
    x, w, b, r, dy = _draw(19, t, k, 264)
    x2, w2, b2, r2, dy2 = _draw(20, 2 * t, k, 264)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(x, w, b, r, dy):
        y, z = muon.linear(x, w, bias=b, activation="gelu", residual=r, save_preact=True)
        return (y, z, *muon.linear_backward(dy, x, w, bias=True, activation="gelu", preact=z))

    want, want2 = call(x, w, b, r, dy), call(x2, w2, b2, r2, dy2)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(call(x, w, b, r, dy))
        graphs.append(g)
    torch.cuda.synchronize()
    for order in ((0, 1), (1, 0, 1)):
        for o in outs:
            for v in o:
                v.fill_(3.0)
        torch.cuda.synchronize()
        eager = call(x2, w2, b2, r2, dy2)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, c) for a, c in zip(o, want))
        assert all(torch.equal(a, c) for a, c in zip(eager, want2))


def test_streams_and_threads():
    cases = [_draw(21 + i, t, 1032, 264) for i, t in enumerate((9, 40, 300, 3))]
    want = [muon.linear(x, w, bias=b, residual=r) for x, w, b, r, _ in cases]
    wg = [muon.linear_backward(dy, x, w, bias=True) for x, w, b, r, dy in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    bad = []

    def work(i, stream):
        x, w, b, r, dy = cases[i]
        for _ in range(20):
            y = muon.linear(x, w, bias=b, residual=r, stream=stream)
            g = muon.linear_backward(dy, x, w, bias=True, stream=stream)
            (stream or torch.cuda.current_stream()).synchronize()
            if not torch.equal(y, want[i]) or not all(torch.equal(a, c) for a, c in zip(g, wg[i])):
                bad.append(i)

    for shared in (False, True):                # a stream each, then all on the default stream
        threads = [threading.Thread(target=work, args=(i, None if shared else streams[i]))
                   for i in range(len(cases))]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        assert not bad


@pytest.mark.parametrize("t,k", [(3, 512), (33, 4096), (1003, 264), (300, 11008)])
def test_after_a_failure_nothing_is_stored_until_the_word_is_cleared(t, k):
    x, w, b, r, dy = _draw(30, t, k, 264)
    ws = muon.Workspace(muon.linear_workspace_bytes(t, k, 264))
    want, z = muon.linear(x, w, bias=b, activation="gelu", residual=r, save_preact=True)
    wg = muon.linear_backward(dy, x, w, activation="gelu", preact=z)
    muon.selftest_wait_timeout(ws, limit_us=1000)
    y, z2, dx, dw = (torch.full_like(v.contiguous(), 3.0) for v in (want, z, wg[0], wg[1]))
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    muon.linear(x, w, bias=b, activation="gelu", residual=r, preact=z2, out=y, workspace=ws)
    muon.linear_backward(dy, x, w, activation="gelu", preact=z, dx=dx, dweight=dw, workspace=ws)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 100.0      # no wait runs out
    assert all(torch.all(v == 3.0) for v in (y, z2, dx, dw))
    assert muon.workspace_status(ws, clear=True) == 4
    muon.linear(x, w, bias=b, activation="gelu", residual=r, preact=z2, out=y, workspace=ws)
    muon.linear_backward(dy, x, w, activation="gelu", preact=z, dx=dx, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    assert muon.workspace_status(ws) == 0
    assert all(torch.equal(a, c) for a, c in zip((y, z2, dx, dw), (want, z, wg[0], wg[1])))


def test_refusals():
    x, w, b, r, dy = _draw(31, 20, 64, 72)
    for bad, exc in [((x.float(), w), TypeError), ((x, w.half()), TypeError),
                     ((x, w[:, :32]), ValueError), ((x[0], w), ValueError), ((x, w[0]), ValueError),
                     ((x.t(), w), ValueError), ((x, w.cpu()), ValueError)]:
        with pytest.raises(exc):
            muon.linear(*bad)
    for kw, exc in [(dict(bias=b.float()), TypeError), (dict(bias=b[:8]), ValueError),
                    (dict(residual=x), ValueError), (dict(residual=r.float()), TypeError),
                    (dict(out=x), ValueError), (dict(preact=x), ValueError),
                    (dict(activation="tanh"), ValueError)]:
        with pytest.raises(exc):
            muon.linear(x, w, **kw)
    with pytest.raises(ValueError):             # an activation's gradient needs preact
        muon.linear_backward(dy, x, w, activation="gelu")
    with pytest.raises(ValueError):
        muon.linear_backward(dy[:, :8], x, w)
    odd = torch.empty(20, 65, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(muon.MuonError):         # rows that are not 16-byte aligned
        muon.linear(odd[:, :64], w)
    with pytest.raises(muon.MuonError):
        muon.linear(odd[:, 1:], torch.zeros(72, 64, dtype=torch.bfloat16, device=DEV))
    square = torch.zeros(20, 20 * 4, dtype=torch.bfloat16, device=DEV)[:, :64]
    with pytest.raises(muon.MuonError):         # out over x
        muon.linear(square, torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV), out=square)
    for v in (x, w, b, r):
        v.requires_grad_(True)
        with pytest.raises(ValueError, match="linear_backward"):
            muon.linear(x, w, bias=b, residual=r)
        with torch.no_grad():
            muon.linear(x, w, bias=b, residual=r)
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


@pytest.mark.parametrize("t,k,n", [(4, 264, 136), (70, 264, 131), (40, 1032, 264)])
def test_offsets_past_32_bits(t, k, n):
    x, w, b, r, dy = _draw(41, t, k, n)
    want = muon.linear(x, w, bias=b, activation="gelu", residual=r, save_preact=True)
    wg = muon.linear_backward(dy, x, w, bias=True, activation="gelu", preact=want[1])
    X, R, DY, O, Z, DX, W, DW = (_spread(v, e) for v, e in (
        (x, False), (r, False), (dy, False), (r, True), (r, True), (x, True), (w, False), (w, True)))
    muon.linear(X, W, bias=b, activation="gelu", residual=R, preact=Z, out=O)
    got = muon.linear_backward(DY, X, W, bias=True, activation="gelu", preact=Z, dx=DX, dweight=DW)
    assert torch.equal(O, want[0]) and torch.equal(Z, want[1])
    assert all(torch.equal(a, c) for a, c in zip(got, wg))


@pytest.mark.parametrize("t", [0, 3, 300])
@pytest.mark.parametrize("k", [13, 130, 136])
def test_weight_gradients_of_any_width_go_to_clipping_and_the_optimizers(t, k):
    x, w, b, r, dy = _draw(50, t, k, 77)
    given = torch.full((77, (k + 7) // 8 * 8), 5.0, dtype=torch.bfloat16, device=DEV)[:, :k]
    _, want, _ = muon.linear_backward(dy, x, w, dweight=given)
    assert want is given
    _, dw, db = muon.linear_backward(dy, x, w, bias=True)
    assert dw.is_contiguous() and torch.equal(dw, want)
    norm = float(muon.clip_grad_norm([dw, db], 1.0))
    sq = f64(want) ** 2
    assert abs(norm - np.sqrt(sq.sum() + (f64(dy).sum(0) ** 2).sum())) <= 2.0 ** -7 * norm + 1e-6
    p, m = (torch.zeros(77, k, device=DEV) for _ in range(2))
    muon.step(p, dw, m, momentum=0.9, lr=0.02, weight_decay=0.0)
    muon.adam_step([(p, dw, m, torch.zeros_like(p))], 1)
    torch.cuda.synchronize()
    assert torch.isfinite(p).all()


@pytest.mark.parametrize("t", [1, 3, 300])
@pytest.mark.parametrize("kind", [None, "gelu"])
def test_gradients_of_rows_that_begin_anywhere(t, kind):
    x, w, b, r, dy = _draw(51, t, 136, 257)
    y, z = muon.linear(x, w, bias=b, activation=kind, save_preact=True)
    assert y.stride() == (264, 1)
    z = z if kind else None
    want = muon.linear_backward(dy, x, w, bias=True, activation=kind, preact=z)
    wide = torch.full((t, 261), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 3:260] = dy
    for rows in (dy.contiguous(), wide[:, 3:260]):     # odd strides; an odd address
        got = muon.linear_backward(rows, x, w, bias=True, activation=kind, preact=z)
        assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    rows = dy.contiguous()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = muon.linear_backward(rows, x, w, bias=True, activation=kind, preact=z)
    for v in got:
        v.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_an_output_head_whose_width_is_odd():
    # logits, the gradient as torch makes it of them, and the head's gradients
    t, d, n = 200, 72, 1001
    x, w, _, _, _ = _draw(52, t, d, n, bias=False, residual=False)
    targets = torch.randint(0, n, (t,), generator=torch.Generator().manual_seed(1)).to(DEV)
    logits = muon.linear(x, w)
    g = torch.softmax(logits.float(), 1)
    g[torch.arange(t, device=DEV), targets] -= 1
    g = (g / t).bfloat16()
    assert g.stride() == (n, 1)
    dx, dw, _ = muon.linear_backward(g, x, w)
    _check_backward(g, x, w, None, None, False, (dx, dw, None))
    muon.clip_grad_norm([dw], 1.0)


def test_refused_rows_are_named():
    x, w, b, r, dy = _draw(53, 20, 130, 77, pad=None)
    for kw, name in ((dict(residual=r.contiguous()), "residual"),
                     (dict(out=torch.empty(20, 77, dtype=x.dtype, device=DEV)), "out")):
        with pytest.raises(muon.MuonError, match=f"rows of {name} "):
            muon.linear(x, w, **kw)
    with pytest.raises(muon.MuonError, match="rows of weight "):
        muon.linear(x, w.contiguous())
    with pytest.raises(muon.MuonError, match="rows of x "):
        muon.linear_backward(dy, x.contiguous(), w)
    with pytest.raises(muon.MuonError, match="rows of dweight "):
        muon.linear_backward(dy, x, w, dweight=torch.empty(77, 130, dtype=x.dtype, device=DEV))
