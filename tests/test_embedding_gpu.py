"""GPU parity of the embedding and its table's gradient with the float64 oracle.

The lookup is one product and one rounding.  A row of the gradient is a sum of its n tokens' rows in
fp32, in chains of at most 32 and then of the pieces: off by at most (n + 2) 2^-24 of the sum of
magnitudes, plus the rounding of a bf16 output, 2^-8.
"""

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import block_oracle as ref

pytestmark = pytest.mark.gpu

kBf16 = 2.0 ** -8
DEV = "cuda"


def f64(t):
    return t.detach().double().cpu().numpy()


def _draw(seed, t, rows, dim, *, dtype=torch.bfloat16, table=torch.float32, ids=torch.int64,
          skew=True):
    gen = torch.Generator().manual_seed(seed)
    r = torch.rand(t, generator=gen)
    i = (rows * (r ** 4 if skew else r)).long().clamp_max(rows - 1)
    tab = torch.randn(rows, dim, generator=gen).to(table).to(DEV)
    dy = torch.randn(t, dim, generator=gen).to(dtype).to(DEV)
    return i.to(ids).to(DEV), tab, dy


def _check_gradient(ids, dy, rows, scale, got):
    I, G = ids.cpu().numpy(), f64(dy)
    want = ref.embedding_backward(G, I, rows, scale)
    mag = ref.embedding_backward(np.abs(G), I, rows, abs(scale))
    n = np.bincount(I[(I >= 0) & (I < rows)], minlength=rows)[:, None]
    e = (n + 2) * 2.0 ** -24 * mag
    u = kBf16 if got.dtype == torch.bfloat16 else 0.0
    err = np.abs(f64(got) - want) - (e + u * (np.abs(want) + e))
    assert np.all(err <= 0), float(err.max())


# one token; a chunk of sorted positions and past it; more tokens than a batch of the sort
# holds (65536); one to three passes of digits; one row that takes all tokens
@pytest.mark.parametrize("t,rows,dim", [
    (1, 1, 8), (1, 300, 16), (31, 5, 264), (32, 5, 8), (33, 5, 256), (64, 1, 520), (300, 1, 8),
    (1000, 1024, 72), (1000, 1025, 72), (4099, 257, 64), (5000, 50257, 24), (9000, 3, 1032),
    (70001, 700, 8), (40000, 1100000, 8), (65536, 2, 16), (65537, 40, 16)])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_parity(t, rows, dim, ids):
    i, tab, dy = _draw(t + rows, t, rows, dim, ids=ids)
    y = muon.embedding(i, tab, scale=3.0)
    want = ref.embedding(i.cpu().numpy(), f64(tab), 3.0)
    assert np.all(np.abs(f64(y) - want) <= (kBf16 + 2.0 ** -22) * np.abs(want))
    _check_gradient(i, dy, rows, 3.0, muon.embedding_backward(dy, i, rows, scale=3.0))
    assert muon.workspace_status(None) == 0


@pytest.mark.parametrize("table", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_types(table, out):
    i, tab, dy = _draw(1, 500, 90, 136, dtype=out, table=table)
    y = muon.embedding(i, tab, scale=-1.5, dtype=out)
    assert y.dtype == out
    want = ref.embedding(i.cpu().numpy(), f64(tab), -1.5)
    u = kBf16 if out == torch.bfloat16 else 0.0
    assert np.all(np.abs(f64(y) - want) <= (u + 2.0 ** -23) * np.abs(want))
    _check_gradient(i, dy, 90, -1.5, muon.embedding_backward(dy, i, 90, scale=-1.5, dtype=table))
    if table == out:
        assert torch.equal(muon.embedding(i, tab, dtype=out), tab[i])


@pytest.mark.parametrize("t", [7, 40, 3000, 70000])
@pytest.mark.parametrize("share", [0.3, 1.0])
def test_ids_outside_the_table(t, share):
    i, tab, dy = _draw(2, t, 50, 16)
    gen = torch.Generator().manual_seed(3)
    bad = (torch.rand(t, generator=gen) < share).to(DEV)
    far = torch.tensor([-1, 50, 2 ** 31, 2 ** 32 + 3, -2 ** 40, 51], device=DEV)
    i = torch.where(bad, far[torch.arange(t, device=DEV) % 6], i)
    y = muon.embedding(i, tab)
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    dy[bad] = float("nan")                      # rows that no sum may read
    dy32 = dy.clone()
    dy32[bad] = 0.0
    got = muon.embedding_backward(dy, i, 50)
    _check_gradient(i, dy32, 50, 1.0, got)
    assert torch.equal(got, muon.embedding_backward(dy32, i, 50))


def test_strided_rows_and_outputs_given():
    i, tab, dy = _draw(4, 400, 60, 72)
    wide = torch.full((60, 88), float("nan"), device=DEV)
    wide[:, 8:80] = tab
    out = torch.full((400, 96), 7.0, dtype=torch.bfloat16, device=DEV)
    y = muon.embedding(i, wide[:, 8:80], out=out[:, 16:88])
    assert torch.equal(y, muon.embedding(i, tab)) and y.data_ptr() == out[:, 16:88].data_ptr()
    g = torch.full((400, 88), float("nan"), dtype=torch.bfloat16, device=DEV)
    g[:, 8:80] = dy
    grad = torch.full((60, 80), 7.0, device=DEV)
    got = muon.embedding_backward(g[:, 8:80], i, 60, out=grad[:, 4:76])
    assert torch.equal(got, muon.embedding_backward(dy, i, 60))
    for full, cols in ((out, (slice(0, 16), slice(88, 96))), (grad, (slice(0, 4), slice(76, 80)))):
        for c in cols:
            assert torch.all(full[:, c] == 7.0)


def test_a_token_that_is_not_finite_reaches_its_row_alone():
    i, tab, dy = _draw(5, 2000, 30, 64)
    dy[11, 3] = float("inf")
    g = muon.embedding_backward(dy, i, 30)
    bad = ~torch.isfinite(g)
    assert bad.sum() == 1 and bad[i[11], 3]


def test_gradient_is_the_difference_quotient_of_the_forward_kernel():
    i, tab, dy = _draw(6, 300, 40, 24, dtype=torch.float32)
    d = torch.randn(40, 24, generator=torch.Generator().manual_seed(7)).to(DEV)
    g = muon.embedding_backward(dy, i, 40, scale=2.0)

    def loss(s):
        return (f64(muon.embedding(i, tab + s * d, scale=2.0, dtype=torch.float32)) * f64(dy)).sum()

    # linear: fp32 rounding alone, 2^-23 of about 4 a term, 7200 terms at random, over 2 h
    h = 0.5
    assert abs((loss(h) - loss(-h)) / (2 * h) - (f64(g) * f64(d)).sum()) <= 2.0 ** -21 * 85 * 8


def test_repeated_captured_streams_and_status():
    cases = [_draw(8, t, 700, 264) for t in (3000, 20)]
    want = [muon.embedding_backward(dy, i, 700) for i, _, dy in cases]
    for _ in range(4):
        for (i, _, dy), w in zip(cases, want):
            assert torch.equal(muon.embedding_backward(dy, i, 700), w)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, tab, dy in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append((muon.embedding(i, tab), muon.embedding_backward(dy, i, 700)))
        graphs.append(g)
    for order in ((0, 1), (1, 0)):
        for o in outs:
            for v in o:
                v.fill_(3.0)
        eager = muon.embedding_backward(cases[0][2], cases[0][0], 700)
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        for (i, tab, _), o, w in zip(cases, outs, want):
            assert torch.equal(o[0], muon.embedding(i, tab)) and torch.equal(o[1], w)
    got = [muon.embedding_backward(dy, i, 700, stream=stream) for i, _, dy in cases]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = muon.Workspace(muon.embedding_workspace_bytes(3000, 264))
    muon.selftest_wait_timeout(ws, limit_us=1000)
    grad = torch.full((700, 264), 3.0, device=DEV)
    i, _, dy = cases[0]
    muon.embedding_backward(dy, i, 700, out=grad, workspace=ws)
    assert muon.workspace_status(ws, clear=True) == 4 and torch.all(grad == 3.0)
    muon.embedding_backward(dy, i, 700, out=grad, workspace=ws)
    assert muon.workspace_status(ws) == 0 and torch.equal(grad, want[0])


def test_a_workspace_shared_with_the_other_operators():
    # the status block of a workspace holds the tickets of another operator's sums
    i, tab, dy = _draw(9, 3000, 700, 64)
    q = torch.randn(200, 4, 64, device=DEV).bfloat16()
    cos, sin = muon.rope_tables(200, 64)
    w = torch.ones(64, device=DEV)
    ws = muon.Workspace(max(muon.embedding_workspace_bytes(3000, 64),
                            muon.norm_rope_workspace_bytes(64), muon.rms_norm_workspace_bytes(64)))
    want = muon.qk_norm_rope_backward(q, q, q, q, cos, sin, q_weight=w, k_weight=w)
    for _ in range(2):
        g = muon.embedding_backward(dy, i, 700, workspace=ws)
        got = muon.qk_norm_rope_backward(q, q, q, q, cos, sin, q_weight=w, k_weight=w, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.equal(g, muon.embedding_backward(dy, i, 700))
    assert muon.workspace_status(ws) == 0 and torch.count_nonzero(ws.tensor[:256]) == 0


def test_zero_tokens():
    i, tab, dy = _draw(10, 4, 60, 64)
    before = muon.kernel_launch_count()
    assert muon.embedding(i[:0], tab).shape == (0, 64)
    wide = torch.full((60, 72), 7.0, device=DEV)
    g = muon.embedding_backward(dy[:0], i[:0], 60, out=wide[:, :64])
    assert torch.count_nonzero(g) == 0 and torch.all(wide[:, 64:] == 7.0)
    assert muon.kernel_launch_count() == before


def test_refusals():
    i, tab, dy = _draw(11, 20, 60, 64)
    for args, kw, exc in [((i.float(), tab), {}, TypeError), ((i[None], tab), {}, ValueError),
                          ((i[::2], tab), {}, ValueError), ((i, tab.half()), {}, TypeError),
                          ((i, tab[0]), {}, ValueError), ((i.cpu(), tab), {}, ValueError),
                          ((i, tab.t()), {}, ValueError), ((i, tab), dict(dtype=torch.half), TypeError),
                          ((i, tab), dict(out=dy[:5]), ValueError)]:
        with pytest.raises(exc):
            muon.embedding(*args, **kw)
    for args, kw, exc in [((dy, i[:5], 60), {}, ValueError), ((dy.half(), i, 60), {}, TypeError),
                          ((dy[0], i, 60), {}, ValueError), ((dy, i.cpu(), 60), {}, ValueError),
                          ((dy, i, 60), dict(out=tab[:5]), ValueError)]:
        with pytest.raises(exc):
            muon.embedding_backward(*args, **kw)
    with pytest.raises(muon.MuonError):
        muon.embedding(i, tab[:, :60])
    with pytest.raises(muon.MuonError):
        muon.embedding_backward(dy, i, 0)
    with pytest.raises(muon.MuonError):                 # out over the table
        muon.embedding(i, tab, out=tab[:20])
    with pytest.raises(muon.MuonError):
        muon.embedding_backward(tab[:20], i, 60, out=tab)
    tab.requires_grad_(True)
    with pytest.raises(ValueError, match="embedding_backward"):
        muon.embedding(i, tab)


def test_offsets_past_32_bits():
    rows, dim = 270_000, 8192                   # 2.2 10^9 elements
    table = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV)
    table.view(torch.int16).random_(0x1000, 0x3f80)
    gen = torch.Generator().manual_seed(45)
    ids = torch.cat((torch.tensor([0, rows - 1, rows - 1, rows, 262_144]),
                     torch.randint(0, rows, (95,), generator=gen))).to(DEV)
    out = muon.embedding(ids, table, scale=0.5)
    ok = ids < rows
    assert torch.equal(out[ok], table[ids[ok]] * 0.5) and torch.isnan(out[~ok]).all()
    dout = torch.randn(len(ids), dim, generator=gen).bfloat16().to(DEV)
    for dtype in (torch.bfloat16, torch.float32):
        d = muon.embedding_backward(dout, ids, rows, dtype=dtype)
        assert torch.equal(d[rows - 1].float(), (dout[1].float() + dout[2].float()).to(dtype).float())
        d[ids[ok]] = 0
        assert not d.any()
        del d


def test_many_tokens_past_the_registers_of_the_sort():
    # more items a warp than are kept between count and placing, three passes of the sort
    t, rows, dim = 2_200_000, 3_000_000, 8
    ids = torch.randint(0, rows, (t,), device=DEV)
    ids[::20] = 7
    dout = torch.randint(-4, 5, (t, dim), device=DEV).bfloat16()
    want = torch.zeros(rows, dim, device=DEV).index_add_(0, ids, dout.float())   # (whole numbers)
    assert torch.equal(muon.embedding_backward(dout, ids, rows), want)
