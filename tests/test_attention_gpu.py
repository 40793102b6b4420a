"""GPU parity of attention and its gradients with the float64 oracle.

Bounds are element by element, from the roundings the kernels make (u = 2^-8: rounding to bf16;
sums and softmax in fp32, whose errors c = 2^-16 of the magnitudes entering a sum covers):
  a weight p is off by Ep p,  Ep = c (1 + scale |q| . |k|)       (error of its exponent)
  out:  u |out| + (1 + u) (u + Ep) sum p |v|                     (p rounded for the product)
  dv:   u |dv|  + (1 + u) (u + Ep) sum p |dout|
  ds = p (dp - delta) is off by Ep |ds| + (c + u) p (|dout| . |v| + |dout| . |out|), the u for
  the bf16 out that delta may come from, then rounded;
  dq, dk: u of the result, and those errors times scale |k|, scale |q|
The oracle takes the same bf16 inputs, and for the gradients its own out and the lse handed to
the kernel.
Each result's Frobenius error is also held to 1e-2 (rounding error rms 2^-8 / sqrt 3 = 2.3e-3 for
each of at most three roundings on a result's way, with room for cancellation).
"""

import threading

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import attention_oracle as ref

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -8, 2.0 ** -16
REL = 1e-2


def f64(t):
    return t.detach().double().cpu().numpy()


def _draw(seed, t, hq, hk, d, *, fused=True, sharp=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(t, hq + 2 * hk, d, generator=gen)
    x[:, :hq] *= sharp
    x = x.to(torch.bfloat16).cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if not fused:
        q, k, v = (y.contiguous() for y in (q, k, v))
    do = torch.randn(t, hq, d, generator=gen).to(torch.bfloat16).cuda()
    return q, k, v, do


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()


def _rel(got, want):
    n = np.linalg.norm(want)
    return np.linalg.norm(got - want) / n if n else np.linalg.norm(got)


def _magnitudes(q, k, v, do, out, lse, cu, scale):
    """Bounds of the errors of out, lse, dq, dk, dv before their own rounding."""
    t, hq, d = q.shape
    group = hq // k.shape[1]
    b_out, b_lse = np.zeros_like(q), np.zeros((hq, t))
    b_dq, b_dk, b_dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(k)
    for a, b in ref.spans(cu, t):
        vis = np.tril(np.ones((b - a, b - a), dtype=bool))
        for h in range(hq):
            g = h // group
            qq, kk, vv, dd, oo = q[a:b, h], k[a:b, g], v[a:b, g], do[a:b, h], out[a:b, h]
            p = np.where(vis, np.exp(np.where(vis, scale * (qq @ kk.T), -np.inf)
                                     - lse[h, a:b, None]), 0)
            size = scale * (np.abs(qq) @ np.abs(kk).T)
            ep = C * (1 + np.max(np.where(vis, size, 0), axis=1, keepdims=True))
            b_lse[h, a:b] = ep[:, 0]
            b_out[a:b, h] = (p * (U + ep)) @ np.abs(vv)
            b_dv[a:b, g] += (p * (U + ep)).T @ np.abs(dd)
            delta = np.sum(dd * oo, 1, keepdims=True)
            out_size = np.sum(np.abs(dd * oo), 1, keepdims=True)
            e = p * (C * (np.abs(dd) @ np.abs(vv).T) + (C + U) * out_size)
            e += (U + ep) * p * np.abs(dd @ vv.T - delta)
            b_dq[a:b, h] = scale * (e @ np.abs(kk))
            b_dk[a:b, g] += scale * (e.T @ np.abs(qq))
    return b_out, b_lse, b_dq, b_dk, b_dv


def _check(q, k, v, do, lengths=None, scale=None, stream=None, cu=None):
    cu = _cu(lengths) if lengths is not None else cu
    out, lse = muon.attention(q, k, v, cu, scale=scale, stream=stream)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu, scale=scale, stream=stream)
    torch.cuda.synchronize()
    Q, K, V, D = (f64(x) for x in (q, k, v, do))
    c = None if cu is None else cu.cpu().numpy()
    scale = q.shape[2] ** -0.5 if scale is None else scale
    r_out, r_lse = ref.attention(Q, K, V, c, scale)
    b = _magnitudes(Q, K, V, D, r_out, f64(lse), c, scale)
    r_grads = ref.attention_backward(D, Q, K, V, r_out, f64(lse), c, scale)
    L = f64(lse)
    assert np.array_equal(np.isneginf(L), np.isneginf(r_lse))
    fin = np.isfinite(r_lse)
    assert np.all(np.abs(L - r_lse, where=fin, out=np.zeros_like(L)) <= b[1] + 1e-30)
    for name, got, want, bound in [("out", out, r_out, b[0]),
                                   *zip(("dq", "dk", "dv"), grads, r_grads, b[2:])]:
        G = f64(got)
        err = np.abs(G - want) - (U * np.abs(want) + (1 + U) * bound + 1e-30)
        assert np.all(err <= 0), (name, float(err.max()))
        # (a single query's dq and dk are exact zeros up to cancellation)
        assert np.linalg.norm(G - want) <= REL * np.linalg.norm(want) + np.linalg.norm(
            (1 + U) * bound) * U, (name, _rel(G, want))
    return out, lse, grads


LENGTHS = [[1], [2], [64], [127], [128], [129], [255], [257], [385], [1] * 7,
           [0, 1, 0, 200, 0], [3, 200, 77, 1, 130], [100, 28, 128, 129], [31, 33, 64, 5, 250]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=[",".join(map(str, x)) for x in LENGTHS])
@pytest.mark.parametrize("hq,hk,d", [(2, 1, 64), (2, 2, 128)])
def test_parity_at_tile_edges(lengths, hq, hk, d):
    _check(*_draw(sum(lengths) + d, sum(lengths), hq, hk, d), lengths)


@pytest.mark.parametrize("hq,hk,d", [(8, 4, 64), (6, 6, 64), (4, 1, 128), (5, 5, 80), (3, 1, 96),
                                     (2, 1, 8), (4, 2, 24), (2, 2, 72), (2, 1, 120), (12, 2, 32)])
def test_parity_over_heads(hq, hk, d):
    _check(*_draw(d, 300, hq, hk, d, fused=d != 96), [77, 0, 150, 73])


@pytest.mark.parametrize("lengths", [[1], [2], [3], [2, 1], [5, 1, 2, 17], [128, 60, 3, 65],
                                     [125, 0, 3, 1, 1, 2, 50]],
                         ids=lambda x: ",".join(map(str, x)))
@pytest.mark.parametrize("hq,hk,d", [(24, 8, 64), (4, 2, 128), (3, 1, 80), (8, 8, 32)])
def test_short_sequences_round_dq_and_dk_once(lengths, hq, hk, d):
    # Sequences inside a tile of 128 tokens: delta is sum p dp of the block, off by the errors of
    # p and dp only, and ds goes into the products as two bf16 (U^2 = C); what is left of the
    # bounds above is the result's own rounding and terms of C.
    q, k, v, do = _draw(40 + sum(lengths) + d, sum(lengths), hq, hk, d)
    cu = _cu(lengths)
    out, lse = muon.attention(q, k, v, cu)
    got = muon.attention_backward(do, q, k, v, out, lse, cu)[:2]
    Q, K, V, D = (f64(x) for x in (q, k, v, do))
    c, scale = cu.cpu().numpy(), d ** -0.5
    r_out, _ = ref.attention(Q, K, V, c)
    want = ref.attention_backward(D, Q, K, V, r_out, f64(lse), c)[:2]
    bound = [np.zeros_like(Q), np.zeros_like(K)]
    for a, b in ref.spans(c, sum(lengths)):
        assert a // 128 == (b - 1) // 128
        vis = np.tril(np.ones((b - a, b - a), dtype=bool))
        for h in range(hq):
            g = h // (hq // hk)
            qq, kk, vv, dd = Q[a:b, h], K[a:b, g], V[a:b, g], D[a:b, h]
            s = scale * (qq @ kk.T)
            p = np.where(vis, np.exp(np.where(vis, s, -np.inf) - f64(lse)[h, a:b, None]), 0)
            size = np.where(vis, scale * (np.abs(qq) @ np.abs(kk).T), 0)
            ep = C * (1 + size.max(1, keepdims=True))
            dp = np.abs(dd) @ np.abs(vv).T
            # |dp - delta| <= dp + sum p dp; delta is off by 3 ep of its terms at most
            mean = np.sum(p * dp, 1, keepdims=True)
            e = p * (C * dp + 3 * (C + ep) * mean) + (C + ep) * p * (dp + mean)
            bound[0][a:b, h] = scale * (e @ np.abs(kk))
            bound[1][a:b, g] += scale * (e.T @ np.abs(qq))
    for name, x, w, e in zip(("dq", "dk"), got, want, bound):
        err = np.abs(f64(x) - w) - (U * np.abs(w) + (1 + U) * e + 1e-30)
        assert np.all(err <= 0), (name, float(err.max()))


@pytest.mark.parametrize("lengths", [[900, 700, 124], [1000, 10, 1100], [130, 1700, 300]],
                         ids=lambda x: ",".join(map(str, x)))
@pytest.mark.parametrize("hq,hk,d", [(80, 20, 64), (80, 40, 16), (80, 20, 128)])
def test_parity_of_two_tiles_with_different_walks(lengths, hq, hk, d):
    # many heads: a block takes two tiles, of which one may begin its walk blocks later
    q, k, v, do = _draw(50 + d, sum(lengths), hq, hk, d)
    cu = _cu(lengths)
    out, lse = muon.attention(q, k, v, cu)
    some = [0, hq - 1]
    g = [h // (hq // hk) for h in some]
    Q, K, V = f64(q[:, some]), f64(k[:, g]), f64(v[:, g])
    r_out, r_lse = ref.attention(Q, K, V, cu.cpu().numpy())
    b_out, b_lse, *_ = _magnitudes(Q, K, V, np.zeros_like(Q), r_out, r_lse, cu.cpu().numpy(),
                                   d ** -0.5)
    err = np.abs(f64(out[:, some]) - r_out) - (U * np.abs(r_out) + (1 + U) * b_out + 1e-30)
    assert np.all(err <= 0), float(err.max())
    assert np.all(np.abs(f64(lse[some]) - r_lse) <= b_lse + 1e-30)


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (2, 1, 128)])
def test_parity_on_longer_sequences(hq, hk, d):
    _check(*_draw(1, 1500, hq, hk, d), [1100, 400])
    _check(*_draw(2, 1030, hq, hk, d))               # no offsets: one sequence


@pytest.mark.parametrize("sharp,scale", [(8.0, None), (1.0, 2.0), (1.0, 1e-3), (30.0, None)])
def test_parity_with_sharp_and_flat_weights(sharp, scale):
    # scores far apart: the running maximum moves by more than a rescale's threshold
    _check(*_draw(3, 700, 2, 1, 64, sharp=sharp), [500, 200], scale=scale)


def test_parity_over_more_than_one_wave_of_blocks():
    # documents of different lengths: blocks take the tiles by their work
    _check(*_draw(30, 1290, 40, 20, 16), [300, 7, 0, 511, 130, 1, 341])
    # more tiles than are ranked in the backward kernels
    _check(*_draw(31, 40030, 1, 1, 8), [100] * 400 + [30])


def test_growing_scores_move_the_maximum_in_every_block():
    q, k, v, do = _draw(4, 900, 2, 1, 64, fused=False)
    k *= (1 + torch.arange(900, device="cuda")[:, None, None] / 30).to(torch.bfloat16)
    _check(q, k, v, do)


def test_tokens_past_the_last_sequence():
    # the packed buffer is longer than the documents in it, and holds NaN past them
    for d in (64, 128):
        q, k, v, do = _draw(5, 400, 4, 2, d, fused=False)
        cu = _cu([150, 101])
        want = _check(*(x[:251] for x in (q, k, v, do)), [150, 101])
        for x in (q, k, v, do):
            x[251:] = float("nan")
        out, lse = muon.attention(q, k, v, cu)
        grads = muon.attention_backward(do, q, k, v, out, lse, cu)
        assert torch.equal(out[:251], want[0]) and torch.equal(lse[:, :251], want[1])
        assert torch.count_nonzero(out[251:]) == 0 and torch.isneginf(lse[:, 251:]).all()
        for g, w in zip(grads, want[2]):
            assert torch.equal(g[:251], w) and torch.count_nonzero(g[251:]) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_non_finite_values_reach_only_what_depends_on_them(which, value, d):
    lengths = [60, 70, 200]
    q, k, v, do = _draw(6, 330, 4, 2, d, fused=False)
    t0, h0, e0 = 90, 1, 3                 # a token of the second sequence
    {"q": q, "k": k, "v": v, "do": do}[which][t0, h0, e0] = value
    cu = _cu(lengths)
    out, lse = muon.attention(q, k, v, cu)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu)
    Q, K, V, D = (f64(x) for x in (q, k, v, do))
    with np.errstate(all="ignore"):
        r_out, r_lse = ref.attention(Q, K, V, cu.cpu().numpy())
        r_grads = ref.attention_backward(D, Q, K, V, f64(out), f64(lse), cu.cpu().numpy())
    # rows (a token of a head) with no non-finite value in the oracle have none here
    for name, got, want in [("out", out, r_out), *zip(("dq", "dk", "dv"), grads, r_grads)]:
        G = f64(got)
        clean = np.isfinite(want).all(axis=2)
        assert np.isfinite(G[clean]).all(), name
        assert _rel(G[clean], want[clean]) <= REL, name
        assert not np.isfinite(G[~clean]).all(axis=1).any(), name
    fin = np.isfinite(r_lse)
    assert np.isfinite(f64(lse)[fin]).all()


@pytest.mark.parametrize("heads,d", [(20, 64), (40, 64), (40, 128)])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_non_finite_values_with_many_heads(which, heads, d):
    # as above where 2 blocks or 1 share a tile of the gradients (few heads: 4)
    lengths = [60, 70, 200]
    q, k, v, do = _draw(16, 330, heads, heads, d, fused=False)
    x = {"q": q, "k": k, "v": v, "do": do}[which]
    x[90, 1, 3], x[200, heads - 1, 0] = float("inf"), float("nan")
    cu = _cu(lengths)
    out, lse = muon.attention(q, k, v, cu)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu)
    some = [1, heads - 1]                 # the other heads hold finite values only
    Q, K, V, D, O = (f64(y[:, some]) for y in (q, k, v, do, out))
    with np.errstate(all="ignore"):
        want = ref.attention_backward(D, Q, K, V, O, f64(lse[some]), cu.cpu().numpy())
    for name, got, w in zip(("dq", "dk", "dv"), grads, want):
        G = f64(got[:, some])
        clean = np.isfinite(w).all(axis=2)
        assert np.isfinite(G[clean]).all(), name
        assert _rel(G[clean], w[clean]) <= REL, name
        assert not np.isfinite(G[~clean]).all(axis=1).any(), name
        rest = [h for h in range(heads) if h not in some]
        assert torch.isfinite(got[:, rest]).all()


def test_gradient_is_the_difference_quotient():
    # the oracle's forward differenced along a direction, against the kernel's gradients
    lengths = [40, 90]
    q, k, v, do = _draw(7, 130, 4, 2, 64)
    out, lse, grads = _check(q, k, v, do, lengths)
    r = np.random.default_rng(0)
    x = [f64(a) for a in (q, k, v)]
    cu = _cu(lengths).cpu().numpy()
    for n in range(3):
        d = r.standard_normal(x[n].shape)
        hi, lo = list(x), list(x)
        hi[n], lo[n] = x[n] + 1e-5 * d, x[n] - 1e-5 * d
        diff = np.sum(f64(do) * (ref.attention(*hi, cu)[0] - ref.attention(*lo, cu)[0])) / 2e-5
        g = f64(grads[n])
        # independent errors of rel. size REL, summed at random along the direction
        assert abs(np.sum(g * d) - diff) <= 4 * REL * np.linalg.norm(g)


def test_repeated_calls_give_equal_bits():
    q, k, v, do = _draw(8, 1000, 8, 2, 64)
    cu = _cu([600, 400])
    out, lse = muon.attention(q, k, v, cu)
    first = muon.attention_backward(do, q, k, v, out, lse, cu)
    for _ in range(3):
        o, z = muon.attention(q, k, v, cu)
        again = muon.attention_backward(do, q, k, v, o, z, cu)
        assert torch.equal(o, out) and torch.equal(z, lse)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_packed_equals_each_sequence_alone():
    # equal up to the order of the sums: the tiles of a packed sequence start elsewhere
    lengths = [200, 300, 77]
    q, k, v, do = _draw(9, 577, 4, 2, 128)
    out, lse = muon.attention(q, k, v, _cu(lengths))
    a = 0
    for n in lengths:
        o, z = muon.attention(*(x[a:a + n] for x in (q, k, v)))
        assert _rel(f64(o), f64(out[a:a + n])) <= REL
        assert np.allclose(f64(z), f64(lse[:, a:a + n]), rtol=0, atol=1e-4)
        a += n


def test_strided_outputs_and_head_major_storage():
    q, k, v, do = _draw(10, 333, 4, 2, 64)
    out, lse, grads = _check(q, k, v, do, [300, 33])
    cu = _cu([300, 33])
    fused = torch.full((333, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    muon.attention_backward(do, q, k, v, out, lse, cu, dq=fused[:, :4], dk=fused[:, 4:6],
                            dv=fused[:, 6:])
    assert torch.equal(fused, torch.cat(grads, 1))
    # [heads, tokens, dim] storage
    q2, k2, v2, do2 = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, do))
    o2 = torch.empty(4, 333, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    muon.attention(q2, k2, v2, cu, out=o2)
    assert torch.equal(o2, out)
    for a, b in zip(muon.attention_backward(do2, q2, k2, v2, o2, lse, cu), grads):
        assert torch.equal(a, b)
    # rows around a strided output keep their values
    wide = torch.full((335, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    muon.attention(q, k, v, cu, out=wide[1:334])
    assert torch.equal(wide[1:334], out) and torch.all(wide[0] == 5) and torch.all(wide[334] == 5)


def test_offsets_past_32_bits():
    # tokens 2^23 elements apart: the last one starts at element 2.5e9
    t, ts = 300, 1 << 23
    q, k, v, do = _draw(11, t, 2, 1, 64, fused=False)
    buf = torch.empty(t * ts, dtype=torch.bfloat16, device="cuda")
    far, at = [], 0
    for x in (q, k, v, do, q, k, v, q):
        h = x.shape[1]
        view = buf.as_strided((t, h, 64), (ts, 64, 1), at)
        view.copy_(x)
        far.append(view)
        at += 64 * h
    out, lse = muon.attention(q, k, v)
    grads = muon.attention_backward(do, q, k, v, out, lse)
    o2, z2 = muon.attention(*far[:3], out=far[7])
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    far_grads = muon.attention_backward(far[3], *far[:3], far[7], lse, dq=far[4], dk=far[5],
                                        dv=far[6])
    assert all(torch.equal(a, b) for a, b in zip(far_grads, grads))


def test_zero_tokens_and_only_empty_sequences():
    q, k, v, do = _draw(12, 5, 2, 1, 64)
    before = muon.kernel_launch_count()
    out, lse = muon.attention(q[:0], k[:0], v[:0])
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    muon.attention_backward(do[:0], q[:0], k[:0], v[:0], out, lse)
    assert muon.kernel_launch_count() == before
    out, lse = muon.attention(q, k, v, _cu([0, 0]))
    assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()
    for g in muon.attention_backward(do, q, k, v, out, lse, _cu([0, 0])):
        assert torch.count_nonzero(g) == 0


def test_offsets_that_do_not_ascend_stay_inside_the_tensors():
    # undefined results, but no access outside: the call ends and later calls are right
    q, k, v, do = _draw(13, 400, 2, 1, 64)
    for cu in ([50, 400], [0, 300, 100, 400], [0, 1000], [-5, 200, 400], [0, 200, 2 ** 31 - 1]):
        c = torch.tensor(cu, dtype=torch.int32).cuda()
        out, lse = muon.attention(q, k, v, c)
        muon.attention_backward(do, q, k, v, out, lse, c)
    torch.cuda.synchronize()
    _check(q, k, v, do, [400])


def test_two_streams_at_once():
    # each stream has its own default workspace
    data = [_draw(20 + i, 900, 4, 2, 64) for i in range(2)]
    want = [_check(*x) for x in data]
    streams = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for (q, k, v, do), st in zip(data, streams):
            out, lse = muon.attention(q, k, v, stream=st)
            got.append((out, lse, muon.attention_backward(do, q, k, v, out, lse, stream=st)))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and all(torch.equal(a, b) for a, b in zip(g[2], w[2]))


def test_in_a_cuda_graph():
    q, k, v, do = _draw(22, 500, 4, 2, 64)
    cu = _cu([280, 220])
    ws = muon.Workspace(muon.attention_workspace_bytes(500, 4, 2, 64))
    bufs = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in (q, q, k, v)]
    lse = torch.empty(4, 500, device="cuda")

    def step():
        muon.attention(q, k, v, cu, out=bufs[0], lse=lse, workspace=ws)
        muon.attention_backward(do, q, k, v, bufs[0], lse, cu, dq=bufs[1], dk=bufs[2], dv=bufs[3],
                                workspace=ws)

    step()
    want = [x.clone() for x in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in bufs:
        x.zero_()
    cu.copy_(_cu([100, 400]))              # the offsets are read on the device
    graph.replay()
    cu.copy_(_cu([280, 220]))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))
    assert muon.workspace_status(ws) == 0


def test_a_failed_workspace_is_left_alone():
    q, k, v, do = _draw(23, 200, 2, 1, 64)
    ws = muon.Workspace(muon.attention_workspace_bytes(200, 2, 1, 64))
    out, lse = muon.attention(q, k, v, workspace=ws)
    muon.selftest_wait_timeout(ws, limit_us=1000)
    o2 = torch.full_like(out, 3.0)
    muon.attention(q, k, v, out=o2, workspace=ws)
    grads = [torch.full_like(x, 3.0, memory_format=torch.contiguous_format) for x in (q, k, v)]
    muon.attention_backward(do, q, k, v, out, lse, dq=grads[0], dk=grads[1], dv=grads[2],
                            workspace=ws)
    assert muon.workspace_status(ws, clear=True) == 4
    assert all(torch.all(x == 3.0) for x in (o2, *grads))
    assert torch.equal(muon.attention(q, k, v, workspace=ws)[0], out)


def test_refusals():
    q, k, v, do = _draw(24, 20, 4, 2, 64)
    out, lse = muon.attention(q, k, v)
    for args, exc in [((q.float(), k.float(), v.float()), TypeError), ((q, k, v.half()), TypeError),
                      ((q[:, :3], k, v), ValueError), ((q, k[:5], v[:5]), ValueError),
                      ((q, k, v[:, :1]), ValueError), ((q[..., :32], k, v), ValueError),
                      ((q, k, v, torch.zeros(2, device="cuda")), TypeError),
                      ((q, k, v, torch.zeros(0, dtype=torch.int32, device="cuda")), ValueError),
                      ((q, k, v, torch.zeros(2, dtype=torch.int32)), ValueError)]:
        with pytest.raises(exc):
            muon.attention(*args)
    with pytest.raises(muon.MuonError):
        muon.attention(q, k, v, scale=0.0)
    with pytest.raises(muon.MuonError):                     # zero strides: a broadcast gradient
        muon.attention_backward(do[:1].expand_as(do), q, k, v, out, lse)
    with pytest.raises(muon.MuonError):                     # heads of 20 elements
        muon.attention(*(torch.zeros(4, 1, 20, dtype=q.dtype, device="cuda") for _ in range(3)))
    with pytest.raises(ValueError):
        muon.attention_backward(do, q, k, v, out, lse[:, :3])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tokens", [1, 3])       # of the sequence that see minus infinity only
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_whose_visible_scores_are_all_minus_infinity(sign, tokens, d):
    # exp(s - max s) is exp(-inf + inf): NaN, as by the definition; not the 0 of a row without keys
    q, k, v, do = _draw(60 + d, 330, 4, 2, d, fused=False)
    h0, e0, rows = 1, 3, slice(60, 60 + tokens)           # the second sequence's first tokens
    q[rows, h0, e0] = sign * float("inf")
    k[rows, h0 // 2, e0] = -sign
    cu = _cu([60, 70, 150])                               # and 50 tokens of no sequence
    out, lse = muon.attention(q, k, v, cu)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu)
    Q, K, V, D = (f64(x) for x in (q, k, v, do))
    with np.errstate(all="ignore"):
        r_out, r_lse = ref.attention(Q, K, V, cu.cpu().numpy())
        r_grads = ref.attention_backward(D, Q, K, V, f64(out), f64(lse), cu.cpu().numpy())
    assert np.isnan(r_out[rows, h0]).all() and np.isnan(r_lse[h0, rows]).all()
    for name, got, want in [("out", out, r_out), *zip(("dq", "dk", "dv"), grads, r_grads)]:
        G = f64(got)
        clean = np.isfinite(want).all(axis=2)
        assert np.isfinite(G[clean]).all(), name
        assert _rel(G[clean], want[clean]) <= REL, name
        assert not np.isfinite(G[~clean]).all(axis=1).any(), name
    assert np.array_equal(np.isnan(f64(lse)), np.isnan(r_lse))
    assert np.array_equal(np.isneginf(f64(lse)), np.isneginf(r_lse))


def test_two_threads_on_one_stream():
    # the two launches of a gradient call hand over through the stream's default workspace
    data = [_draw(70 + i, 257 + 640 * i, 4, 2, 64) for i in range(2)]
    want = []
    for q, k, v, do in data:
        out, lse = muon.attention(q, k, v)
        want.append((out, lse, muon.attention_backward(do, q, k, v, out, lse)))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        q, k, v, do = data[i]
        start.wait()
        for _ in range(200):
            grads = muon.attention_backward(do, q, k, v, *want[i][:2], stream=stream)
            got[i].append(grads)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 200
        assert all(torch.equal(a, b) for grads in g for a, b in zip(grads, w[2]))


def test_cuda_graphs_with_the_default_workspace():
    # Two graphs captured on one stream, replayed in the other order, while eager calls on that
    # stream and on another one need larger workspaces.
    def case(seed, t):
        q, k, v, do = _draw(seed, t, 4, 2, 64)
        cos, sin = muon.rope_tables(t, 64)
        w = [torch.linspace(0.5, 1.5, 64, device="cuda") for _ in range(2)]

        def step():
            qn, kn = muon.qk_norm_rope(q, k, cos, sin, q_weight=w[0], k_weight=w[1])
            out, lse = muon.attention(qn, kn, v)
            dq, dk, dv = muon.attention_backward(do, qn, kn, v, out, lse)
            grads = muon.qk_norm_rope_backward(dq, dk, q, k, cos, sin, q_weight=w[0],
                                               k_weight=w[1])
            return (out, lse, dv, *grads)

        return step

    stream = torch.cuda.Stream()
    steps = [case(80, 200), case(81, 333)]
    want = [step() for step in steps]
    large = case(82, 1900)
    large_want = large()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for step in steps:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            outs.append(step())
        graphs.append(graph)
    for order in ((1, 0), (0, 1), (1, 1, 0)):
        for x in (y for out in outs for y in out):
            x.fill_(3.0)
        with torch.cuda.stream(stream):
            eager = large()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for got, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, w))
        assert all(torch.equal(a, b) for a, b in zip(eager, large_want))


def test_a_failed_default_workspace_is_seen_and_cleared():
    q, k, v, do = _draw(90, 200, 2, 1, 64)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = muon.attention(q, k, v, stream=stream)
    assert muon.workspace_status(None, stream=stream) == 0
    ws = muon._stream_ws[(torch.cuda.current_device(), stream.cuda_stream)][2]
    muon.selftest_wait_timeout(ws, limit_us=1000, stream=stream)
    o2 = torch.full_like(out, 3.0)
    torch.cuda.synchronize()
    muon.attention(q, k, v, out=o2, stream=stream)
    assert muon.workspace_status(None, stream=stream) == 4
    assert torch.all(o2 == 3.0)
    assert muon.workspace_status(None, clear=True, stream=stream) == 4
    assert muon.workspace_status(None, stream=stream) == 0
    muon.attention(q, k, v, out=o2, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(o2, out)
    # another stream has another one
    assert muon.workspace_status(None) == 0


def test_outputs_over_inputs_are_refused():
    q, k, v, do = _draw(91, 50, 4, 4, 64)
    out, lse = muon.attention(q, k, v)
    before = [x.clone() for x in (q, k, v, do, out, lse)]
    for x in (q, k, v):
        with pytest.raises(muon.MuonError):
            muon.attention(q, k, v, out=x)
    spare = torch.empty(50, 12, 64, dtype=q.dtype, device="cuda")
    for name in ("dq", "dk", "dv"):
        for x in (q, k, v, do, out):
            with pytest.raises(muon.MuonError):
                muon.attention_backward(do, q, k, v, out, lse, **{name: x})
    with pytest.raises(muon.MuonError):
        muon.attention_backward(do, q, k, v, out, lse, dk=spare[:, :4], dv=spare[:, 3:7])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((q, k, v, do, out, lse), before))
    # columns of one tensor that holds the inputs too
    wide = torch.empty(50, 24, 64, dtype=q.dtype, device="cuda")
    wide[:, :4], wide[:, 4:8], wide[:, 8:12], wide[:, 12:16] = q, k, v, do
    part = [wide[:, i:i + 4] for i in range(0, 24, 4)]
    o2, z2 = muon.attention(*part[:3], out=part[4])
    assert torch.equal(o2, out) and torch.equal(z2, lse)
    got = muon.attention_backward(part[3], *part[:3], o2, z2, dk=part[5])
    for a, b in zip(got, muon.attention_backward(do, q, k, v, out, lse)):
        assert torch.equal(a, b)


def test_tensors_that_require_grad_are_refused_while_autograd_records():
    q, k, v, do = _draw(92, 40, 4, 2, 64, fused=False)
    cos, sin = muon.rope_tables(40, 64)
    w = torch.ones(64, device="cuda")
    out, lse = muon.attention(q, k, v)
    rotated = muon.qk_norm_rope(q, k, cos, sin, q_weight=w, k_weight=w)
    for x in (q, k, v):
        x.requires_grad_(True)
        with pytest.raises(ValueError, match="attention_backward"):
            muon.attention(q, k, v)
        with torch.no_grad():
            assert torch.equal(muon.attention(q, k, v)[0], out)
        muon.attention_backward(do, q, k, v, out, lse)      # no gradient is lost here
        x.requires_grad_(False)
    for x in (q, k, w):
        x.requires_grad_(True)
        with pytest.raises(ValueError, match="qk_norm_rope_backward"):
            muon.qk_norm_rope(q, k, cos, sin, q_weight=w, k_weight=w)
        x.requires_grad_(False)

    class Attention(torch.autograd.Function):               # the way into a module
        @staticmethod
        def forward(ctx, q, k, v):
            o, z = muon.attention(q, k, v)
            ctx.save_for_backward(q, k, v, o, z)
            return o

        @staticmethod
        def backward(ctx, g):
            q, k, v, o, z = ctx.saved_tensors
            return muon.attention_backward(g, q, k, v, o, z)

    leaves = [x.detach().clone().requires_grad_(True) for x in (q, k, v)]
    Attention.apply(*leaves).backward(do)
    for x, g in zip(leaves, muon.attention_backward(do, q, k, v, out, lse)):
        assert torch.equal(x.grad, g)


# where a value that is not finite may stand: first, middle and last token of the second document,
# the neighbours' tokens next to it (in its first and last tile), each in one element or a row
BAD_TOKENS = [270, 271, 383, 384, 600, 768, 899, 269, 900]


@pytest.mark.parametrize("hq,hk,d", [(4, 2, 64), (24, 24, 64), (2, 1, 128)])
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_non_finite_values_over_several_tiles(which, whole, hq, hk, d):
    lengths = [270, 630, 100]
    cu = _cu(lengths)
    for token in BAD_TOKENS:
        for value in (float("nan"), float("inf")):
            q, k, v, do = _draw(100 + token, 1000, hq, hk, d, fused=False)
            x, h0 = {"q": q, "k": k, "v": v, "do": do}[which], 1 if which in "q do" else 0
            if whole:
                x[token, h0] = value
            else:
                x[token, h0, 5] = value
            out, lse = muon.attention(q, k, v, cu)
            grads = muon.attention_backward(do, q, k, v, out, lse, cu)
            some = sorted({0, 1, hq - 1})             # the rest holds finite values only
            g = sorted({h // (hq // hk) for h in some})
            pick = [h for h in range(hq) if h // (hq // hk) in g]
            Q, K, V, D, O = (f64(y) for y in (q[:, pick], k[:, g], v[:, g], do[:, pick],
                                              out[:, pick]))
            Z = f64(lse[pick])
            c = cu.cpu().numpy()
            with np.errstate(all="ignore"):
                r_out, r_lse = ref.attention(Q, K, V, c)
                want = ref.attention_backward(D, Q, K, V, O, Z, c)
            # out and dv element by element: other columns of a row keep their values
            for name, got, w in [("out", O, r_out), ("dv", f64(grads[2][:, g]), want[2])]:
                fin = np.isfinite(w)
                assert np.array_equal(np.isfinite(got), fin), (name, token, value)
                assert _rel(got[fin], w[fin]) <= REL, (name, token, value)
            assert np.array_equal(np.isfinite(Z), np.isfinite(r_lse))
            for name, got, w in [("dq", f64(grads[0][:, pick]), want[0]),
                                 ("dk", f64(grads[1][:, g]), want[1])]:
                clean = np.isfinite(w).all(axis=2)
                assert np.isfinite(got[clean]).all(), (name, token, value)
                assert _rel(got[clean], w[clean]) <= REL, (name, token, value)
                assert not np.isfinite(got[~clean]).all(axis=1).any(), (name, token, value)
            rest = [h for h in range(hk) if h not in g]
            assert all(torch.isfinite(y[:, rest]).all() for y in grads[1:])


@pytest.mark.parametrize("hq,hk,d", [(8, 4, 64), (8, 2, 128)])
def test_non_finite_values_cost_no_walk_of_every_row(hq, hk, d):
    # 8192 tokens take about 0.3 ms forward, 1 ms backward; a walk of all keys by every row that
    # one value reaches took 470 and 360 ms.  What may still be walked: a tile's rows.
    t = 8192
    two = _cu([300, t - 300]), _cu([t - 300, 300])
    cases = [(which, token, whole, None) for which in range(4)
             for token in (0, t // 2 + 5, t - 1) for whole in (False, True)]
    cases += [(None, 299, True, two[0]), (None, t - 300, True, two[1])]
    for which, token, whole, cu in cases:
        x = _draw(7, t, hq, hk, d, fused=False)
        for i, y in enumerate(x):
            if which is None or i == which:
                y[token, 0, 3] = float("nan")
                if whole:
                    y[token] = float("nan")
        q, k, v, do = x

        def call():
            out, lse = muon.attention(q, k, v, cu)
            return muon.attention_backward(do, q, k, v, out, lse, cu)

        call()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        assert start.elapsed_time(end) < 60.0, (which, token, whole)


@pytest.mark.parametrize("d", [16, 128])
def test_parity_where_blocks_take_the_tiles_by_their_work(d):
    # 1 to 4 waves of blocks and few heads a tile, forward and dk/dv; documents of different lengths
    lengths = [700, 3, 0, 1201, 130, 1, 641, 77, 900, 1340]
    q, k, v, do = _draw(110 + d, sum(lengths), 16, 8, d)
    cu = _cu(lengths)
    out, lse = muon.attention(q, k, v, cu)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu)
    for g in (0, 7):                      # a key head at a time, with its two query heads
        h = slice(2 * g, 2 * g + 2)
        Q, D, K, V, L = (f64(x) for x in (q[:, h], do[:, h], k[:, g:g + 1], v[:, g:g + 1], lse[h]))
        c = cu.cpu().numpy()
        r_out, r_lse = ref.attention(Q, K, V, c)
        b = _magnitudes(Q, K, V, D, r_out, L, c, d ** -0.5)
        want = ref.attention_backward(D, Q, K, V, r_out, L, c)
        assert np.all(np.abs(L - r_lse) <= b[1] + 1e-30)
        got = (out[:, h], grads[0][:, h], grads[1][:, g:g + 1], grads[2][:, g:g + 1])
        for name, x, w, e in zip(("out", "dq", "dk", "dv"), got, (r_out, *want), (b[0], *b[2:])):
            err = np.abs(f64(x) - w) - (U * np.abs(w) + (1 + U) * e + 1e-30)
            assert np.all(err <= 0), (name, g, float(err.max()))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_padding_gets_no_gradient_behind_values_that_are_not_finite(which, d):
    # tokens past the last sequence in a tile with tokens that are not finite, and in tiles behind
    q, k, v, do = _draw(120 + d, 500, 4, 2, d, fused=False)
    cu = _cu([100, 190])
    {"q": q, "k": k, "v": v, "do": do}[which][[40, 260, 280, 400], 1] = float("inf")
    out, lse = muon.attention(q, k, v, cu)
    grads = muon.attention_backward(do, q, k, v, out, lse, cu)
    assert torch.count_nonzero(out[290:]) == 0 and torch.isneginf(lse[:, 290:]).all()
    for g in grads:
        assert torch.count_nonzero(g[290:]) == 0


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (8, 8, 128), (32, 8, 128)])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
def test_non_finite_values_before_an_end_inside_a_tile(which, hq, hk, d):
    # the last tile holds fewer than 128 tokens, and its sequence shares a tile with one before
    lengths = [2, 88, 520, 0, 543]
    cu = _cu(lengths)
    for token in (671, 1100, 1152):
        for value in (float("nan"), -float("inf")):
            q, k, v, do = _draw(130 + token, 1153, hq, hk, d, fused=False)
            {"q": q, "k": k, "v": v, "do": do}[which][token] = value
            out, lse = muon.attention(q, k, v, cu)
            grads = muon.attention_backward(do, q, k, v, out, lse, cu)
            for x in (out, *grads):
                assert torch.isfinite(x[:610]).all(), (token, value)
            assert not torch.isfinite(grads[1][token]).all()
