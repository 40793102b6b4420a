"""GPU parity of the norm and the clipping of all gradients with the float64 oracle.

Squares are summed in fp32, at most n / 8 of them an accumulator (n: a thread's elements, a few
hundred here), and the threads' and blocks' sums in some 30 further additions: the sum of squares is
off by at most 2^-15 of itself, the norm by half of that and a few roundings, kNorm = 2^-15.  The factor adds two roundings, an output its own
(2^-24 in fp32, 2^-8 in bf16).
"""

import math

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import block_oracle as ref

pytestmark = pytest.mark.gpu

kNorm, kBf16 = 2.0 ** -15, 2.0 ** -8
DEV = "cuda"
B, F = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def _draw(seed, shapes, dtypes, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return [(std * torch.randn(*s, generator=gen)).to(d).to(DEV) for s, d in zip(shapes, dtypes)]


def _check(grads, max_norm, outs=None, eps=1e-6):
    G = [f64(g) for g in grads]
    norm = muon.clip_grad_norm(grads, max_norm, outs=outs, eps=eps)
    torch.cuda.synchronize()
    want = ref.grad_norm(G)
    assert norm.shape == () and abs(float(norm) - want) <= kNorm * want
    c = ref.clip_factor(want, max_norm, eps)
    for g, o in zip(G, grads if outs is None else outs):
        u = kBf16 if o.dtype == B else 2.0 ** -24
        assert np.all(np.abs(f64(o) - c * g) <= (u * (1 + kNorm) + kNorm + 2.0 ** -22) * np.abs(c * g)
                      + 1e-37)


SHAPES = [(1,), (7,), (8,), (16384,), (16385,), (3, 5, 7), (128, 256), (100003,), (0,), (40000, 3)]


@pytest.mark.parametrize("dtypes", [[B] * 10, [F] * 10, [B, F] * 5])
@pytest.mark.parametrize("max_norm", [1.0, 1e6, 0.0])
def test_parity_in_place(dtypes, max_norm):
    _check(_draw(1, SHAPES, dtypes), max_norm)


@pytest.mark.parametrize("g,o", [(B, B), (B, F), (F, B), (F, F)])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_parity_into_outputs(g, o, max_norm):
    grads = _draw(2, SHAPES, [g] * 10)
    before = [x.clone() for x in grads]
    outs = [torch.full_like(x, 3.0, dtype=o) for x in grads]
    _check(grads, max_norm, outs)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_more_tensors_than_a_launch_takes():
    for n in (64, 65, 130):
        grads = _draw(n, [(100 + i,) for i in range(n)], [B, F] * n)
        _check(grads, 2.0)
        _check(grads, 2.0, [torch.empty_like(g, dtype=F) for g in grads])


def test_one_large_tensor():
    _check([torch.randn(20_000_003, device=DEV).bfloat16()], 3.0)


def test_factor_one_leaves_the_gradients_as_they_are():
    grads = _draw(3, SHAPES, [B, F] * 5)
    before = [g.clone() for g in grads]
    muon.clip_grad_norm(grads, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    norm = muon.grad_norm(grads)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    want = ref.grad_norm([f64(g) for g in grads])
    assert abs(float(norm) - want) <= kNorm * want


def test_extreme_values():
    zero = [torch.zeros(100, device=DEV), torch.zeros(33, dtype=B, device=DEV)]
    assert float(muon.clip_grad_norm(zero, 1.0)) == 0.0 and all(torch.all(z == 0) for z in zero)
    # squares below fp32's smallest add nothing; sums past its largest are held in another unit
    assert float(muon.grad_norm([torch.full((100,), 1e-30, device=DEV)])) == 0.0
    big = torch.full((1 << 20,), 1e18, device=DEV)
    assert abs(float(muon.grad_norm([big])) / (1e18 * 1024) - 1) < kNorm
    assert math.isinf(float(muon.grad_norm([torch.full((8,), 1e20, device=DEV)])))
    for value, rest in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        g = torch.ones(3000, device=DEV)
        g[5] = value
        norm = float(muon.clip_grad_norm([g], 1.0))
        assert norm == value or math.isnan(norm) and math.isnan(value)
        assert torch.isnan(g[5])
        assert math.isnan(rest) and torch.isnan(g).all() or torch.all(g[6:] == rest)


def test_prepared_repeated_captured_and_streams():
    grads = _draw(4, SHAPES, [B] * 10)
    outs = [torch.empty_like(g) for g in grads]
    clip = muon.ClipGradNorm(grads, 1.0, outs=outs)
    first = clip()
    want = [o.clone() for o in outs]
    for _ in range(3):
        for o in outs:
            o.fill_(9.0)
        again = clip()
        assert torch.equal(again, first) and again.data_ptr() != first.data_ptr()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        norm = clip()
    for o in outs:
        o.fill_(9.0)
    norm.fill_(0.0)
    graph.replay()
    muon.grad_norm(grads[:3])
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(outs, want))
    for o in outs:
        o.fill_(9.0)
    torch.cuda.synchronize()
    norm = clip(stream)
    torch.cuda.synchronize()
    assert torch.equal(norm, first) and all(torch.equal(a, b) for a, b in zip(outs, want))
    # new values at the same addresses
    for g in grads:
        g.mul_(2.0)
    assert abs(float(clip()) / (2 * float(first)) - 1) < kNorm


def test_after_a_failure_nothing_is_stored():
    grads = _draw(5, [(5000,)], [B])
    before = grads[0].clone()
    ws = muon.Workspace(4096 * 4)
    muon.selftest_wait_timeout(ws, limit_us=1000)
    muon.clip_grad_norm(grads, 0.1, workspace=ws)
    assert muon.workspace_status(ws, clear=True) == 4 and torch.equal(grads[0], before)
    muon.clip_grad_norm(grads, 0.1, workspace=ws)
    assert muon.workspace_status(ws) == 0
    assert abs(np.linalg.norm(f64(grads[0])) / 0.1 - 1) < 2 * kBf16


def test_refusals():
    g = _draw(6, [(64,), (64,)], [B, F])
    wide = torch.zeros(200, dtype=B, device=DEV)
    for grads, kw, exc in [([], {}, ValueError), ([g[0].half()], {}, TypeError),
                           ([wide.view(10, 20).t()], {}, ValueError),
                           (g, dict(outs=g[:1]), ValueError),
                           (g, dict(outs=[g[0][:8], g[1]]), ValueError),
                           ([wide[:64], wide[32:96]], {}, ValueError),
                           ([g[0], g[0]], {}, ValueError),
                           ([wide[:64]], dict(outs=[wide[8:72]]), ValueError)]:
        with pytest.raises(exc):
            muon.clip_grad_norm(grads, 1.0, **kw)
    for bad in (-1.0, float("nan")):
        with pytest.raises(muon.MuonError):
            muon.clip_grad_norm(g, bad)
    with pytest.raises(muon.MuonError):                 # not 16-byte aligned
        muon.clip_grad_norm([wide[1:65]], 1.0)


@pytest.mark.parametrize("o", [B, F])
def test_an_infinite_max_norm_copies_to_outs(o):
    grads = _draw(8, SHAPES, [B, F] * 5)
    outs = [torch.full_like(g, 3.0, dtype=o) for g in grads]
    before = [g.clone() for g in grads]
    norm = muon.clip_grad_norm(grads, math.inf, outs=outs)
    assert torch.equal(norm, muon.grad_norm(grads))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert all(torch.equal(a, b.to(o)) for a, b in zip(outs, grads))


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 1e20])
def test_an_infinite_max_norm_is_factor_one_whatever_the_norm(value):
    # (1e20: squares past fp32's range, an infinite norm of finite gradients)
    grads = _draw(9, SHAPES, [B, F] * 5)
    grads[5].view(-1)[7] = value
    in_place = {1, 5, 6}                                # beside tensors with outs of their own
    before = [g.clone() for g in grads]
    outs = [g if i in in_place else torch.full_like(g, 3.0) for i, g in enumerate(grads)]
    norm = float(muon.clip_grad_norm(grads, math.inf, outs=outs))
    assert not math.isfinite(norm)
    for g, o, b in zip(grads, outs, before):
        bits = torch.int16 if g.dtype == B else torch.int32
        assert torch.equal(g.view(bits), b.view(bits))
        assert torch.equal(o.nan_to_num(nan=7.0), b.nan_to_num(nan=7.0))
    # into the other type, where the value is not in place
    outs = [torch.full_like(g, 3.0, dtype=F if g.dtype == B else B) for g in grads]
    muon.clip_grad_norm(grads, math.inf, outs=outs)
    for o, b in zip(outs, before):
        assert torch.equal(o.nan_to_num(nan=7.0), b.to(o.dtype).nan_to_num(nan=7.0))


def test_magnitudes_below_2_58_of_more_elements_than_a_chain_takes():
    # 6e9 of 1.875 2^57: the sum of squares passes 2^128 thousands of times, and a thread's share of
    # them (4800 squares a chain, unless they are cut) passes it as well
    n = 6_000_000_007
    g = torch.full((n,), 1.875 * 2.0 ** 57, dtype=B, device=DEV)
    small = torch.full((1000,), 3.0, device=DEV)
    want = 1.875 * 2.0 ** 57 * math.sqrt(n)
    assert abs(float(muon.grad_norm([g, small])) / want - 1) <= kNorm
    # sums in units of 1: chains that are cut, ordinary values
    g.fill_(0.0078125)
    g[:n // 2].fill_(2.0)
    want = math.sqrt(4.0 * (n // 2) + 0.0078125 ** 2 * (n - n // 2) + 9000)
    assert abs(float(muon.grad_norm([g, small])) / want - 1) <= kNorm
    # both: most threads' sums stay small, some do not
    g[n - 100_000:] = 2.0 ** 56
    want = math.sqrt(want * want + 100_000 * 2.0 ** 112)
    assert abs(float(muon.grad_norm([small, g])) / want - 1) <= kNorm
