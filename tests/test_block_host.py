"""Host-only checks of the block operators' C entry points and of the binding: refusals before
anything is enqueued, workspace sizes."""

import ctypes
import os

import pytest
import torch

import newton_schulz_step_gb300 as muon

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(6)
NONE = muon._Matrix(None, 0)
WS, WS_BYTES = 0x40000000, 1 << 30


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(muon.library_path()):
        from newton_schulz_step_gb300 import build
        build.build()
    return muon.load_library()


def _m(i, stride=64, shift=0):
    """The i-th of views that share nothing (16 rows of 64)."""
    return muon._Matrix(0x100000 * (i + 1) + shift, stride)


BAD_VIEWS = [dict(data=None), dict(data=0x100008), dict(row_stride=0), dict(row_stride=-64),
             dict(row_stride=56), dict(row_stride=68), dict(row_stride=1 << 38)]


def _bad(view, kw):
    return muon._Matrix(kw.get("data", view.data), kw.get("row_stride", view.row_stride))


# ------------------------------------------------------------ linear
def _lspec(**kw):
    a = dict(tokens=16, in_features=64, out_features=64, activation=0, bias=None)
    a.update(kw)
    return muon._LinearSpec(*[a[n] for n, _ in muon._LinearSpec._fields_])


def _linear(lib, spec, views=None, ws=WS, n=WS_BYTES):
    v = views or [_m(0), _m(1), NONE, NONE, _m(2)]
    return lib.muon_linear(spec, *v, ws, n, None)


def _linear_back(lib, spec, views=None, db=None, ws=WS, n=WS_BYTES):
    v = views or [_m(i) for i in range(7)]
    return lib.muon_linear_backward(spec, *v, db, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=2 ** 31 - 1), dict(in_features=0), dict(out_features=0),
    dict(in_features=(1 << 20) + 1), dict(out_features=(1 << 20) + 1), dict(activation=-1),
    dict(activation=3), dict(bias=0x1008)])
def test_linear_refuses_a_bad_spec(lib, kw):
    assert _linear(lib, _lspec(**kw)) == INVALID
    assert _linear_back(lib, _lspec(**kw)) == INVALID
    assert _linear(lib, None) == INVALID and _linear_back(lib, None) == INVALID


@pytest.mark.parametrize("kw", BAD_VIEWS)
def test_linear_refuses_a_bad_view(lib, kw):
    for at in range(5):
        v = [_m(i) for i in range(5)]
        v[at] = _bad(v[at], kw)
        if at in (2, 3) and kw.get("data", 1) is None:
            continue                            # residual and preact may be left out
        assert _linear(lib, _lspec(), v) == INVALID
    for at in range(7):
        v = [_m(i) for i in range(7)]
        v[at] = _bad(v[at], kw)
        assert _linear_back(lib, _lspec(activation=1), v) == INVALID
    assert _linear_back(lib, _lspec(), db=0x1008) == INVALID


def test_linear_refuses_outputs_over_inputs_and_each_other(lib):
    row = 128
    for shift in (0, row, 15 * row, -15 * row):
        for out, others in ((4, (0, 1, 3)), (3, (0, 1, 2, 4))):
            for other in others:
                v = [_m(i) for i in range(5)]
                v[out] = _m(other, shift=shift)
                assert _linear(lib, _lspec(), v) == INVALID, (out, other, shift)
        # dz, dx, dweight over the inputs and over each other
        for out, others in ((4, range(4)), (5, range(5)), (6, range(6))):
            for other in others:
                v = [_m(i) for i in range(7)]
                v[out] = _m(other, shift=shift)
                assert _linear_back(lib, _lspec(activation=1), v) == INVALID, (out, other, shift)
    v = [_m(i) for i in range(5)]
    v[4] = _m(2, shift=row)                     # not the very view of the residual
    assert _linear(lib, _lspec(), v) == INVALID
    assert _linear(lib, _lspec(bias=0x100000 * 5 + 32), [_m(i) for i in range(5)]) == INVALID
    for at in range(7):
        assert _linear_back(lib, _lspec(activation=1), db=0x100000 * (at + 1) + 256) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the views are no memory of a GPU")
def test_linear_takes_views_that_are_allowed(lib):
    v = [_m(i) for i in range(5)]
    v[4] = v[2]                                 # out is the residual
    assert _linear(lib, _lspec(), v) in (UNSUPPORTED, CUDA)
    # columns of one tensor of 256: x, residual, out
    wide = [muon._Matrix(0x100000 + 128 * i, 256) for i in range(3)]
    assert _linear(lib, _lspec(), [wide[0], _m(5), wide[1], NONE, wide[2]]) in (UNSUPPORTED, CUDA)
    # without an activation preact and dz are not looked at
    v = [_m(0), _m(1), _m(2), NONE, NONE, _m(5), _m(6)]
    assert _linear_back(lib, _lspec(), v) in (UNSUPPORTED, CUDA)
    # a stride of one row is ignored
    v = [muon._Matrix(_m(i).data, 0 if i != 1 else 64) for i in range(5)]
    assert _linear(lib, _lspec(tokens=1), v) in (UNSUPPORTED, CUDA)


def test_linear_sizes_and_workspace(lib):
    assert _linear(lib, _lspec(tokens=0)) == OK
    for call in (_linear, _linear_back):
        assert call(lib, _lspec(), ws=None) == WORKSPACE
        assert call(lib, _lspec(), ws=WS + 16) == WORKSPACE
        assert call(lib, _lspec(), n=128) == WORKSPACE
    f = lib.muon_linear_workspace_bytes
    assert f(0, 64, 64) >= 256 and f(4, 4096, 4096) >= 256
    for bad in ((-1, 64, 64), (2 ** 31 - 1, 64, 64), (4, 0, 64), (4, 64, 0), (4, 1 << 21, 64)):
        assert f(*bad) == 0
    # splits of few tiles leave fp32 sums, of whole tiles, at most two a pair of CTAs each
    for t in (5, 100, 1003, 8192, 100000):
        for k, n in ((64, 64), (520, 1000), (11008, 4096), (17, 50257)):
            got = f(t, k, n)
            assert 256 <= got <= 256 + 2 * 152 * 256 * 256 * 4 + 128 * n * 4 + 1024
            # it is enough: the views are looked at next
            spec, none = _lspec(tokens=t, in_features=k, out_features=n), [muon._Matrix(0, 0)]
            assert _linear(lib, spec, none * 5, n=got) == INVALID
            assert _linear_back(lib, spec, none * 7, n=got) == INVALID


# ------------------------------------------------------------ RMS norm
def _nspec(**kw):
    a = dict(dtype=1, tokens=16, dim=64, eps=1e-6, weight=None)
    a.update(kw)
    return muon._RmsNormSpec(*[a[n] for n, _ in muon._RmsNormSpec._fields_])


def _norm(lib, spec, views=None):
    v = views or [_m(0), _m(1), _m(2), _m(3)]    # x, residual, out, sum
    return lib.muon_rms_norm(spec, *v, None)


def _norm8(lib, spec, group=128, views=None, scales=0x900000):
    v = views or [_m(0), _m(1), _m(2), _m(3)]
    return lib.muon_rms_norm_fp8(spec, group, *v[:3], scales, v[3], None)


def _norm_back(lib, spec, views=None, dw=None, ws=WS, n=WS_BYTES):
    v = views or [_m(0), _m(1), _m(2), _m(3)]    # dout, sum, dresidual, dx
    return lib.muon_rms_norm_backward(spec, *v, dw, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(tokens=-1), dict(tokens=2 ** 31 - 1), dict(dim=0), dict(dim=60),
    dict(dim=16392), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(weight=0x1004)])
def test_rms_norm_refuses_a_bad_spec(lib, kw):
    assert _norm(lib, _nspec(**kw)) == INVALID
    assert _norm8(lib, _nspec(**kw)) == INVALID
    assert _norm_back(lib, _nspec(**kw), dw=0x2000 if "weight" in kw else None) == INVALID


@pytest.mark.parametrize("kw", BAD_VIEWS)
def test_rms_norm_refuses_a_bad_view(lib, kw):
    for at in range(4):
        v = [_m(i) for i in range(4)]
        v[at] = _bad(v[at], kw)
        assert _norm(lib, _nspec(), v) == INVALID
        if not (at == 2 and kw.get("data", 1) is None):
            assert _norm_back(lib, _nspec(), v) == INVALID
        if not (at == 2 and kw.get("row_stride") in (68,)):
            assert _norm8(lib, _nspec(), views=v) == INVALID
    assert _norm8(lib, _nspec(), group=64) == INVALID
    assert _norm8(lib, _nspec(), scales=None) == INVALID
    assert _norm8(lib, _nspec(), scales=0x900002) == INVALID
    v = [_m(0), _m(1), _m(2, stride=68), _m(3)]  # rows of bytes are 8-byte aligned
    assert _norm8(lib, _nspec(), views=v) == INVALID


def test_rms_norm_outputs_apart(lib):
    row = 128
    for shift in (row, 15 * row, -15 * row):
        for out in (2, 3):
            for other in (0, 1):
                v = [_m(i) for i in range(4)]
                v[out] = _m(other, shift=shift)
                assert _norm(lib, _nspec(), v) == INVALID
    for other in range(4):
        v = [_m(i) for i in range(4)]
        v[2] = _m(other)
        if other != 2:
            # 8 bits over anything: refused, also at the same address
            assert _norm8(lib, _nspec(), views=v) == INVALID
        if other == 3:
            assert _norm(lib, _nspec(), v) == INVALID
        assert _norm8(lib, _nspec(), scales=0x100000 * (other + 1) + 256) == INVALID
    v = [_m(i) for i in range(4)]
    for shift in (row, -row):
        for other in range(3):
            v[3] = _m(other, shift=shift)
            assert _norm_back(lib, _nspec(), v) == INVALID
    assert _norm_back(lib, _nspec(weight=0x9000), dw=0x9010) == INVALID
    for at in range(4):
        assert _norm_back(lib, _nspec(weight=0x9000), dw=0x100000 * (at + 1) + 256) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the views are no memory of a GPU")
def test_rms_norm_takes_views_that_are_allowed(lib):
    for out, total in ((0, 1), (1, 0), (0, 3), (2, 0), (2, 1)):
        assert _norm(lib, _nspec(), [_m(0), _m(1), _m(out), _m(total)]) in (UNSUPPORTED, CUDA)
    for dx in range(3):
        assert _norm_back(lib, _nspec(), [_m(0), _m(1), _m(2), _m(dx)]) in (UNSUPPORTED, CUDA)
    assert _norm(lib, _nspec(), [_m(0), NONE, _m(0), NONE]) in (UNSUPPORTED, CUDA)


def test_rms_norm_residual_and_sum_come_together(lib):
    assert _norm(lib, _nspec(), [_m(0), NONE, _m(2), _m(3)]) == INVALID
    assert _norm(lib, _nspec(), [_m(0), _m(1), _m(2), NONE]) == INVALID
    assert _norm_back(lib, _nspec(weight=0x1000)) == INVALID
    assert _norm_back(lib, _nspec(), dw=0x1000) == INVALID


def test_rms_norm_sizes_and_workspace(lib):
    assert _norm(lib, _nspec(tokens=0)) == OK and _norm8(lib, _nspec(tokens=0)) == OK
    assert _norm_back(lib, _nspec(tokens=0)) == OK
    for bad in (dict(ws=None), dict(ws=WS + 16), dict(n=256)):
        assert _norm_back(lib, _nspec(), **bad) == WORKSPACE
    f = lib.muon_rms_norm_workspace_bytes
    assert f(64) == 256 + 304 * 64 * 4
    assert [f(b) for b in (0, -8, 12, 16392)] == [0] * 4


# ------------------------------------------------------------ embedding
def _espec(**kw):
    a = dict(tokens=16, rows=16, dim=64, id_bytes=8, ids=0x900000, scale=1.0)
    a.update(kw)
    return muon._EmbeddingSpec(*[a[n] for n, _ in muon._EmbeddingSpec._fields_])


def _emb(lib, spec, views=None, td=1, od=1):
    v = views or [_m(0), _m(1)]
    return lib.muon_embedding(spec, td, v[0], od, v[1], None)


def _emb_back(lib, spec, views=None, gd=1, od=1, ws=WS, n=WS_BYTES):
    v = views or [_m(0), _m(1)]
    return lib.muon_embedding_backward(spec, gd, v[0], od, v[1], ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(tokens=2 ** 31 - 1), dict(rows=0), dict(rows=(1 << 30) + 1), dict(dim=0),
    dict(dim=60), dict(dim=65544), dict(id_bytes=2), dict(ids=None), dict(ids=0x900004),
    dict(id_bytes=4, ids=0x900002), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_embedding_refuses_a_bad_spec(lib, kw):
    assert _emb(lib, _espec(**kw)) == INVALID
    assert _emb_back(lib, _espec(**kw)) == INVALID
    assert _emb(lib, None) == INVALID and _emb_back(lib, None) == INVALID


@pytest.mark.parametrize("kw", BAD_VIEWS)
def test_embedding_refuses_a_bad_view(lib, kw):
    for at in range(2):
        v = [_m(i) for i in range(2)]
        v[at] = _bad(v[at], kw)
        assert _emb(lib, _espec(), v) == INVALID
        assert _emb_back(lib, _espec(), v) == INVALID


def test_embedding_types_overlap_and_workspace(lib):
    for bad in (-1, 2):
        assert _emb(lib, _espec(), td=bad) == INVALID and _emb(lib, _espec(), od=bad) == INVALID
        assert _emb_back(lib, _espec(), gd=bad) == INVALID
        assert _emb_back(lib, _espec(), od=bad) == INVALID
    for shift in (0, 128, -15 * 128):
        assert _emb(lib, _espec(), [_m(0), _m(0, shift=shift)]) == INVALID
        assert _emb_back(lib, _espec(), [_m(0), _m(0, shift=shift)]) == INVALID
    assert _emb(lib, _espec(ids=0x200000 + 64)) == INVALID
    assert _emb_back(lib, _espec(ids=0x200000 + 64)) == INVALID
    assert _emb(lib, _espec(tokens=0, ids=None)) == OK
    for bad in (dict(ws=None), dict(ws=WS + 16), dict(n=256)):
        assert _emb_back(lib, _espec(), **bad) == WORKSPACE
    f = lib.muon_embedding_workspace_bytes
    assert f(32, 64) == 512 + 4 * 256               # one chunk: no pieces
    assert f(33, 64) == 512 + 4 * 256 + 2 * 2 * 64 * 4
    assert [f(*b) for b in ((-1, 64), (4, 0), (4, 12), (2 ** 31 - 1, 64))] == [0] * 4


# ------------------------------------------------------------ clipping
def _clip(lib, tensors, max_norm=1.0, eps=1e-6, norm=0x9000, ws=WS, n=WS_BYTES, count=None):
    arr = (muon._GradTensor * max(1, len(tensors)))(*[muon._GradTensor(*t) for t in tensors])
    return lib.muon_clip_grad_norm(arr, len(tensors) if count is None else count, max_norm, eps,
                                   norm, ws, n, None)


def test_clip_refusals(lib):
    good = (0x1000, 0x1000, 64, 1, 1)
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0),
               dict(eps=float("nan")), dict(norm=None), dict(norm=0x9002), dict(count=-1)):
        assert _clip(lib, [good], **kw) == INVALID, kw
    for bad in ((None, 0x1000, 64, 1, 1), (0x1008, 0x1008, 64, 1, 1), (0x1000, None, 64, 1, 1),
                (0x1000, 0x2008, 64, 1, 1), (0x1000, 0x1000, -1, 1, 1), (0x1000, 0x1000, 64, 2, 1),
                (0x1000, 0x2000, 64, 1, 3), (0x1000, 0x1000, 64, 1, 0), (0x1000, 0x1040, 64, 1, 1)):
        assert _clip(lib, [bad]) == INVALID, bad
        assert _clip(lib, [good, bad]) == INVALID
    for bad in (dict(ws=None), dict(ws=WS + 16), dict(n=256)):
        assert _clip(lib, [good], **bad) == WORKSPACE
    assert lib.muon_clip_workspace_bytes(-1) == 0
    assert lib.muon_clip_workspace_bytes(64) == 256 + 608 * 8
    assert lib.muon_clip_workspace_bytes(65) == 256 + 2 * 608 * 8


# ------------------------------------------------------------ binding
def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: muon.linear(x, x), lambda: muon.linear_backward(x, x, x),
                 lambda: muon.rms_norm(x), lambda: muon.rms_norm_fp8(x),
                 lambda: muon.rms_norm_backward(x, x), lambda: muon.embedding(ids, x),
                 lambda: muon.embedding_backward(x, ids, 4), lambda: muon.clip_grad_norm([x], 1.0),
                 lambda: muon.grad_norm([x])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        muon.clip_grad_norm([], 1.0)


def test_structures_match_the_header(lib):
    assert ctypes.sizeof(muon._Matrix) == 16
    assert ctypes.sizeof(muon._LinearSpec) == 24
    assert ctypes.sizeof(muon._RmsNormSpec) == 24
    assert ctypes.sizeof(muon._EmbeddingSpec) == 32
    assert ctypes.sizeof(muon._GradTensor) == 32


def test_binding_refuses_sizes_beyond_31_bits(lib, monkeypatch):
    # (as C ints they would be small ones: 2^32 + 8 rows would be 8)
    monkeypatch.setattr(muon, "_cuda_device", lambda t, name: None)
    many = (1 << 32) + 8
    tall, wide, small = (torch.empty(shape, dtype=torch.bfloat16, device="meta")
                         for shape in ((many, 8), (8, many), (8, 8)))
    ids = torch.zeros(8, dtype=torch.int64)
    for call in (lambda: muon._linear_spec(tall, small, None, None),
                 lambda: muon._linear_spec(small, tall, None, None),
                 lambda: muon._linear_spec(wide, wide, None, None),
                 lambda: muon._norm_spec(tall, "x", None, 0.0),
                 lambda: muon._norm_spec(wide, "x", None, 0.0),
                 lambda: muon._embedding_spec(ids, many, 8, 1.0),
                 lambda: muon._embedding_spec(ids, -1, 8, 1.0),
                 lambda: muon._embedding_spec(ids, 8, many, 1.0),
                 lambda: muon.linear_workspace_bytes(many, 8, 8),
                 lambda: muon.rms_norm_workspace_bytes(many),
                 lambda: muon.embedding_workspace_bytes(many, 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_clip_norm_apart_and_outputs_without_clipping(lib):
    good, out = (0x1000, 0x1000, 64, 1, 1), (0x1000, 0x2000, 64, 1, 0)
    for norm in (0x1000, 0x107c, 0x2000, 0x20fc):
        assert _clip(lib, [out], norm=norm) == INVALID
    # an infinite max_norm: outs other than the gradients are written, and so have to be valid
    inf = float("inf")
    for bad in ((0x4000, 0x5008, 64, 1, 0), (0x4000, 0x4040, 64, 1, 1), (0x4000, None, 64, 1, 0)):
        assert _clip(lib, [out, bad], max_norm=inf) == INVALID
    for one in ([good], [good, (0x4000, None, 64, 1, 0)]):
        assert _clip(lib, one, max_norm=inf, n=256) == WORKSPACE
