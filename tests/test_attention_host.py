"""Host-only checks of the attention path's C entry points and of the binding: refusals
before anything is enqueued, workspace sizes."""

import ctypes
import gc
import os
import random
import threading
import time
import weakref

import pytest
import torch

import newton_schulz_step_gb300 as muon

OK, INVALID, UNSUPPORTED, CUDA, TIMEOUT, WORKSPACE = range(6)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(muon.library_path()):
        from newton_schulz_step_gb300 import build
        build.build()
    return muon.load_library()


def _view(data=0x1000, ts=512, hs=64):
    return muon._Heads(data, ts, hs)


def _rope_spec(**kw):
    a = dict(dtype=1, tokens=16, q_heads=8, k_heads=4, head_dim=64, rot_dim=64, norm=1,
             interleaved=0, eps=1e-6, table_len=16, cos=0x1000, sin=0x2000, positions=None,
             q_weight=None, k_weight=None)
    a.update(kw)
    return muon._NormRope(*[a[n] for n, _ in muon._NormRope._fields_])


ROPE_BAD = [dict(dtype=2), dict(tokens=-1), dict(q_heads=-1), dict(q_heads=0, k_heads=0),
            dict(q_heads=70000), dict(head_dim=0), dict(head_dim=60), dict(head_dim=264),
            dict(rot_dim=-8), dict(rot_dim=72), dict(rot_dim=20), dict(norm=2),
            dict(interleaved=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(table_len=0),
            dict(table_len=15), dict(cos=None), dict(sin=None), dict(cos=0x1004),
            dict(q_weight=0x1004), dict(norm=0, q_weight=0x1000), dict(norm=0, k_weight=0x1000)]
VIEW_BAD = [dict(data=None), dict(data=0x1008), dict(ts=0), dict(ts=-512), dict(ts=516),
            dict(hs=4), dict(hs=0), dict(hs=-64)]


@pytest.mark.parametrize("kw", ROPE_BAD)
def test_norm_rope_refuses_a_bad_spec(lib, kw):
    v = _view()
    assert lib.muon_qk_norm_rope(_rope_spec(**kw), v, v, v, v, None) == INVALID
    assert lib.muon_qk_norm_rope_backward(_rope_spec(**kw), v, v, v, v, v, v, None, None, 0x10000,
                                          1 << 30, None) == INVALID


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("kw", VIEW_BAD)
def test_norm_rope_refuses_a_bad_view(lib, at, kw):
    views = [_view() for _ in range(4)]
    views[at] = _view(**kw)
    assert lib.muon_qk_norm_rope(_rope_spec(), *views, None) == INVALID


def test_norm_rope_refuses_overlapping_output_rows(lib):
    v = _view()
    # heads 64 apart but tokens only 256 apart: 8 heads of one token span 512
    assert lib.muon_qk_norm_rope(_rope_spec(), v, v, _view(ts=256), v, None) == INVALID
    assert lib.muon_qk_norm_rope(_rope_spec(), v, v, _view(hs=32), v, None) == INVALID
    # [heads, tokens, dim] storage is fine (refused later here, for want of a GPU)
    if not torch.cuda.is_available():
        assert lib.muon_qk_norm_rope(_rope_spec(), v, v, _view(ts=64, hs=1024), v, None) in (
            UNSUPPORTED, CUDA)


def test_norm_rope_sizes(lib):
    v = _view()
    assert lib.muon_qk_norm_rope(None, v, v, v, v, None) == INVALID
    assert lib.muon_qk_norm_rope(_rope_spec(tokens=0), v, v, v, v, None) == OK
    assert lib.muon_qk_norm_rope(_rope_spec(tokens=2 ** 31 - 1, table_len=2 ** 31 - 1), v, v, v, v,
                                 None) == UNSUPPORTED
    assert lib.muon_norm_rope_workspace_bytes(64) == 256 + 640 * 2 * 64 * 4
    for bad in (0, -8, 12, 264):
        assert lib.muon_norm_rope_workspace_bytes(bad) == 0


def test_norm_rope_backward_needs_its_workspace_and_gradients(lib):
    v = _view()

    def call(spec, dqw=None, dkw=None, ws=0x10000, n=1 << 30):
        return lib.muon_qk_norm_rope_backward(spec, v, v, v, v, v, v, dqw, dkw, ws, n, None)

    assert call(_rope_spec(), ws=None) == WORKSPACE
    assert call(_rope_spec(), ws=0x10010) == WORKSPACE
    assert call(_rope_spec(), n=4096) == WORKSPACE
    # a weight and its gradient come together
    assert call(_rope_spec(q_weight=0x1000)) == INVALID
    assert call(_rope_spec(), dkw=0x1000) == INVALID


def _attn_spec(**kw):
    a = dict(tokens=16, q_heads=8, kv_heads=4, head_dim=64, n_seqs=2, cu_seqlens=0x1000,
             scale=0.125)
    a.update(kw)
    return muon._AttentionSpec(*[a[n] for n, _ in muon._AttentionSpec._fields_])


def _attn(lib, spec, views=None, lse=0x1000, ws=0x10000, n=1 << 30):
    views = views or [_view()] * 4
    return lib.muon_attention(spec, *views, lse, ws, n, None)


def _attn_back(lib, spec, views=None, lse=0x1000, ws=0x10000, n=1 << 30):
    w = views or [_view()] * 8
    return lib.muon_attention_backward(spec, *w[:5], lse, *w[5:], ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(tokens=-1), dict(q_heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(q_heads=70000),
    dict(head_dim=0), dict(head_dim=60), dict(head_dim=136), dict(n_seqs=-1),
    dict(cu_seqlens=None), dict(cu_seqlens=0x1002), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=2 ** 31 - 1)])
def test_attention_refuses_a_bad_spec(lib, kw):
    assert _attn(lib, _attn_spec(**kw)) == INVALID
    assert _attn_back(lib, _attn_spec(**kw)) == INVALID


@pytest.mark.parametrize("kw", VIEW_BAD)
def test_attention_refuses_a_bad_view(lib, kw):
    for at in range(4):
        views = [_view() for _ in range(4)]
        views[at] = _view(**kw)
        assert _attn(lib, _attn_spec(), views) == INVALID
    for at in range(8):
        views = [_view() for _ in range(8)]
        views[at] = _view(**kw)
        assert _attn_back(lib, _attn_spec(), views) == INVALID


def test_attention_refuses_overlap_lse_and_workspace(lib):
    v, bad = _view(), _view(ts=256)
    assert _attn(lib, _attn_spec(), [v, v, v, bad]) == INVALID
    assert _attn_back(lib, _attn_spec(), [v] * 5 + [bad, v, v]) == INVALID
    assert _attn(lib, _attn_spec(), lse=None) == INVALID
    assert _attn_back(lib, _attn_spec(), lse=0x1004) == INVALID
    for call in (_attn, _attn_back):
        assert call(lib, None) == INVALID
        assert call(lib, _attn_spec(), ws=None) == WORKSPACE
        assert call(lib, _attn_spec(), ws=0x10010) == WORKSPACE
        assert call(lib, _attn_spec(), n=128) == WORKSPACE
        assert call(lib, _attn_spec(tokens=0)) == OK


def test_attention_workspace_bytes(lib):
    f = lib.muon_attention_workspace_bytes
    assert f(0, 8, 4, 64) >= 256
    assert f(1000, 8, 4, 64) <= f(2000, 8, 4, 64)
    for bad in ((-1, 8, 4, 64), (10, 8, 3, 64), (10, 0, 0, 64), (10, 8, 4, 65), (10, 8, 4, 256)):
        assert f(*bad) == 0


def test_binding_refuses_cpu_tensors(lib):
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        muon.attention(q, q, q)
    with pytest.raises(ValueError):
        muon.qk_norm_rope(q, q, c, c)


def test_rope_tables_scale_the_positions():
    c1, s1 = muon.rope_tables(64, 16, device="cpu")
    c2, s2 = muon.rope_tables(256, 16, scale=4.0, device="cpu")
    assert c1.shape == (64, 8) and c1.dtype == torch.float32
    assert torch.equal(c2[::4], c1) and torch.equal(s2[::4], s1)
    assert torch.equal(c1[0], torch.ones(8)) and torch.equal(s1[0], torch.zeros(8))
    assert ctypes.sizeof(muon._Heads) == 24


class _FakeWorkspace:
    """A Workspace without a device: its address is its own, and only while it lives."""

    def __init__(self, nbytes, device=None):
        self.nbytes = max(256, nbytes)
        self.buf = bytearray(8)
        self.ptr = id(self.buf)


@pytest.fixture
def default_workspaces(monkeypatch):
    monkeypatch.setattr(muon, "_stream_ws", {})
    monkeypatch.setattr(muon, "Workspace", _FakeWorkspace)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return muon._stream_ws


def test_an_outgrown_default_workspace_stays_alive(default_workspaces):
    # another thread may have looked its pointer up and be about to launch with it
    alive = []

    class Watched(_FakeWorkspace):
        def __init__(self, *args):
            super().__init__(*args)
            alive.append(weakref.ref(self))

    muon.Workspace = Watched                    # (undone by the fixture)
    for need in (300, 1000, 1001, 5000, 400):
        ptr, nbytes = muon._stream_workspace(None, need, 0, 7)[:2]
        assert nbytes >= need and ptr == alive[-1]().ptr
    gc.collect()
    assert len(alive) == 4 and all(ref() is not None for ref in alive)
    assert sum(ref().nbytes for ref in alive) < 2 * alive[-1]().nbytes


def test_threads_on_one_stream_share_one_default_workspace(default_workspaces):
    made, got, start = [], [], threading.Barrier(8)

    class Slow(_FakeWorkspace):
        def __init__(self, *args):
            super().__init__(*args)
            time.sleep(0.02)                    # a thread that also looks now finds none yet
            made.append(self)

    muon.Workspace = Slow

    def look_up():
        start.wait()
        got.append(muon._stream_workspace(None, 1000, 0, 7)[0])

    threads = [threading.Thread(target=look_up) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and got == [made[0].ptr] * 8


def test_a_captured_call_gets_a_workspace_of_its_own(default_workspaces, monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    cpu = torch.empty
    made = []

    def empty(n, dtype, device):
        made.append(cpu(n, dtype=dtype).fill_(255))       # as memory used before
        return made[-1]

    monkeypatch.setattr(torch, "empty", empty)
    first, second = (muon._stream_workspace(None, 1000, 0, 7) for _ in range(2))
    assert [x[0] for x in (first, second)] == [m.data_ptr() for m in made]
    assert len(made) == 2 and not default_workspaces
    for ptr, nbytes, owner in (first, second):
        assert nbytes == 1000 and owner.data_ptr() == ptr
        assert torch.count_nonzero(owner[:256]) == 0      # error word and tickets
    # the caller's own is used as it is
    ws = _FakeWorkspace(400)
    assert muon._stream_workspace(ws, 1000, 0, 7) == (ws.ptr, 400, ws)


def test_status_of_the_default_workspace(default_workspaces, monkeypatch):
    words = {}

    class Library:
        @staticmethod
        def muon_workspace_status(ptr, nbytes, handle, clear):
            assert nbytes >= 256 and handle == 7
            word = words.get(ptr, OK)
            if clear:
                words[ptr] = OK
            return word

    monkeypatch.setattr(muon, "load_library", lambda: Library)
    monkeypatch.setattr(muon, "_current_device", lambda: 0)
    assert muon.workspace_status(None, stream=7) == OK        # no call needed one yet
    first, second = (muon._stream_workspace(None, n, 0, 7)[0] for n in (300, 9000))
    assert muon.workspace_status(None, stream=7) == OK
    for ptr in (first, second):                               # also of a call before it grew
        words[ptr] = TIMEOUT
        assert muon.workspace_status(None, stream=7) == TIMEOUT
        assert muon.workspace_status(None, clear=True, stream=7) == TIMEOUT
        assert muon.workspace_status(None, stream=7) == OK


def _spread(n, ts=512):
    """n views that share nothing (16 tokens of 8 heads of 64)."""
    return [_view(0x100000 * (i + 1), ts) for i in range(n)]


@pytest.mark.parametrize("entry,outputs,inputs", [("fwd", [3], [0, 1, 2]),
                                                  ("bwd", [5, 6, 7], [0, 1, 2, 3, 4])])
def test_attention_refuses_outputs_over_inputs_and_each_other(lib, entry, outputs, inputs):
    call, n = (_attn, 4) if entry == "fwd" else (_attn_back, 8)
    lse = 0x8000000
    row = 2 * 64                                # bytes of a head
    for o in outputs:
        for other in inputs + [x for x in outputs if x != o]:
            at = 0x100000 * (other + 1)
            # the same view, one a token on, its last row, one that ends in its first row
            for shift in (0, 1024, 15 * 1024, -15 * 1024 - 3 * row):
                views = _spread(n)
                views[o] = _view(at + shift)
                assert call(lib, _attn_spec(), views, lse=lse) == INVALID, (o, other, shift)
    # log-sum-exps (8 heads of 16) inside a view
    for at in (inputs + outputs if entry == "fwd" else outputs):
        assert call(lib, _attn_spec(), _spread(n), lse=0x100000 * (at + 1) + 1024) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the views are no memory of a GPU")
def test_attention_takes_views_that_only_interleave(lib):
    # the columns of one tensor of 8 + 4 + 4 + 8 heads: q, k, v, out
    ts, head = 24 * 64, 128
    views = [_view(0x100000 + head * first, ts) for first in (0, 8, 12, 16)]
    assert _attn(lib, _attn_spec(), views, lse=0x8000000) in (UNSUPPORTED, CUDA)
    views[3] = _view(0x100000 + head * 15, ts)
    assert _attn(lib, _attn_spec(), views, lse=0x8000000) == INVALID
    # every third head each, as [tokens, heads, (q, k, out), dim]
    spec = _attn_spec(kv_heads=8)
    views = [_view(0x100000 + head * i, ts, 192) for i in (0, 1, 1, 2)]
    assert _attn(lib, spec, views, lse=0x8000000) in (UNSUPPORTED, CUDA)
    views[3] = _view(0x100000 + head, ts, 192)
    assert _attn(lib, spec, views, lse=0x8000000) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the views are no memory of a GPU")
def test_overlap_is_found_as_by_listing_the_bytes(lib):
    rng = random.Random(0)
    seen = set()
    for _ in range(4000):
        t, hq, hk = rng.choice([1, 2, 5]), rng.choice([1, 2, 4]), rng.choice([1, 2])
        hk = min(hk, hq)
        d = 8
        ts = 8 * rng.randint(1, 24)

        def rand(heads):
            hs = 8 * rng.randint(1, 6)
            return muon._Heads(0x100000 + 16 * rng.randint(0, 60), ts, hs), heads

        def rows(v, heads):
            hs = v.head_stride if heads > 1 else d
            tok = v.token_stride if t > 1 else heads * d
            return [v.data + 2 * (i * tok + h * hs) for i in range(t) for h in range(heads)]

        (q, _), (out, _) = rand(hq), rand(hq)
        far = _view(0x10000000, 512)
        a = sorted(rows(out, hq))
        if any(y - x < 2 * d for x, y in zip(a, a[1:])):
            continue                            # rows of the output overlap
        hs, tok = out.head_stride if hq > 1 else d, out.token_stride if t > 1 else hq * d
        inner, outer, n = (hs, tok, hq) if hs <= tok else (tok, hs, t)
        if t > 1 and hq > 1 and outer < inner * (n - 1) + d:
            continue                            # (its rows do, by the rule of one span a row)
        want = any(abs(x - y) < 2 * d for x in rows(q, hq) for y in a)
        spec = _attn_spec(tokens=t, q_heads=hq, kv_heads=hk, head_dim=d)
        got = _attn(lib, spec, [q, far, far, out], lse=0x20000000)
        assert (got == INVALID) == want, (t, hq, ts, q.data, q.head_stride, out.data, hs)
        seen.add((t, hq, want))
    assert len(seen) >= 15
