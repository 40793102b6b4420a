"""The example's training step: the gradients of every weight against 64-bit automatic
differentiation of the same model, the clipping, and that the steps run."""

import importlib.util
import math
import os
import threading

import pytest
import torch

import newton_schulz_step_gb300 as muon

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("gpt_step",
                                                  os.path.join(ROOT, "examples", "gpt_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _model64(ex, model, ids, targets, pos, lengths, tables):
    """Loss of the model in 64 bits on the CPU, and its leaves (the bf16 weights that the products
    take, in the order of the gradients)."""
    leaves = [w.bfloat16().double().cpu() for w in model.matrices]
    leaves += [model.table.double().cpu(), model.head.bfloat16().double().cpu()]
    leaves += [w.double().cpu() for w in model.norms]
    leaves = [w.requires_grad_(True) for w in leaves]
    qkv_w, proj_w, fc_w, out_w, table, head = leaves[:6]
    norms = leaves[6:]

    def norm(x, w, eps=muon.NORM_EPS):
        return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w

    cos, sin = (t.double().cpu()[pos.cpu().long()][:, None] for t in tables)

    def rotate(x):
        a, b = x.chunk(2, -1)
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    x0 = ex.SCALE * table[ids.cpu()]
    qkv = (norm(x0, norms[0]) @ qkv_w.T).unflatten(1, (-1, ex.HEAD))
    q, k, v = qkv.split((ex.Q_HEADS, ex.KV_HEADS, ex.KV_HEADS), dim=1)
    q, k = rotate(norm(q, norms[3], muon.ROPE_EPS)), rotate(norm(k, norms[4], muon.ROPE_EPS))
    k, v = (t.repeat_interleave(ex.Q_HEADS // ex.KV_HEADS, 1) for t in (k, v))
    parts = []
    for a, b, c in zip(*(t.split(lengths) for t in (q, k, v))):
        s = torch.einsum("ihd,jhd->hij", a, b) / math.sqrt(ex.HEAD)
        s = s.masked_fill(torch.ones(len(a), len(a), dtype=torch.bool).triu(1), -math.inf)
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), c))
    x1 = torch.cat(parts).flatten(1) @ proj_w.T + x0
    x2 = (norm(x1, norms[1]) @ fc_w.T).clamp_min(0).square() @ out_w.T + x1
    logits = norm(x2, norms[2]) @ head.T
    return torch.nn.functional.cross_entropy(logits, targets.cpu()), leaves


def test_gradients_match_automatic_differentiation(ex):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(3)
    model = ex.Model(gen, dev)
    model.norms = [1 + 0.2 * torch.randn(w.shape, generator=gen, device=dev) for w in model.norms]
    ids, targets, pos, cu = ex.batch(gen, dev)
    tables = muon.rope_tables(max(ex.LENGTHS), ex.HEAD, device=dev)
    logits, saved = model.forward(ids, pos, cu, tables)
    loss, dlogits = ex.loss_and_gradient(logits, targets)
    grads, rest = model.backward(dlogits, saved, ids, pos, cu, tables)
    want, leaves = _model64(ex, model, ids, targets, pos, ex.LENGTHS, tables)
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 1e-2
    # up to about 25 roundings to bf16 on the way (2^-9 rms each, added at random: 1 %), with room
    for got, leaf in zip(grads + rest, leaves):
        g = got.double().cpu()
        assert (g - leaf.grad).norm() <= 0.04 * leaf.grad.norm(), tuple(leaf.shape)
    # the norm of them all, and the clipped ones
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads + rest))
    before = [g.clone() for g in grads + rest]
    norm = float(muon.clip_grad_norm(grads + rest, 0.5 * total))
    assert abs(norm / total - 1) <= 2.0 ** -15
    for g, b in zip(grads + rest, before):
        assert (g.double() - 0.5 * b.double()).norm() <= 2.0 ** -8 * b.double().norm()


def test_example_runs(ex):
    for loss, norm in ex.main(steps=3):
        assert math.isfinite(loss) and math.isfinite(norm) and norm > 0


def test_a_step_is_the_same_in_every_run(ex):
    assert ex.main(steps=2) == ex.main(steps=2)


def test_threads_with_calls_of_every_kind_on_one_stream():
    # calls of several launches hand over through the one workspace of the stream
    gen = torch.Generator().manual_seed(9)

    def draw(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen).to(dtype).cuda()

    x, w, dy = draw(300, 1032), draw(264, 1032), draw(300, 264)
    h, dh, nw = draw(500, 1024), draw(500, 1024), draw(1024, dtype=torch.float32)
    ids, de = torch.randint(0, 97, (1500,), generator=gen).cuda(), draw(1500, 264)
    grads = [draw(n) for n in (70001, 33, 4096)]
    q, k, v, do = draw(257, 4, 64), draw(257, 2, 64), draw(257, 2, 64), draw(257, 4, 64)
    out, lse = muon.attention(q, k, v)
    tables = muon.rope_tables(257, 64)
    qw, kw = draw(64, dtype=torch.float32), draw(64, dtype=torch.float32)

    def clip():
        outs = [torch.empty_like(g) for g in grads]
        return [muon.clip_grad_norm(grads, 0.5, outs=outs), *outs]

    calls = [
        lambda: [muon.linear(x, w), *muon.linear_backward(dy, x, w, bias=True)],
        lambda: muon.rms_norm_backward(dh, h, nw),
        lambda: [muon.embedding_backward(de, ids, 101)],
        clip,
        lambda: muon.attention_backward(do, q, k, v, out, lse),
        lambda: muon.qk_norm_rope_backward(do, k, q, k, *tables, q_weight=qw, k_weight=kw),
    ]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    stream, start = torch.cuda.Stream(), threading.Barrier(len(calls))
    got = [[] for _ in calls]

    def work(i):
        with torch.cuda.stream(stream):
            start.wait()
            for _ in range(60):
                got[i].append(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert muon.workspace_status(None) == 0
    for g, r in zip(got, want):
        assert len(g) == 60
        assert all(torch.equal(a, b) for one in g for a, b in zip(one, r))
