"""The example block: its gradients against the float64 chain rule, and that it learns."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import newton_schulz_step_gb300 as muon
from oracle import attention_oracle as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location(
        "attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def f64(t):
    return t.detach().double().cpu().numpy()


def test_block_gradients_match_the_chain_rule(ex):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(3)
    block = ex.Block(gen, dev)
    block.norm = [1 + 0.2 * torch.randn(ex.HEAD, generator=gen, device=dev) for _ in range(2)]
    lengths = [60, 1, 139]
    cu = torch.tensor([0, 60, 61, 200], dtype=torch.int32, device=dev)
    pos = torch.cat([torch.arange(n) for n in lengths]).int().to(dev)
    tables = muon.rope_tables(139, ex.HEAD, device=dev)
    x = torch.randn(200, ex.D, generator=gen, device=dev).bfloat16()
    dy = torch.randn(200, ex.D, generator=gen, device=dev).bfloat16()
    y, saved = block.forward(x, pos, cu, tables)
    grads, norm_grads = block.backward(dy, saved, x, pos, cu, tables)
    # the same in float64, from the bf16 weights the block multiplies with
    X, DY = f64(x), f64(dy)
    W = [f64(w.bfloat16()) for w in block.w]
    N = [f64(n) for n in block.norm]
    C, S, P, CU = f64(tables[0]), f64(tables[1]), pos.cpu().numpy(), cu.cpu().numpy()
    q, k, v = (np.reshape(X @ w.T, (200, -1, ex.HEAD)) for w in W[:3])
    qn, kn = ref.norm_rope(q, N[0], C, S, P), ref.norm_rope(k, N[1], C, S, P)
    o, lse = ref.attention(qn, kn, v, CU)
    want_y = o.reshape(200, -1) @ W[3].T
    do = np.reshape(DY @ W[3], (200, ex.Q_HEADS, ex.HEAD))
    dqn, dkn, dv = ref.attention_backward(do, qn, kn, v, o, lse, CU)
    dq, dnq = ref.norm_rope_backward(dqn, q, N[0], C, S, P)
    dk, dnk = ref.norm_rope_backward(dkn, k, N[1], C, S, P)
    want = [*(g.reshape(200, -1).T @ X for g in (dq, dk, dv)), DY.T @ o.reshape(200, -1)]
    # about six bf16 roundings on the way (2^-9 rms each, added at random), with room: 2 %
    for got, w in zip([y, *grads, *norm_grads], [want_y, *want, dnq, dnk]):
        assert np.linalg.norm(f64(got) - w) <= 0.02 * np.linalg.norm(w)


def test_example_learns(ex):
    losses = ex.main(steps=25)
    assert np.isfinite(losses).all()
    assert losses[-1] < 0.75 * losses[0]
