"""Train the attention half of a GPT block with the library's kernels.

One block (d = 512, 8 query heads on 4 key/value heads) learns to imitate another one of
random weights, on documents packed along the tokens.  A step is

  q, k, v = x W_qkv^T                       (fused projection; torch.matmul)
  q, k    = qk_norm_rope(q, k)              positions restart with each document
  o       = attention(q, k, v)
  y       = o W_proj^T
  gradients of |y - target|^2 / 2 through the same operators, written into one fused
  gradient of q, k, v, and a Muon step on c_q, c_k, c_v and proj, an Adam step on the
  norm weights.

Run:  python examples/attention_block.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_step_gb300 as muon  # noqa: E402

D, Q_HEADS, KV_HEADS, HEAD = 512, 8, 4, 64
LENGTHS = [700, 33, 1024, 291]


class Block:
    def __init__(self, gen, device):
        def randn(*shape):
            return torch.randn(*shape, generator=gen, device=device)

        # fp32 master weights: c_q, c_k, c_v, proj
        self.w = [randn(h * HEAD, D) * D ** -0.5 for h in (Q_HEADS, KV_HEADS, KV_HEADS)]
        self.w.append(randn(D, Q_HEADS * HEAD) * D ** -0.5)
        self.norm = [torch.ones(HEAD, device=device) for _ in range(2)]

    def forward(self, x, pos, cu, tables):
        w_qkv = torch.cat(self.w[:3]).bfloat16()
        qkv = (x @ w_qkv.T).unflatten(1, (Q_HEADS + 2 * KV_HEADS, HEAD))
        q, k, v = qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
        qn, kn = muon.qk_norm_rope(q, k, *tables, q_weight=self.norm[0], k_weight=self.norm[1],
                                   positions=pos)
        o, lse = muon.attention(qn, kn, v, cu)
        y = o.flatten(1) @ self.w[3].bfloat16().T
        return y, (w_qkv, q, k, v, qn, kn, o, lse)

    def backward(self, dy, saved, x, pos, cu, tables):
        """Gradients of the four matrices (bf16) and the two norm weights (fp32)."""
        w_qkv, q, k, v, qn, kn, o, lse = saved
        d_proj = dy.T @ o.flatten(1)
        do = (dy @ self.w[3].bfloat16()).unflatten(1, (Q_HEADS, HEAD))
        d_qkv = torch.empty(x.shape[0], Q_HEADS + 2 * KV_HEADS, HEAD, dtype=x.dtype,
                            device=x.device)
        dq, dk, dv = d_qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
        dqn, dkn, _ = muon.attention_backward(do, qn, kn, v, o, lse, cu, dv=dv)
        _, _, d_nq, d_nk = muon.qk_norm_rope_backward(
            dqn, dkn, q, k, *tables, q_weight=self.norm[0], k_weight=self.norm[1], positions=pos,
            dq=dq, dk=dk)
        d_w = d_qkv.flatten(1).T @ x
        return [*(g.contiguous() for g in d_w.split([w.shape[0] for w in self.w[:3]])), d_proj], [
            d_nq, d_nk]


def main(steps: int = 30, seed: int = 0):
    """Losses of the steps (half the mean square of y - target)."""
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    cu = torch.tensor([0, *torch.tensor(LENGTHS).cumsum(0).tolist()], dtype=torch.int32,
                      device=device)
    tokens = sum(LENGTHS)
    pos = torch.cat([torch.arange(n) for n in LENGTHS]).int().to(device)
    tables = muon.rope_tables(max(LENGTHS), HEAD, device=device)
    teacher, student = Block(gen, device), Block(gen, device)
    bufs = [torch.zeros_like(w) for w in student.w]
    moments = [(torch.zeros_like(w), torch.zeros_like(w)) for w in student.norm]
    losses = []
    for step in range(1, steps + 1):
        x = torch.randn(tokens, D, generator=gen, device=device).bfloat16()
        target, _ = teacher.forward(x, pos, cu, tables)
        y, saved = student.forward(x, pos, cu, tables)
        err = y.float() - target.float()
        losses.append(0.5 * float(err.square().mean()))
        grads, norm_grads = student.backward((err / tokens).bfloat16(), saved, x, pos, cu, tables)
        muon.step_grouped(list(zip(student.w, grads, bufs)), momentum=0.9, lr=0.02,
                          weight_decay=0.0)
        muon.adam_step([(w, g, *m) for w, g, m in zip(student.norm, norm_grads, moments)], step,
                       lr=1e-3)
    return losses


if __name__ == "__main__":
    out = main(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
    for i, loss in enumerate(out):
        if i % 5 == 0 or i + 1 == len(out):
            print(f"step {i:3d}  loss {loss:.4f}")
