"""A training step of a small GPT with the library's kernels, from token ids to updated weights.

One block (d = 256, 4 query heads on 2 key/value heads, relu^2 MLP of 512) over documents packed
along the tokens:

  x0      = embedding(ids)
  n1      = rms_norm(x0)
  q, k, v = n1 W_qkv^T, q and k normed and rotated, o = attention(q, k, v)
  n2, x1  = rms_norm(o W_proj^T + x0)                 the residual added inside the norm
  x2      = relu^2(n2 W_fc^T) W_out^T + x1            the residual added inside the product
  logits  = rms_norm(x2) W_head^T, cross entropy with the next token

then every gradient through the operators' backward passes, all of them clipped by their common
norm, a Muon step on the matrices of the block and an Adam step on the embedding, the head and the
norms' weights.

Run:  python examples/gpt_step.py [steps]
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_step_gb300 as muon  # noqa: E402

VOCAB, D, Q_HEADS, KV_HEADS, HEAD, HIDDEN = 1000, 256, 4, 2, 64, 512
LENGTHS = [300, 33, 512, 179]
SCALE = D ** 0.5                                   # of the embedding


class Model:
    def __init__(self, gen, device):
        def randn(*shape, std):
            return torch.randn(*shape, generator=gen, device=device) * std

        # fp32 master weights: the matrices that Muon trains, and the rest
        heads = (Q_HEADS + 2 * KV_HEADS) * HEAD
        self.matrices = [randn(heads, D, std=D ** -0.5),
                         randn(D, Q_HEADS * HEAD, std=(Q_HEADS * HEAD) ** -0.5),
                         randn(HIDDEN, D, std=D ** -0.5), randn(D, HIDDEN, std=HIDDEN ** -0.5)]
        self.table = randn(VOCAB, D, std=D ** -0.5)
        self.head = randn(VOCAB, D, std=D ** -0.5)
        # of the three norms along d, and of the query and key heads
        self.norms = [torch.ones(n, device=device) for n in (D, D, D, HEAD, HEAD)]

    def others(self):
        return [self.table, self.head, *self.norms]

    def forward(self, ids, pos, cu, tables):
        qkv_w, proj_w, fc_w, out_w = (w.bfloat16() for w in self.matrices)
        head_w = self.head.bfloat16()
        x0 = muon.embedding(ids, self.table, scale=SCALE)
        n1, _ = muon.rms_norm(x0, self.norms[0])
        q, k, v = muon.linear(n1, qkv_w).unflatten(1, (-1, HEAD)).split(
            (Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
        qn, kn = muon.qk_norm_rope(q, k, *tables, q_weight=self.norms[3], k_weight=self.norms[4],
                                   positions=pos)
        o, lse = muon.attention(qn, kn, v, cu)
        n2, x1 = muon.rms_norm(muon.linear(o.flatten(1), proj_w), self.norms[1], residual=x0)
        f, z = muon.linear(n2, fc_w, activation="relu2", save_preact=True)
        x2 = muon.linear(f, out_w, residual=x1)
        n3, _ = muon.rms_norm(x2, self.norms[2])
        logits = muon.linear(n3, head_w)
        saved = (qkv_w, proj_w, fc_w, out_w, head_w, x0, n1, q, k, v, qn, kn, o, lse, n2, x1, f, z,
                 x2, n3)
        return logits, saved

    def backward(self, dlogits, saved, ids, pos, cu, tables):
        """Gradients of the matrices, and of the embedding, the head and the norms' weights."""
        (qkv_w, proj_w, fc_w, out_w, head_w, x0, n1, q, k, v, qn, kn, o, lse, n2, x1, f, z, x2,
         n3) = saved
        dn3, d_head, _ = muon.linear_backward(dlogits, n3, head_w)
        dx2, d_norm2 = muon.rms_norm_backward(dn3, x2, self.norms[2])
        df, d_out, _ = muon.linear_backward(dx2, f, out_w)
        dn2, d_fc, _ = muon.linear_backward(df, n2, fc_w, activation="relu2", preact=z)
        dx1, d_norm1 = muon.rms_norm_backward(dn2, x1, self.norms[1], dresidual=dx2)
        do, d_proj, _ = muon.linear_backward(dx1, o.flatten(1), proj_w)
        d_qkv = torch.empty(len(ids), Q_HEADS + 2 * KV_HEADS, HEAD, dtype=torch.bfloat16,
                            device=ids.device)
        dq, dk, dv = d_qkv.split((Q_HEADS, KV_HEADS, KV_HEADS), dim=1)
        dqn, dkn, _ = muon.attention_backward(do.unflatten(1, (-1, HEAD)), qn, kn, v, o, lse, cu,
                                              dv=dv)
        _, _, d_nq, d_nk = muon.qk_norm_rope_backward(
            dqn, dkn, q, k, *tables, q_weight=self.norms[3], k_weight=self.norms[4],
            positions=pos, dq=dq, dk=dk)
        dn1, d_w, _ = muon.linear_backward(d_qkv.flatten(1), n1, qkv_w)
        dx0, d_norm0 = muon.rms_norm_backward(dn1, x0, self.norms[0], dresidual=dx1)
        d_table = muon.embedding_backward(dx0, ids, VOCAB, scale=SCALE)
        return [d_w, d_proj, d_fc, d_out], [d_table, d_head, d_norm0, d_norm1, d_norm2, d_nq, d_nk]


def batch(gen, device):
    """Token ids of the packed documents, the next tokens, positions and offsets."""
    ids = torch.randint(0, VOCAB, (sum(LENGTHS) + 1,), generator=gen, device=device)
    ids = ids.square() // VOCAB                    # some tokens are frequent
    pos = torch.cat([torch.arange(n) for n in LENGTHS]).int().to(device)
    cu = torch.tensor([0, *torch.tensor(LENGTHS).cumsum(0).tolist()], dtype=torch.int32,
                      device=device)
    return ids[:-1].contiguous(), ids[1:], pos, cu


def loss_and_gradient(logits, targets):
    p = torch.log_softmax(logits.float(), 1)
    d = p.exp()
    rows = torch.arange(len(targets), device=targets.device)
    d[rows, targets] -= 1
    return -p[rows, targets].mean(), (d / len(targets)).bfloat16()


def main(steps: int = 20, seed: int = 0):
    """Losses and gradient norms of the steps."""
    device = torch.device("cuda")
    gen = torch.Generator(device=device).manual_seed(seed)
    model = Model(gen, device)
    bufs = [torch.zeros_like(w) for w in model.matrices]
    moments = [(torch.zeros_like(w), torch.zeros_like(w)) for w in model.others()]
    ids, targets, pos, cu = batch(gen, device)
    tables = muon.rope_tables(max(LENGTHS), HEAD, device=device)
    out = []
    for step in range(1, steps + 1):
        logits, saved = model.forward(ids, pos, cu, tables)
        loss, dlogits = loss_and_gradient(logits, targets)
        grads, rest = model.backward(dlogits, saved, ids, pos, cu, tables)
        norm = muon.clip_grad_norm(grads + rest, 1.0)
        muon.step_grouped(list(zip(model.matrices, grads, bufs)), momentum=0.9, lr=0.02,
                          weight_decay=0.0)
        muon.adam_step([(w, g, *m) for w, g, m in zip(model.others(), rest, moments)], step,
                       lr=1e-3)
        out.append((float(loss), float(norm)))
    return out


if __name__ == "__main__":
    for i, (loss, norm) in enumerate(main(int(sys.argv[1]) if len(sys.argv) > 1 else 20)):
        print(f"step {i:3d}  loss {loss:.4f}  gradient norm {norm:.4f}")
