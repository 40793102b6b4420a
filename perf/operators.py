"""Cases, plain forms and exact results of the attention-path operators.

The operators are the two halves of a GPT block's attention path, the block whose
weights the Muon step trains:

  norm_rope   RMS norm of every query and key head and the rotary position
              embedding, in one pass (`qk_norm_rope`, `qk_norm_rope_backward`)
  attention   causal attention over packed sequences of different lengths with
              grouped key/value heads (`attention`, `attention_backward`)

With `own` false, `run` computes a case from elementary torch operations in 32 bits;
with `own` true, it calls the package.  `exact` restates the definitions in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0


# ---------------------------------------------------------------- cases
def _norm_rope(name, direction, tokens, q_heads, k_heads, head_dim, *, rot_dim=None,
               dtype="bf16", interleaved=False, norm=True, weight=True, packed=True):
    return {"name": name, "op": "norm_rope", "direction": direction, "tokens": tokens,
            "q_heads": q_heads, "k_heads": k_heads, "head_dim": head_dim,
            "rot_dim": head_dim if rot_dim is None else rot_dim, "dtype": dtype,
            "interleaved": interleaved, "norm": norm, "weight": weight, "packed": packed}


def _attention(name, direction, lengths, q_heads, k_heads, head_dim, *, fused_v=True):
    # lengths as a text, so that a case holds plain values only
    return {"name": name, "op": "attention", "direction": direction,
            "lengths": ",".join(str(n) for n in lengths), "q_heads": q_heads,
            "k_heads": k_heads, "head_dim": head_dim, "fused_v": fused_v}


def listed():
    return [
        # one short evaluation prompt on the d = 512 model (8 heads, 4 key/value heads): latency
        _norm_rope("norm_rope-forward-short", "forward", 33, 8, 4, 64),
        # a forward pass of the d = 768 model over an odd number of tokens, weightless norm
        _norm_rope("norm_rope-forward-d768", "forward", 8191, 12, 12, 64, weight=False),
        # the largest forward: the d = 4096 model, interleaved pairs
        _norm_rope("norm_rope-forward-d4096", "forward", 32768, 32, 8, 128, interleaved=True),
        # a training step of the d = 2048 model
        _norm_rope("norm_rope-backward-d2048", "backward", 16384, 16, 16, 128),
        # fp32 activations, a head of 96 rotated in part, odd heads and tokens
        _norm_rope("norm_rope-backward-fp32-partial", "backward", 5003, 9, 3, 96, rot_dim=64,
                   dtype="fp32", interleaved=True, packed=False),
        # one short evaluation prompt on the d = 512 model: latency
        _attention("attention-forward-short", "forward", [33], 8, 4, 64, fused_v=False),
        # documents packed to a d = 768 evaluation batch
        _attention("attention-forward-packed", "forward",
                   [1900, 37, 811, 2400, 5, 640, 1299, 1100], 12, 12, 64),
        # one long document on the d = 4096 model, grouped heads
        _attention("attention-forward-long", "forward", [16384], 32, 8, 128),
        # a training step of the d = 512 model, packed documents
        _attention("attention-training-d512", "training", [1024, 700, 324, 1500, 548], 8, 4, 64),
        # a training step of the d = 2048 model, packed documents
        _attention("attention-training-d2048", "training",
                   [2048, 1311, 977, 3000, 856], 16, 4, 128),
        # odd head size and head counts, lengths of one and zero
        _attention("attention-training-odd", "training", [1, 0, 127, 129, 1001, 790], 5, 5, 80),
        # the largest: a long document trained on the d = 4096 model
        _attention("attention-training-long", "training", [8192], 32, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    if rng.random() < 0.4:
        while True:
            group = rng.choice([1, 2, 3, 4])
            k_heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
            head_dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
            rot = head_dim if rng.random() < 0.7 else head_dim // 16 * 8
            case = _norm_rope(None, rng.choice(["forward", "backward"]),
                              _log_int(rng, 1, 32768), k_heads * group, k_heads, head_dim,
                              rot_dim=rot, dtype=rng.choice(["bf16", "bf16", "fp32"]),
                              interleaved=rng.random() < 0.5, norm=rng.random() < 0.85,
                              weight=rng.random() < 0.7, packed=rng.random() < 0.7)
            if work(case)["bytes"] <= 700e6:
                break
    else:
        while True:
            group = rng.choice([1, 2, 3, 4])
            k_heads = rng.choice([1, 2, 3, 4, 8, 12])
            direction = rng.choice(["forward", "training"])
            tokens = _log_int(rng, 1, 16384)
            lengths, left = [], tokens
            for _ in range(rng.choice([1, 1, 2, 5, 11]) - 1):
                n = min(left, _log_int(rng, 1, max(1, tokens)))
                lengths.append(n)
                left -= n
            if left:
                lengths.append(left)
            if rng.random() < 0.2:
                lengths.insert(rng.randrange(len(lengths) + 1), 0)
            case = _attention(None, direction, lengths, k_heads * group, k_heads,
                              rng.choice([32, 64, 64, 80, 96, 128, 128]),
                              fused_v=rng.random() < 0.7)
            if work(case)["flops"] <= 1.9e12:
                break
    del case["name"]
    return case


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


# ---------------------------------------------------------------- inputs
def _tables(length, rot_dim):
    """cos and sin of position * base^(-2i / rot_dim), [length, rot_dim / 2] fp32."""
    inv = ROPE_BASE ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    ang = torch.arange(length, dtype=torch.float64)[:, None] * inv[None, :]
    return ang.cos().float().cuda(), ang.sin().float().cuda()


def _heads_of(buf, first, heads, head_dim):
    """[tokens, heads, head_dim] view of the columns of a fused projection's output."""
    return buf[:, first * head_dim:(first + heads) * head_dim].unflatten(1, (heads, head_dim))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    hq, hk, d = case["q_heads"], case["k_heads"], case["head_dim"]
    st = {"case": dict(case)}
    if case["op"] == "norm_rope":
        t, rot = case["tokens"], case["rot_dim"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        # q and k are columns of the fused q, k, v projection's output
        qkv = (0.7 * randn(t, (hq + 2 * hk) * d)).to(dt)
        st["q"], st["k"] = _heads_of(qkv, 0, hq, d), _heads_of(qkv, hq, hk, d)
        if case["packed"]:
            # positions restart with each of the documents packed along the tokens
            docs = min(t, 7)
            cuts = torch.randperm(t - 1, generator=gen, device="cuda")[:docs - 1].sort()[0] + 1
            start = torch.zeros(t, dtype=torch.int64, device="cuda")
            start[cuts] = cuts
            pos = torch.arange(t, device="cuda") - start.cummax(0)[0]
            st["positions"] = pos.to(torch.int32)
        else:
            st["positions"] = None
        st["cos"], st["sin"] = _tables(t, rot)
        weighted = case["norm"] and case["weight"]
        st["q_weight"] = 1.0 + 0.2 * randn(d) if weighted else None
        st["k_weight"] = 1.0 + 0.2 * randn(d) if weighted else None
        if case["direction"] == "backward":
            st["dq"] = (1e-2 * randn(t, hq, d)).to(dt)
            st["dk"] = (1e-2 * randn(t, hk, d)).to(dt)
        return st
    lengths = _lengths(case)
    t = sum(lengths)

    # queries and keys as the norm leaves them: unit mean square, times a weight
    def normed(heads, w):
        x = randn(t, heads, d)
        return (w * x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(torch.bfloat16)

    st["q"], st["k"] = normed(hq, 1.3), normed(hk, 1.1)
    if case["fused_v"]:
        qkv = (0.7 * randn(t, (hq + 2 * hk) * d)).to(torch.bfloat16)
        st["v"] = _heads_of(qkv, hq + hk, hk, d)
    else:
        st["v"] = (0.7 * randn(t, hk, d)).to(torch.bfloat16)
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    st["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["direction"] == "training":
        st["do"] = (1e-2 * randn(t, hq, d)).to(torch.bfloat16)
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        return (_own_norm_rope if own else _plain_norm_rope)(state, case)
    return (_own_attention if own else _plain_attention)(state, case)


def _own_norm_rope(st, case):
    import newton_schulz_step_gb300 as muon
    kw = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], positions=st["positions"],
              norm=case["norm"], eps=EPS, interleaved=case["interleaved"])
    if case["direction"] == "forward":
        return muon.qk_norm_rope(st["q"], st["k"], st["cos"], st["sin"], **kw)
    out = muon.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["cos"], st["sin"],
                                     **kw)
    return tuple(x for x in out if x is not None)


def _own_attention(st, case):
    import newton_schulz_step_gb300 as muon
    o, lse = muon.attention(st["q"], st["k"], st["v"], st["cu_seqlens"])
    if case["direction"] == "forward":
        return o, lse
    dq, dk, dv = muon.attention_backward(st["do"], st["q"], st["k"], st["v"], o, lse,
                                         st["cu_seqlens"])
    return o, lse, dq, dk, dv


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] elements of each head rotated in pairs."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :half], r[..., half:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, rest), -1)


def _plain_norm_rope(st, case):
    pos, cos, sin = st["positions"], st["cos"], st["sin"]
    if pos is not None:
        cos, sin = cos[pos.long()], sin[pos.long()]
    cos, sin = cos[:, None, :], sin[:, None, :]
    outs, weights = [], []
    for name in ("q", "k"):
        x, w = st[name].float(), st[name + "_weight"]
        if case["norm"]:
            rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
            n = x * rstd
        if case["direction"] == "forward":
            y = x if not case["norm"] else n if w is None else n * w
            outs.append(_rotate(y, cos, sin, case["interleaved"]).to(st[name].dtype))
            continue
        g = _rotate(st["d" + name].float(), cos, -sin, case["interleaved"])
        if case["norm"]:
            if w is not None:
                weights.append((g * n).sum((0, 1)))
                g = g * w
            g = rstd * (g - n * (g * n).mean(-1, keepdim=True))
        outs.append(g.to(st[name].dtype))
    return tuple(outs + weights)


def _plain_attention(st, case):
    q, k, v = st["q"], st["k"], st["v"]
    t, hq, d = q.shape
    hk = k.shape[1]
    group, scale = hq // hk, 1.0 / math.sqrt(d)
    training = case["direction"] == "training"
    o = torch.empty_like(q)
    lse = torch.empty(hq, t, dtype=torch.float32, device=q.device)
    if training:
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dv = torch.empty_like(v, memory_format=torch.contiguous_format)
    t0 = 0
    for n in _lengths(case):
        t1 = t0 + n
        hidden = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
        # short sequences take all key heads in one product, long ones a few at a time
        step = max(1, min(hk, (1 << 28) // max(1, n * n * group)))
        for h0 in range(0, hk if n else 0, step):
            h1 = min(hk, h0 + step)
            qs = slice(h0 * group, h1 * group)
            qf = q[t0:t1, qs].float().unflatten(1, (-1, group)).permute(1, 2, 0, 3)
            kf = k[t0:t1, h0:h1].float().transpose(0, 1)[:, None]
            vf = v[t0:t1, h0:h1].float().transpose(0, 1)[:, None]
            s = (qf * scale) @ kf.transpose(-1, -2)
            s = s.masked_fill_(hidden, float("-inf"))
            m = s.amax(-1, keepdim=True)
            p = s.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l)
            of = p @ vf
            o[t0:t1, qs] = of.permute(2, 0, 1, 3).flatten(1, 2).to(o.dtype)
            lse[qs, t0:t1] = (m + l.log()).squeeze(-1).flatten(0, 1)
            if not training:
                continue
            dof = st["do"][t0:t1, qs].float().unflatten(1, (-1, group)).permute(1, 2, 0, 3)
            dv[t0:t1, h0:h1] = (p.transpose(-1, -2) @ dof).sum(1).transpose(0, 1).to(dv.dtype)
            delta = (dof * of).sum(-1, keepdim=True)
            ds = (dof @ vf.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
            dq[t0:t1, qs] = (ds @ kf).permute(2, 0, 1, 3).flatten(1, 2).to(dq.dtype)
            dk[t0:t1, h0:h1] = (ds.transpose(-1, -2) @ qf).sum(1).transpose(0, 1).to(dk.dtype)
        t0 = t1
    return (o, lse, dq, dk, dv) if training else (o, lse)


# ---------------------------------------------------------------- work
def work(case):
    hq, hk, d = case["q_heads"], case["k_heads"], case["head_dim"]
    if case["op"] == "norm_rope":
        t, rot = case["tokens"], case["rot_dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        back = case["direction"] == "backward"
        elems = t * (hq + hk) * d
        # one read and one write of the heads (backward: also a read of the gradients),
        # the rows of the two tables, the positions, the weights and their gradients
        nbytes = elems * size * (3 if back else 2) + t * rot * 4 + (4 * t if case["packed"] else 0)
        if case["norm"] and case["weight"]:
            nbytes += 2 * d * 4 * (2 if back else 1)
        return {"bytes": nbytes, "flops": elems * (14 if back else 7)}
    lengths = _lengths(case)
    t = sum(lengths)
    pairs = sum(n * (n + 1) // 2 for n in lengths) * hq
    heads = t * (2 * hq + 2 * hk) * d * 2             # q, k, v in, o out
    stats = t * hq * 4 + 4 * (len(lengths) + 1)       # log-sum-exp out, offsets in
    if case["direction"] == "forward":
        return {"bytes": heads + stats, "flops": 4 * d * pairs}
    grads = t * (2 * hq + 2 * hk) * d * 2             # dout in, dq, dk, dv out
    return {"bytes": heads + stats + grads, "flops": 14 * d * pairs}


# ---------------------------------------------------------------- 64-bit results
def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_norm_rope if case["op"] == "norm_rope" else _exact_attention)(st, case)


def _exact_norm_rope(st, case):
    t, rot, d = case["tokens"], case["rot_dim"], case["head_dim"]
    pos = torch.arange(t, device="cuda") if st["positions"] is None else st["positions"].long()
    i = torch.arange(rot // 2, device="cuda")
    # pair i of a head is elements first[i], second[i]
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    c, s = st["cos"].double()[pos].unsqueeze(1), st["sin"].double()[pos].unsqueeze(1)
    grads, dws = [], []
    for name in ("q", "k"):
        x = st[name].double()
        w = torch.ones(d, dtype=torch.float64, device="cuda")
        if st[name + "_weight"] is not None:
            w = st[name + "_weight"].double()
        r = torch.ones_like(x[..., :1])
        if case["norm"]:
            r = (x.pow(2).sum(-1, keepdim=True) / d + EPS).pow(-0.5)
        if case["direction"] == "forward":
            n = x * r * w
            y = n.clone()
            y[..., first] = n[..., first] * c - n[..., second] * s
            y[..., second] = n[..., first] * s + n[..., second] * c
            grads.append(y)
            continue
        dy = st["d" + name].double()
        g = dy.clone()
        g[..., first] = dy[..., first] * c + dy[..., second] * s
        g[..., second] = dy[..., second] * c - dy[..., first] * s
        if not case["norm"]:
            grads.append(g)
            continue
        if st[name + "_weight"] is not None:
            dws.append((g * x * r).sum(1).sum(0))
        gw = g * w
        # d/dx of r(x) x w, with dr/dx = -r^3 x / d
        grads.append(r * gw - r.pow(3) * x * (gw * x).sum(-1, keepdim=True) / d)
    return tuple(grads + dws)


def _exact_attention(st, case):
    hq, hk, d = case["q_heads"], case["k_heads"], case["head_dim"]
    training = case["direction"] == "training"
    # the products in 64 bits run at about 1e12 operations a second
    if work(case)["flops"] * 2 > 8e12:
        return None
    q, k, v = (st[x].double().transpose(0, 1) for x in ("q", "k", "v"))
    t = q.shape[1]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(hq, t, d, **f64), torch.zeros(hq, t, **f64)
    dq, dk, dv = torch.zeros(hq, t, d, **f64), torch.zeros(hk, t, d, **f64), torch.zeros(
        hk, t, d, **f64)
    do = st["do"].double().transpose(0, 1) if training else None
    begin = 0
    for n in _lengths(case):
        for r0 in range(begin, begin + n, 2048):           # rows r0..r1 see keys begin..r1
            r1 = min(r0 + 2048, begin + n)
            rows = torch.arange(r0, r1, device="cuda")[:, None]
            cols = torch.arange(begin, r1, device="cuda")[None, :]
            for h in range(hq):
                g = h // (hq // hk)
                kk, vv = k[g, begin:r1], v[g, begin:r1]
                s = torch.where(cols <= rows, q[h, r0:r1] @ kk.T / math.sqrt(d), -math.inf)
                z = torch.logsumexp(s, 1)
                p = torch.exp(s - z[:, None])
                out = p @ vv
                o[h, r0:r1], lse[h, r0:r1] = out, z
                if training:
                    g_out = do[h, r0:r1]
                    dv[g, begin:r1] += p.T @ g_out
                    ds = p * (g_out @ vv.T - (g_out * out).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[h, r0:r1] = ds @ kk
                    dk[g, begin:r1] += ds.T @ q[h, r0:r1]
        begin += n
    res = (o.transpose(0, 1), lse)
    if training:
        res += tuple(x.transpose(0, 1) for x in (dq, dk, dv))
    return res
