"""Cases, plain forms and exact results of the operators around a GPT block's weights.

They are what a training step needs beside the attention path and the optimizer:

  linear     the product with a weight matrix, with bias, activation and residual in its
             epilogue, and its gradients (`linear`, `linear_backward`)
  rms_norm   the residual's addition and the RMS norm of the sum in one pass, with an output
             in 8 bits and its scales, and the gradients (`rms_norm`, `rms_norm_fp8`,
             `rms_norm_backward`)
  embedding  the lookup of token rows with a scale, and the table's gradient
             (`embedding`, `embedding_backward`)
  clip       the norm of all gradients together, and the gradients clipped by it
             (`ClipGradNorm`, prepared once like the optimizer's steps)

With `own` false, `run` computes a case from elementary torch operations in 32 bits;
with `own` true, it calls the package.  `exact` restates the definitions in 64 bits.
"""

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def _linear(name, direction, tokens, d_in, d_out, *, bias=False, activation="none",
            residual=False):
    return {"name": name, "op": "linear", "direction": direction, "tokens": tokens, "in": d_in,
            "out": d_out, "bias": bias, "activation": activation, "residual": residual}


def _rms_norm(name, direction, tokens, dim, *, dtype="bf16", residual=True, weight=True, group=0):
    return {"name": name, "op": "rms_norm", "direction": direction, "tokens": tokens, "dim": dim,
            "dtype": dtype, "residual": residual, "weight": weight, "group": group}


def _embedding(name, direction, tokens, rows, dim, *, scale=1.0, table="fp32"):
    return {"name": name, "op": "embedding", "direction": direction, "tokens": tokens,
            "rows": rows, "dim": dim, "scale": scale, "table": table}


def _clip(name, layers, width, hidden, rows, *, dtype="bf16", out="bf16"):
    return {"name": name, "op": "clip", "layers": layers, "width": width, "hidden": hidden,
            "rows": rows, "dtype": dtype, "out": out}


def listed():
    return [
        # one token through the MLP's first matrix of the d = 4096 model
        _linear("linear-forward-token", "forward", 1, 4096, 11008, activation="relu2"),
        # a long evaluation batch through the MLP's second matrix, added to the residual stream
        _linear("linear-forward-d4096", "forward", 8192, 11008, 4096, residual=True),
        # a training step of the MLP's first matrix of the d = 2048 model
        _linear("linear-training-d2048", "training", 8192, 2048, 8192, activation="relu2"),
        # odd tokens and widths, every part of the epilogue at once
        _linear("linear-training-odd", "training", 1003, 520, 1000, bias=True, activation="gelu",
                residual=True),
        # one short evaluation prompt on the d = 512 model: latency
        _rms_norm("rms-norm-forward-short", "forward", 33, 512),
        # the input of an 8-bit product, a scale for each 128 columns, d = 4096 model
        _rms_norm("rms-norm-8-bit-d4096", "8-bit", 16384, 4096, group=128),
        # a training step of the d = 2048 model
        _rms_norm("rms-norm-training-d2048", "training", 16384, 2048),
        # an evaluation batch of the GPT-2 124M model
        _embedding("embedding-forward-d768", "forward", 8191, 50257, 768),
        # a training step of the GPT-2 124M model: the whole table gets a gradient
        _embedding("embedding-training-d768", "training", 32768, 50257, 768),
        # a small vocabulary, every row hit by many tokens, on the d = 512 model
        _embedding("embedding-training-d512", "training", 4099, 1024, 512, scale=22.627417),
        # every weight of the 9-layer d = 512 model as a tensor of its own
        _clip("clip-d512", 9, 512, 1024, 1024),
        # the largest: four layers and both vocabulary matrices at d = 2048
        _clip("clip-d2048", 4, 2048, 8192, 50257),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "rms_norm", "embedding", "clip"])
    while True:
        if kind == "linear":
            case = _linear(None, rng.choice(["forward", "training"]), _log_int(rng, 1, 8192),
                           8 * _log_int(rng, 8, 1376), 8 * _log_int(rng, 8, 1376),
                           bias=rng.random() < 0.4,
                           activation=rng.choice(["none", "none", "relu2", "gelu"]),
                           residual=rng.random() < 0.4)
            if work(case)["flops"] <= 8e11:
                break
        elif kind == "rms_norm":
            direction = rng.choice(["forward", "8-bit", "training"])
            case = _rms_norm(None, direction, _log_int(rng, 1, 32768), 8 * _log_int(rng, 8, 1024),
                             dtype=rng.choice(["bf16", "bf16", "fp32"]),
                             residual=rng.random() < 0.7, weight=rng.random() < 0.8,
                             group=rng.choice([0, 128]) if direction == "8-bit" else 0)
            if work(case)["bytes"] <= 450e6:
                break
        elif kind == "embedding":
            case = _embedding(None, rng.choice(["forward", "training"]), _log_int(rng, 1, 32768),
                              _log_int(rng, 128, 65536), 8 * _log_int(rng, 8, 512),
                              scale=rng.choice([1.0, 1.0, 16.0]),
                              table=rng.choice(["fp32", "fp32", "bf16"]))
            if work(case)["bytes"] <= 300e6:
                break
        else:
            width = 8 * _log_int(rng, 8, 256)
            case = _clip(None, rng.randint(1, 9), width, width * rng.choice([1, 2, 4]),
                         _log_int(rng, 128, 50257), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                         out=rng.choice(["bf16", "fp32"]))
            if work(case)["bytes"] <= 1.6e9:
                break
    del case["name"]
    return case


def _clip_shapes(case):
    """Query and key/value, projection, MLP matrices and norm weights of each layer, then the
    token embedding and the output head."""
    w, h = case["width"], case["hidden"]
    layer = [(w, w), (w, w), (h, w), (w, h), (w,)]
    return layer * case["layers"] + [(case["rows"], w), (case["rows"], w)]


# ---------------------------------------------------------------- inputs
_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    st = {"case": dict(case)}
    if case["op"] == "linear":
        t, k, n = case["tokens"], case["in"], case["out"]
        st["x"], st["w"] = randn(t, k), randn(n, k, std=k ** -0.5)
        st["bias"] = randn(n, std=0.1) if case["bias"] else None
        st["residual"] = randn(t, n) if case["residual"] else None
        st["dy"] = randn(t, n, std=1e-2) if case["direction"] == "training" else None
        return st
    if case["op"] == "rms_norm":
        t, d, dt = case["tokens"], case["dim"], _DTYPES[case["dtype"]]
        st["x"] = randn(t, d, dtype=dt)
        st["residual"] = randn(t, d, std=3.0, dtype=dt) if case["residual"] else None
        st["w"] = 1.0 + 0.2 * randn(d, dtype=torch.float32) if case["weight"] else None
        if case["direction"] == "training":
            st["dy"] = randn(t, d, std=1e-2, dtype=dt)
            st["dres"] = randn(t, d, std=1e-2, dtype=dt) if case["residual"] else None
        return st
    if case["op"] == "embedding":
        t, v, d = case["tokens"], case["rows"], case["dim"]
        st["table"] = randn(v, d, std=0.02, dtype=_DTYPES[case["table"]])
        # token frequencies fall off as one over the rank, as in text; ranks are shuffled ids
        cdf = (1.0 / torch.arange(2, v + 2, dtype=torch.float64)).cumsum(0)
        u = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
        rank = torch.searchsorted(cdf.cuda(), u).clamp_max(v - 1)
        st["ids"] = torch.randperm(v, generator=gen, device="cuda")[rank]
        st["dy"] = randn(t, d, std=1e-2) if case["direction"] == "training" else None
        return st
    dt, out = _DTYPES[case["dtype"]], _DTYPES[case["out"]]
    st["grads"] = [randn(*s, std=1e-3, dtype=dt) for s in _clip_shapes(case)]
    st["outs"] = [torch.empty_like(g, dtype=out) for g in st["grads"]]
    if own:
        # the pointers and sizes of the gradients are laid out once, as for the optimizer
        import newton_schulz_step_gb300 as muon
        st["clip"] = muon.ClipGradNorm(st["grads"], max_norm=1.0, outs=st["outs"], eps=EPS)
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](state, case)
    return _PLAIN[case["op"]](state, case)


def _own_linear(st, case):
    import newton_schulz_step_gb300 as muon
    act = None if case["activation"] == "none" else case["activation"]
    kw = dict(bias=st["bias"], activation=act, residual=st["residual"])
    if case["direction"] == "forward":
        return muon.linear(st["x"], st["w"], **kw)
    y, z = muon.linear(st["x"], st["w"], save_preact=True, **kw) if act else (
        muon.linear(st["x"], st["w"], **kw), None)
    dx, dw, db = muon.linear_backward(st["dy"], st["x"], st["w"], bias=case["bias"],
                                      activation=act, preact=z)
    return (y, dx, dw, db) if case["bias"] else (y, dx, dw)


def _own_rms_norm(st, case):
    import newton_schulz_step_gb300 as muon
    kw = dict(residual=st["residual"], eps=EPS)
    if case["direction"] == "8-bit":
        q, scale, h = muon.rms_norm_fp8(st["x"], st["w"], group=case["group"], **kw)
        # the scales are powers of two: the values are exact in bf16
        y = q.to(torch.bfloat16)
        columns = q.shape[1] if case["group"] == 0 else case["group"]
        scale = scale.to(torch.bfloat16)
        if q.shape[1] % columns == 0:
            y = (y.unflatten(1, (-1, columns)) * scale[:, :, None]).flatten(1)
        else:
            y = y * scale.repeat_interleave(columns, 1)[:, :q.shape[1]]
        return (y, h) if case["residual"] else y
    y, h = muon.rms_norm(st["x"], st["w"], **kw)
    if case["direction"] == "forward":
        return (y, h) if case["residual"] else y
    dx, dw = muon.rms_norm_backward(st["dy"], h, st["w"], dresidual=st["dres"], eps=EPS)
    out = (y, h, dx) if case["residual"] else (y, dx)
    return out + (dw,) if case["weight"] else out


def _own_embedding(st, case):
    import newton_schulz_step_gb300 as muon
    y = muon.embedding(st["ids"], st["table"], scale=case["scale"])
    if case["direction"] == "forward":
        return y
    return y, muon.embedding_backward(st["dy"], st["ids"], case["rows"], scale=case["scale"])


def _own_clip(st, case):
    return (st["clip"](), *st["outs"])


_OWN = {"linear": _own_linear, "rms_norm": _own_rms_norm, "embedding": _own_embedding,
        "clip": _own_clip}

GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, kind):
    if kind == "relu2":
        return z.clamp_min(0.0).square()
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))
    return z


def _act_grad(z, kind):
    if kind == "relu2":
        return 2.0 * z.clamp_min(0.0)
    t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_A * (1.0 + 3.0 * GELU_B * z * z)


def _plain_linear(st, case):
    x, w = st["x"].float(), st["w"].float()
    z = x @ w.T
    if case["bias"]:
        z = z + st["bias"].float()
    y = _act(z, case["activation"])
    if case["residual"]:
        y = y + st["residual"].float()
    y = y.to(torch.bfloat16)
    if case["direction"] == "forward":
        return y
    dz = st["dy"].float()
    if case["activation"] != "none":
        dz = dz * _act_grad(z, case["activation"])
    dx, dw = (dz @ w).to(torch.bfloat16), (dz.T @ x).to(torch.bfloat16)
    return (y, dx, dw, dz.sum(0).to(torch.bfloat16)) if case["bias"] else (y, dx, dw)


def _plain_rms_norm(st, case):
    dt = st["x"].dtype
    h = st["x"].float()
    if case["residual"]:
        h = h + st["residual"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    if case["weight"]:
        y = y * st["w"]
    if case["direction"] == "8-bit":
        t, d = y.shape
        columns = d if case["group"] == 0 else case["group"]
        groups = torch.nn.functional.pad(y, (0, -d % columns)).unflatten(1, (-1, columns))
        amax = groups.abs().amax(2, keepdim=True)
        # the least power of two that brings the group's largest magnitude to 448 or less
        m, e = torch.frexp(amax / E4M3_MAX)
        e = torch.where(m == 0.5, e - 1, e).clamp(-126, 127)
        scale = torch.where(amax == 0, torch.ones_like(amax), torch.ldexp(torch.ones_like(m), e))
        q = (groups / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        y = (q.float() * scale).flatten(1)[:, :d].to(torch.bfloat16)
    else:
        y = y.to(dt)
    h16 = h.to(dt)
    if case["direction"] != "training":
        return (y, h16) if case["residual"] else y
    # the gradients go by the sum as it was stored
    hs, g = h16.float(), st["dy"].float()
    r = torch.rsqrt(hs.square().mean(1, keepdim=True) + EPS)
    n = hs * r
    gw = g * st["w"] if case["weight"] else g
    dx = r * (gw - n * (gw * n).mean(1, keepdim=True))
    if case["residual"]:
        dx = dx + st["dres"].float()
    out = (y, h16, dx.to(dt)) if case["residual"] else (y, dx.to(dt))
    return out + ((g * n).sum(0),) if case["weight"] else out


def _plain_embedding(st, case):
    y = (st["table"][st["ids"]].float() * case["scale"]).to(torch.bfloat16)
    if case["direction"] == "forward":
        return y
    dw = torch.zeros(case["rows"], case["dim"], device=y.device)
    dw.index_add_(0, st["ids"], st["dy"].float())
    return y, dw * case["scale"]


def _plain_clip(st, case):
    total = sum(g.float().square().sum() for g in st["grads"]).sqrt()
    c = torch.clamp(1.0 / (total + EPS), max=1.0)
    for g, o in zip(st["grads"], st["outs"]):
        o.copy_(g.float() * c)
    return (total, *st["outs"])


_PLAIN = {"linear": _plain_linear, "rms_norm": _plain_rms_norm, "embedding": _plain_embedding,
          "clip": _plain_clip}


# ---------------------------------------------------------------- work
def work(case):
    training = case.get("direction") == "training"
    if case["op"] == "linear":
        t, k, n = case["tokens"], case["in"], case["out"]
        nbytes = 2 * (t * k + n * k + t * n)
        nbytes += 2 * (n if case["bias"] else 0) + 2 * (t * n if case["residual"] else 0)
        if training:                    # dy in; dx, dw, db out
            nbytes += 2 * (t * n + t * k + n * k) + 2 * (n if case["bias"] else 0)
        return {"bytes": nbytes, "flops": 2 * t * k * n * (3 if training else 1)}
    if case["op"] == "rms_norm":
        t, d = case["tokens"], case["dim"]
        size = 4 if case["dtype"] == "fp32" else 2
        passes = 4 if case["residual"] else 2       # x, residual in; y, sum out
        nbytes = t * d * size * passes
        if case["direction"] == "8-bit":            # y in 8 bits
            nbytes += t * d * (1 - size) + 4 * t * (-(-d // 128) if case["group"] else 1)
        if training:                                # dy, dresidual in; dx out
            nbytes += t * d * size * (3 if case["residual"] else 2)
        nbytes += d * 4 * (2 if training else 1) if case["weight"] else 0
        return {"bytes": nbytes, "flops": t * d * (14 if training else 6)}
    if case["op"] == "embedding":
        t, d, v = case["tokens"], case["dim"], case["rows"]
        size = 4 if case["table"] == "fp32" else 2
        nbytes = min(t, v) * d * size + t * 8 + t * d * 2
        if training:                                # dy in, the whole table's gradient out
            nbytes += t * d * 2 + v * d * 4
        return {"bytes": nbytes, "flops": t * d * (3 if training else 1)}
    n = sum(math.prod(s) for s in _clip_shapes(case))
    sizes = {"bf16": 2, "fp32": 4}
    return {"bytes": n * (sizes[case["dtype"]] + sizes[case["out"]]), "flops": 3 * n}


# ---------------------------------------------------------------- 64-bit results
def exact(case, seed):
    # (products in 64 bits run at about 1e12 operations a second)
    if case["op"] == "linear" and work(case)["flops"] > 8e12:
        return None
    return _EXACT[case["op"]](prepare(case, seed), case)


def _exact_linear(st, case):
    x, w = st["x"].double(), st["w"].double()
    z = torch.einsum("tk,nk->tn", x, w)
    if st["bias"] is not None:
        z += st["bias"].double()
    kind = case["activation"]
    if kind == "relu2":
        y, slope = torch.where(z > 0, z * z, 0.0), torch.where(z > 0, 2 * z, 0.0)
    elif kind == "gelu":
        # z / (1 + exp(-2 u)) is the tanh form
        u = GELU_A * (z + GELU_B * z ** 3)
        s = torch.sigmoid(2 * u)
        y, slope = z * s, s + 2 * z * s * (1 - s) * GELU_A * (1 + 3 * GELU_B * z ** 2)
    else:
        y, slope = z.clone(), torch.ones_like(z)
    if st["residual"] is not None:
        y += st["residual"].double()
    if case["direction"] == "forward":
        return y
    dz = st["dy"].double() * slope
    out = (y, torch.einsum("tn,nk->tk", dz, w), torch.einsum("tn,tk->nk", dz, x))
    return out + (torch.einsum("tn->n", dz),) if case["bias"] else out


def _exact_rms_norm(st, case):
    t, d = case["tokens"], case["dim"]
    h = st["x"].double()
    if st["residual"] is not None:
        h = h + st["residual"].double()
    w = torch.ones(d, dtype=torch.float64, device="cuda") if st["w"] is None else st["w"].double()
    r = (h.pow(2).sum(1, keepdim=True) / d + EPS).pow(-0.5)
    y = h * r * w
    if case["direction"] == "8-bit":
        step = d if case["group"] == 0 else case["group"]
        for c in range(0, d, step):
            block = y[:, c:c + step]
            top = block.abs().amax(1, keepdim=True)
            s = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, 448.0) / 448.0)))
            block.copy_(_round_e4m3(block / s) * s)
    if case["direction"] != "training":
        return (y, h) if case["residual"] else y
    g = st["dy"].double()
    dx = r * g * w - r.pow(3) * h * (g * w * h).sum(1, keepdim=True) / d
    if st["dres"] is not None:
        dx = dx + st["dres"].double()
    dw = (g * h * r).sum(0) if case["dtype"] == "fp32" or not case["residual"] else None
    if dw is None:
        # the gradients go by the sum as it was stored, in bf16
        hs = (st["x"].double() + st["residual"].double()).float().to(torch.bfloat16).double()
        rs = (hs.pow(2).sum(1, keepdim=True) / d + EPS).pow(-0.5)
        dw = (g * hs * rs).sum(0)
    out = (y, h, dx) if case["residual"] else (y, dx)
    return out + (dw,) if case["weight"] else out


def _round_e4m3(v):
    """Nearest multiple of the spacing at v: 2^(e - 3), e >= -6 the exponent; ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6)))
    spacing = torch.exp2(e - 3)
    return torch.round(v / spacing) * spacing


def _exact_embedding(st, case):
    y = st["table"].double()[st["ids"]] * case["scale"]
    if case["direction"] == "forward":
        return y
    order = torch.argsort(st["ids"])
    dw = torch.zeros(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
    dw.index_put_((st["ids"][order],), st["dy"].double()[order] * case["scale"], accumulate=True)
    return y, dw


def _exact_clip(st, case):
    total = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in st["grads"]))
    c = min(1.0, 1.0 / (total + EPS))
    return (torch.tensor(total, dtype=torch.float64), *(g.double() * c for g in st["grads"]))


_EXACT = {"linear": _exact_linear, "rms_norm": _exact_rms_norm, "embedding": _exact_embedding,
          "clip": _exact_clip}
