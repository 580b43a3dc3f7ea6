"""Cases of the operators around the QLoRA linear: the RMS norm with the
residual addition (bf16 with its backward, and with 8-bit output), the linear
in 8-bit integers that serves a merged weight, and the global gradient norm
with clipping in front of the 8-bit AdamW step.

`run` computes a case in elementary torch operations, or, where `own` is true,
through the package's calls; `exact` is the definition in 64 bits."""

import math

import torch

own = False

EPS = 1e-5
HP = dict(lr=2e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
STEP = 10                   # optimizer steps done, this one included
MAX_NORM = 0.3
# (d_out, d_in) of the linears of a 7B-shaped decoder block: q, k, v, o, gate, up, down
BLOCK = ((4096, 4096),) * 4 + ((11008, 4096),) * 2 + ((4096, 11008),)


def listed():
    return [
        # one token of a generation: the norm in front of q/k/v, latency only
        {"name": "norm_int8_1_token", "op": "norm_int8", "m": 1, "d": 4096, "res": True},
        # a prompt of 4 x 2048 tokens through the same norm
        {"name": "norm_int8_8192", "op": "norm_int8", "m": 8192, "d": 4096, "res": True},
        # the first norm of a model has no residual; ragged batch, the MLP's width
        {"name": "norm_int8_333_wide", "op": "norm_int8", "m": 333, "d": 11008, "res": False},
        # one training step of the layer norm of the training shape, weight trained
        {"name": "norm_train_2048", "op": "norm_train", "m": 2048, "d": 4096, "res": True, "dw": True},
        # a short ragged batch of a small model, weight frozen (QLoRA trains the adapters only)
        {"name": "norm_train_77_small", "op": "norm_train", "m": 77, "d": 1032, "res": True, "dw": False},
        # single-token generation, up projection: the weight is read once
        {"name": "linear_1_token_up", "op": "linear", "m": 1, "n": 11008, "k": 4096, "bf16_in": False},
        # sixteen sequences generating, down projection behind the activation (no norm: x arrives in bf16)
        {"name": "linear_16_tokens_down", "op": "linear", "m": 16, "n": 4096, "k": 11008, "bf16_in": True},
        # a ragged mid-size batch of generating sequences
        {"name": "linear_100_tokens", "op": "linear", "m": 100, "n": 4096, "k": 4096, "bf16_in": False},
        # a prompt of the training shape, and the largest projection at 4 x 2048 tokens
        {"name": "linear_2048_tokens", "op": "linear", "m": 2048, "n": 4096, "k": 4096, "bf16_in": True},
        {"name": "linear_8192_tokens_up", "op": "linear", "m": 8192, "n": 11008, "k": 4096, "bf16_in": False},
        # the optimizer step of one layer's adapters, and of a whole 7B model's (32 layers, rank 16)
        {"name": "clip_step_1_layer", "op": "clip_step", "layers": 1, "r": 16},
        {"name": "clip_step_32_layers", "op": "clip_step", "layers": 32, "r": 16},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_int8", "norm_train", "linear", "linear", "clip_step", "clip"))
    if op == "norm_int8":
        return {"op": op, "m": _log(rng, 1, 8192), "d": 16 * _log(rng, 8, 688), "res": rng.random() < 0.7}
    if op == "norm_train":
        return {"op": op, "m": _log(rng, 1, 8192), "d": 8 * _log(rng, 8, 1376), "res": rng.random() < 0.7,
                "dw": rng.random() < 0.5}
    if op == "linear":
        n, k = 8 * _log(rng, 8, 1376), 16 * _log(rng, 4, 688)
        return {"op": op, "m": min(_log(rng, 1, 8192), 8192 * 11008 * 4096 // (n * k)), "n": n, "k": k,
                "bf16_in": rng.random() < 0.5}
    if op == "clip_step":
        return {"op": op, "layers": _log(rng, 1, 32), "r": 8 * rng.randint(1, 2)}
    return {"op": op, "tensors": rng.randint(1, 60), "longest": _log(rng, 100, 1000000), "half": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _hidden(g, m, d):
    """Activations with a few channels far larger than the others."""
    big = 1 + 19 * (torch.rand(d, generator=g, device="cuda") < 0.005).float()
    return (_normal(g, m, d) * big).to(torch.bfloat16)


def _block_scales(g, n):
    """Magnitudes by blocks of 256 values, log-uniform in [1e-6, 1e-1]."""
    e = torch.rand((n + 255) // 256, generator=g, device="cuda") * 5 - 6
    return (10.0 ** e).repeat_interleave(256)[:n]


def _to_int8(x):
    """bf16 rows -> int8 codes and fp32 scales, one per row."""
    v = x.float()
    amax = v.abs().amax(1, keepdim=True)
    codes = torch.where(amax > 0, torch.round(v * 127 / amax), torch.zeros_like(v)).to(torch.int8)
    return codes, amax.squeeze(1) / 127


def _to_e4m3(x):
    """fp32 [n] -> E4M3 codes [n] and fp32 scales, one per block of 256."""
    n = x.numel()
    pad = torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)
    amax = pad.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, pad * (torch.full_like(amax, 448.0) / amax), torch.zeros_like(pad))
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:n]
    return codes.clone(), (amax / torch.full_like(amax, 448.0)).view(-1)


def _from_e4m3(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(256)[:codes.numel()]


def _sizes(case):
    return [v for _ in range(case["layers"]) for n, k in BLOCK for v in (case["r"] * k, n * case["r"])]


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm_int8", "norm_train"):
        m, d = case["m"], case["d"]
        s["x"] = _hidden(g, m, d)
        s["res"] = _hidden(g, m, d) if case["res"] else None
        s["w"] = (1 + 0.1 * _normal(g, d)).to(torch.bfloat16)
        if op == "norm_train":
            s["dy"] = (0.01 * _normal(g, m, d)).to(torch.bfloat16)
            s["dh"] = (0.01 * _normal(g, m, d)).to(torch.bfloat16) if case["res"] else None
    elif op == "linear":
        s["codes"], s["scale"] = _to_int8((0.02 * _normal(g, case["n"], case["k"])).to(torch.bfloat16))
        x = _hidden(g, case["m"], case["k"])
        if case["bf16_in"]:
            s["x"] = x
        else:
            s["xq"], s["xs"] = _to_int8(x)
    elif op == "clip_step":
        sizes = _sizes(case)
        n = sum(sizes)
        scales = _block_scales(g, n)
        s["grad"] = _normal(g, n) * scales
        s["grads"] = list(torch.split(s["grad"], sizes))      # dA and dB of every linear, in one array
        s["p"] = 0.02 * _normal(g, n)
        s["pb"] = s["p"].to(torch.bfloat16)
        s["mc"], s["ms"] = _to_e4m3(0.3 * _normal(g, n) * scales)
        s["vc"], s["vs"] = _to_e4m3((_normal(g, n) * scales).square() * 0.01)
    else:
        sizes = [_one_size(case, i) for i in range(case["tensors"])]
        s["grads"] = [(_normal(g, n) * 10.0 ** (-1 - i % 4)).to(torch.bfloat16 if case["half"] and i % 2 else torch.float32)
                      for i, n in enumerate(sizes)]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
    return s


def _one_size(case, i):
    """Sizes of a ragged list: from the longest down to single values."""
    return max(1, int(case["longest"] * (0.37 ** (i % 7))) - (i * i) % 5)


# ---------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import bit_nf4_quantized_28_b200 as qn
    from bit_nf4_quantized_28_b200 import grads, int8, norm
    case = s["case"]
    op = case["op"]
    if op == "norm_int8":
        codes, scale, h = norm.forward_int8(s["x"], s["w"], residual=s["res"], eps=EPS)
        values = torch.empty_like(h)
        return {"h": h, "values": torch.mul(codes, scale[:, None], out=values), "scale": scale}
    if op == "norm_train":
        y, h, rstd = norm.forward(s["x"], s["w"], residual=s["res"], eps=EPS)
        dx, dw = norm.backward(s["dy"], h, s["w"], rstd, dh=s["dh"], need_dw=case["dw"])
        return {"y": y, "h": h, "dx": dx, "dw": dw}
    if op == "linear":
        w = int8.Weight(case["n"], case["k"], s["codes"], s["scale"])
        xq, xs = int8.quantize(s["x"]) if case["bf16_in"] else (s["xq"], s["xs"])
        return int8.linear(xq, xs, w)
    if "list" not in s:                    # the program's handle on its gradients, made once
        s["list"] = grads.TensorList(s["grads"])
        s["out_list"] = grads.TensorList(s["out"]) if op == "clip" else None
        s["ws"] = grads.make_workspace(s["list"])
    total, coef = grads.norm(s["list"], MAX_NORM, workspace=s["ws"])
    if op == "clip":
        grads.clip(s["list"], coef, out=s["out_list"])
        return {"norm": total, "clipped": s["out"]}
    st = qn.AdamW8State(s["mc"], s["ms"], s["vc"], s["vs"])
    qn.adamw8_step(s["p"], s["grad"], st, STEP, param_bf16=s["pb"], grad_scale=coef, **HP)
    return _step_outputs(s, total)


def _step_outputs(s, total):
    """The updated parameters and states: the moments as E4M3 values in units of their blocks' scales."""
    return {"norm": total, "p": s["p"], "pb": s["pb"], "m": s["mc"].view(torch.float8_e4m3fn), "m_scale": s["ms"],
            "v": s["vc"].view(torch.float8_e4m3fn), "v_scale": s["vs"]}


def _run_plain(s):
    return {"norm_int8": _plain_norm_int8, "norm_train": _plain_norm_train, "linear": _plain_linear,
            "clip_step": _plain_clip_step, "clip": _plain_clip}[s["case"]["op"]](s)


def _stream(s):
    """The residual stream h as it is stored, and its values in fp32."""
    h = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(torch.bfloat16)
    return h, h.float()


def _plain_norm_int8(s):
    h, v = _stream(s)
    rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    t = v * s["w"].float()
    amax = t.abs().amax(1, keepdim=True)
    q = torch.where(amax > 0, torch.round(t * 127 / amax), torch.zeros_like(t))
    scale = amax * rstd / 127
    return {"h": h, "values": (q * scale).to(torch.bfloat16), "scale": scale.squeeze(1)}


def _plain_norm_train(s):
    h, v = _stream(s)
    w = s["w"].float()
    rstd = torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)
    y = (v * rstd * w).to(torch.bfloat16)
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - v * rstd.square() * (g * v).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dw = (dy * v * rstd).sum(0) if s["case"]["dw"] else None
    return {"y": y, "h": h, "dx": dx.to(torch.bfloat16), "dw": dw}


def _plain_linear(s):
    if s["case"]["bf16_in"]:
        xq, xs = _to_int8(s["x"])
    else:
        xq, xs = s["xq"], s["xs"]
    acc = xq.float() @ s["codes"].float().T
    return (acc * xs[:, None] * s["scale"][None, :]).to(torch.bfloat16)


def _norm_and_coef(ts):
    """The norm of all tensors together (a long sum: in 64 bits), in fp32, and the clipping coefficient."""
    total = torch.stack([t.double().square().sum() for t in ts]).sum().sqrt().float()
    return total, torch.clamp(MAX_NORM / (total + 1e-6), max=1.0)


def _plain_clip(s):
    total, coef = _norm_and_coef(s["grads"])
    return {"norm": total, "clipped": [(t.float() * coef).to(t.dtype) for t in s["grads"]]}


def _plain_clip_step(s):
    total, coef = _norm_and_coef(s["grads"])
    b1, b2 = HP["beta1"], HP["beta2"]
    g = s["grad"] * coef
    m = _from_e4m3(s["mc"], s["ms"]) * b1 + g * (1 - b1)
    v = _from_e4m3(s["vc"], s["vs"]) * b2 + g * g * (1 - b2)
    den = v.sqrt() * (1 / math.sqrt(1 - b2 ** STEP)) + HP["eps"]
    p = s["p"] * (1 - HP["lr"] * HP["weight_decay"]) - (m / den) * (HP["lr"] / (1 - b1 ** STEP))
    s["p"].copy_(p)
    s["pb"].copy_(p)
    (mc, ms), (vc, vs) = _to_e4m3(m), _to_e4m3(v)
    s["mc"].copy_(mc)
    s["ms"].copy_(ms)
    s["vc"].copy_(vc)
    s["vs"].copy_(vs)
    return _step_outputs(s, total)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm_int8", "norm_train"):
        m, d = case["m"], case["d"]
        res = 2 if case["res"] else 1
        if op == "norm_int8":             # x (and the residual) in, codes and scales (and the new stream) out
            per = 2 * res + 1 + (2 if case["res"] else 0)     # (the values returned beside are not the operator's)
            return {"bytes": m * d * per + 2 * d + 4 * m, "flops": 6 * m * d}
        per = 2 * res + 2 * res + 2 + 2 + (2 if case["res"] else 0)    # x, res, dy, dh in; y, dx, h out
        return {"bytes": m * d * per + 2 * d + (4 * d if case["dw"] else 0), "flops": 16 * m * d}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        x = 2 * m * k if case["bf16_in"] else m * k + 4 * m
        return {"bytes": x + n * k + 4 * n + 2 * m * n, "flops": 2 * m * n * k}
    if op == "clip_step":                  # gradient, parameters and their copy, codes and scales of both moments
        n = sum(_sizes(case))
        return {"bytes": n * (4 + 8 + 2 + 4) + 4 * 4 * ((n + 255) // 256), "flops": 20 * n}
    sizes = [(_one_size(case, i), 2 if case["half"] and i % 2 else 4) for i in range(case["tensors"])]
    return {"bytes": sum(2 * n * b for n, b in sizes), "flops": 3 * sum(n for n, _ in sizes)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(s)
    if op in ("norm_int8", "norm_train"):
        return _exact_norm(s)
    return _exact_clip(s)


def _exact_linear(s):
    if s["case"]["bf16_in"]:
        x = s["x"].to(torch.float64)
        xs = torch.linalg.vector_norm(x, ord=math.inf, dim=1) / 127
        xq = torch.where(xs[:, None] > 0, (x / xs[:, None]).round(), 0.0)
    else:
        xq, xs = s["xq"].to(torch.float64), s["xs"].to(torch.float64)
    left, right = xq * xs.unsqueeze(1), s["codes"].to(torch.float64) * s["scale"].to(torch.float64).unsqueeze(1)
    return torch.einsum("mk,nk->mn", left, right)


def _exact_norm(s):
    case = s["case"]
    h = s["x"].to(torch.float64)
    if case["res"]:
        h = (h + s["res"].to(torch.float64)).to(torch.bfloat16).to(torch.float64)
    w = s["w"].to(torch.float64)
    r = (torch.einsum("md,md->m", h, h) / case["d"] + EPS).pow(-0.5)
    y = torch.einsum("md,m,d->md", h, r, w)
    if case["op"] == "norm_int8":
        unit = y.abs().max(dim=1).values / 127
        # codes from the stream and the weight: the same for every r
        top = (h * w).abs().max(dim=1).values
        return {"h": h, "values": torch.round(127 * (h * w) / top[:, None]) * unit[:, None], "scale": unit}
    dy = s["dy"].to(torch.float64)
    n = h * r[:, None]                                            # the normalised rows
    g = dy * w
    dx = (g - n * torch.einsum("md,md->m", g, n)[:, None] / case["d"]) * r[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].to(torch.float64)
    return {"y": y, "h": h, "dx": dx, "dw": torch.einsum("md,md->d", dy, n) if case["dw"] else None}


def _round_e4m3(x, n):
    """x [n] in units of its blocks' absmax / 448, rounded to the grid of 3-bit mantissas (exponents from -6 up), and those units."""
    pad = torch.cat([x, x.new_zeros(-n % 256)]).view(-1, 256)
    unit = pad.abs().max(dim=1, keepdim=True).values / 448
    t = torch.where(unit > 0, pad / unit, 0.0)
    grid = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(t / grid) * grid).view(-1)[:n], unit.view(-1)


def _exact_clip(s):
    wide = [t.to(torch.float64) for t in s["grads"]]
    total = torch.cat(wide).norm()
    coef = min(1.0, MAX_NORM / (float(total) + 1e-6))
    if s["case"]["op"] == "clip":
        return {"norm": total, "clipped": [t * coef for t in wide]}
    n = s["p"].numel()
    g = torch.cat(wide) * coef
    b1, b2 = HP["beta1"], HP["beta2"]
    ms, vs = (torch.repeat_interleave(s[k].to(torch.float64), 256)[:n] for k in ("ms", "vs"))
    m = b1 * s["mc"].view(torch.float8_e4m3fn).to(torch.float64) * ms + (1 - b1) * g
    v = b2 * s["vc"].view(torch.float8_e4m3fn).to(torch.float64) * vs + (1 - b2) * g ** 2
    up = (m / (1 - b1 ** STEP)) / (torch.sqrt(v / (1 - b2 ** STEP)) + HP["eps"])
    p = s["p"].to(torch.float64)
    p = p - HP["lr"] * HP["weight_decay"] * p - HP["lr"] * up
    (m, ms), (v, vs) = _round_e4m3(m, n), _round_e4m3(v, n)
    return {"norm": total, "p": p, "pb": p, "m": m, "m_scale": ms, "v": v, "v_scale": vs}
