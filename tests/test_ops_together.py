"""The operators around the QLoRA linear used together, as a training step and
as the served model run them."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_28_b200 as qn
from bit_nf4_quantized_28_b200 import grads, int8, norm
from bit_nf4_quantized_28_b200 import workloads as wl

pytestmark = pytest.mark.gpu

D, M, R, ALPHA, EPS = 256, 48, 8, 16.0, 1e-5


def _layer(seed):
    t = wl.make_linear(seed, D, D, M, R, ALPHA)
    return t, qn.quantize(t.W.cuda()), t.A.cuda(), t.B.cuda()


def test_training_step():
    """norm -> linear, twice along a residual stream; backward; clipping; the
    8-bit optimizer.  The gradients are compared with autograd in fp64 on the
    dequantized weight: every stored tensor on the way is bf16, so the rule of
    the layer's own tests holds (mean relative error 5e-3, here over a chain
    of six roundings: 2e-2)."""
    g = torch.Generator().manual_seed(0)
    x0 = wl.normal_bf16(g, (M, D), 1.0).cuda()
    layers = [_layer(s) for s in (1, 2)]
    ws = [(1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in layers]
    dout = wl.normal_bf16(g, (M, D), 1.0).cuda()

    # forward: h1 = x0, o1 = lin1(norm(h1)); h2 = h1 + o1, o2 = lin2(norm(h2)); out = h2 + o2
    saved, h, o = [], x0, None
    for (t, w, A, B), nw in zip(layers, ws):
        y, h, rstd = norm.forward(h, nw, eps=EPS) if o is None else norm.forward(o, nw, residual=h, eps=EPS)
        o, u = qn.linear_fwd(y, w, A, B, ALPHA)
        saved.append((y, h, rstd, u))
    # backward of sum(dout * out): the stream's gradient runs through every norm
    dh, d_lin = dout, dout
    got = []
    for (t, w, A, B), nw, (y, h, rstd, u) in reversed(list(zip(layers, ws, saved))):
        dy, dA, dB = qn.linear_bwd(d_lin, y, w, A, B, ALPHA, u)
        dh, dw = norm.backward(dy, h, nw, rstd, dh=dh, need_dw=True)
        d_lin = dh
        got = [dA, dB, dw] + got
    got.append(dh)

    f64 = lambda v: v.double().detach().requires_grad_(True)
    xr = f64(x0)
    params, h, o = [], xr, None
    for (t, w, A, B), nw in zip(layers, ws):
        Ar, Br, nr, W = f64(A), f64(B), f64(nw), qn.dequantize(w).double()
        h = h if o is None else h + o
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * nr
        o = y @ W.T + ALPHA / R * (y @ Ar.T) @ Br.T
        params += [Ar, Br, nr]
    ((h + o) * dout.double()).sum().backward()
    for v, p in zip(got, params + [xr]):
        ref = p.grad
        assert float((v.double() - ref).abs().sum() / ref.abs().sum()) < 2e-2

    # clipping and the step over all adapters in one array
    flat = torch.cat([v.reshape(-1) for v in got[0:2] + got[3:5]])
    total, coef = grads.norm([got[0], got[1], got[3], got[4]], max_norm=0.3)
    assert float(coef) < 1
    p = torch.cat([v.float().reshape(-1) for _, _, A, B in layers for v in (A, B)])
    before = p.clone()
    st = qn.AdamW8State.zeros(p.numel())
    qn.adamw8_step(p, flat, st, 1, lr=1e-3, grad_scale=coef)
    ref = torch.nn.Parameter(before.clone())
    ref.grad = flat.clone()
    torch.nn.utils.clip_grad_norm_([ref], 0.3)
    torch.optim.AdamW([ref], lr=1e-3, weight_decay=0.0).step()
    # two fp32 evaluations of the same step: 24 u of an update of at most lr, 2 ulp of p
    # (and the coefficients 4 u apart, to which the first step's update m / sqrt(v) is blind but for eps)
    tol = 2.0 ** -24 * (40 * 1e-3 + 4 * before.abs())
    assert bool(((p - ref.detach()).abs() <= tol).all())
    assert qn.device_error() == 0


def test_served_layer():
    """Merge to 8 bits, then norm -> linear in 8 bits for one token and for
    many, against fp64 on the merged bf16 weight.  Bound: a quantized row or
    channel is off by at most half a step, scale / 2, per element, so
    |y - ref| <= sum_k (|x| sw / 2 + |w| sx / 2 + sx sw / 4), and a bf16
    rounding (2^-8); 2^-12 of the sum of magnitudes covers fp32."""
    t, w, A, B = _layer(5)
    merged = qn.merge(w, A, B, ALPHA)
    w8 = int8.merge(w, A, B, ALPHA)
    direct = int8.quantize_weight(merged)
    assert torch.equal(w8.codes, direct.codes) and torch.equal(w8.scale, direct.scale)
    g = torch.Generator().manual_seed(6)
    nw = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    for m in (1, 5, 40, 300):
        x, res = (wl.normal_bf16(g, (m, D), 1.0).cuda() for _ in range(2))
        codes, scale, h = norm.forward_int8(x, nw, residual=res, eps=EPS)
        y = int8.linear(codes, scale, w8)
        hd = (x + res).double()
        assert torch.equal(hd, h.double())
        xn = hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + EPS) * nw.double()
        W = merged.double()
        ref = xn @ W.T
        sx, sw = scale.double()[:, None], w8.scale.double()[None, :]
        tol = xn.abs().sum(1, keepdim=True) * sw / 2 + sx / 2 * W.abs().sum(1)[None, :] + D * sx * sw / 4
        tol = tol * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8 + 2.0 ** -12 * (xn.abs() @ W.abs().T)
        assert bool(((y.double() - ref).abs() <= tol).all())
    assert qn.device_error() == 0


@pytest.mark.parametrize("m", [1, 7, 30, 300])
def test_kernels_in_a_row_see_one_another(m):
    """The kernels start before their predecessors end and wait for them on
    the device: a chain that rewrites its buffers every turn, without a wait
    on the host, gives what the same chain gives with one after each call."""
    g = torch.Generator().manual_seed(m)
    Ws = [wl.normal_bf16(g, (520, D), 0.05).cuda() for _ in range(4)]
    xs = [wl.normal_bf16(g, (m, D), 1.0).cuda() for _ in range(4)]
    back = wl.normal_bf16(g, (D, 520), 0.05).cuda()
    nw = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    w8, b8 = int8.quantize_weight(Ws[0]), int8.quantize_weight(torch.cat([back, back])[:D].contiguous())
    h = torch.zeros(m, D, dtype=torch.bfloat16, device="cuda")
    codes, scale = torch.empty(m, D, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty(m, 520, dtype=torch.bfloat16, device="cuda")
    yq, ys = torch.empty(m, 528, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    b8 = int8.Weight(D, 528, torch.cat([b8.codes, b8.codes[:, :8]], 1).contiguous(), b8.scale)
    yp = torch.zeros(m, 528, dtype=torch.bfloat16, device="cuda")

    def turn(i, wait):
        done = torch.cuda.synchronize if wait else (lambda: None)
        int8.quantize(Ws[i % 4], codes=w8.codes, scale=w8.scale)
        done()
        norm.forward_int8(xs[i % 4], nw, residual=h, h=h, codes=codes, scale=scale)
        done()
        int8.linear(codes, scale, w8, y=y)
        done()
        yp[:, :520] = y
        int8.quantize(yp, codes=yq, scale=ys)
        done()
        out = int8.linear(yq, ys, b8)
        done()
        total, coef = grads.norm([h, out], 10.0)
        done()
        grads.clip([out], coef)
        done()
        norm.forward(out, nw, residual=h, h=h)
        done()
        return total

    def run(wait):
        h.zero_()
        totals = [turn(i, wait) for i in range(40)]
        return torch.stack(totals), h.clone(), y.clone()

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
    assert bool(torch.isfinite(want[0]).all()) and qn.device_error() == 0
