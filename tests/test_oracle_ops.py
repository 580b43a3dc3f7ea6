"""Pins of the oracle's RMS norm, 8-bit rows, 8-bit linear and gradient norm
(CPU): torch's autograd and finite differences, textbook loops, closed forms."""

import numpy as np
import pytest
import torch

from oracle import grads, int8, norm
from oracle.nf4 import bf16_bits_to_f64, f32_to_bf16_bits


def _bits(rng, *shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def test_norm_forward_by_loops():
    rng = np.random.default_rng(0)
    h, w = _bits(rng, 3, 8), _bits(rng, 8)
    y, rstd = norm.forward(h, w, 1e-5)
    hv, wv = bf16_bits_to_f64(h), bf16_bits_to_f64(w)
    for i in range(3):
        ms = sum(v * v for v in hv[i]) / 8
        assert np.isclose(rstd[i], (ms + float(np.float32(1e-5))) ** -0.5, rtol=1e-14)
        for j in range(8):
            assert np.isclose(y[i, j], hv[i, j] * rstd[i] * wv[j], rtol=1e-14)


def test_stream_is_the_rounded_sum():
    rng = np.random.default_rng(1)
    x, r = _bits(rng, 5, 16), _bits(rng, 5, 16)
    want = (torch.tensor(bf16_bits_to_f64(x)).to(torch.bfloat16) + torch.tensor(bf16_bits_to_f64(r)).to(torch.bfloat16))
    assert np.array_equal(bf16_bits_to_f64(norm.stream(x, r)), want.double().numpy())
    assert np.array_equal(norm.stream(x), x)


@pytest.mark.parametrize("with_dh", [False, True])
def test_norm_backward_matches_autograd_and_differences(with_dh):
    rng = np.random.default_rng(2)
    m, d, eps = 4, 24, 1e-3
    h, w, dy, dh = (rng.standard_normal(s) for s in ((m, d), (d,), (m, d), (m, d)))
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    dx, dw = norm.backward(dy, h, w, rstd, dh if with_dh else None)

    def loss(hv, wv):
        y = hv * torch.rsqrt(hv.square().mean(1, keepdim=True) + eps) * wv
        out = (y * torch.tensor(dy)).sum()
        return out + (hv * torch.tensor(dh)).sum() if with_dh else out

    ht, wt = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    loss(ht, wt).backward()
    assert np.allclose(dx, ht.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-11, atol=1e-12)
    for i, j in ((0, 0), (3, 23), (1, 7)):
        e = np.zeros_like(h)
        e[i, j] = 1e-6
        num = (loss(torch.tensor(h + e), torch.tensor(w)) - loss(torch.tensor(h - e), torch.tensor(w))) / 2e-6
        assert np.isclose(dx[i, j], float(num), rtol=1e-6, atol=1e-7)


def test_codes_ties_extremes_zero_and_bad_rows():
    t = np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5],
                  [0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0, -0.0],
                  [1.0, np.nan, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0],
                  [1.0, np.inf, 2.0, 3.0, 4.0, 5.0, 6.0, 7.0]], np.float32)
    q, amax = norm.codes(t)
    assert q[0].tolist() == [127, -127, 0, 2, 2, 0, -2, 126]      # ties to even
    assert not q[1:].any()
    assert amax[0] == 127.0 and amax[1] == 0.0 and np.isnan(amax[2]) and np.isnan(amax[3])


def test_codes_are_nearest_and_scale_restores():
    rng = np.random.default_rng(3)
    x = _bits(rng, 6, 40, scale=3.0)
    q, s = norm.quantize(x)
    v = bf16_bits_to_f64(x)
    assert np.abs(q).max(axis=1).tolist() == [127] * 6
    # half a step, and the rounding of the quotient to fp32 (127 * 2^-24 of a step)
    assert np.all(np.abs(q * s[:, None] - v) <= s[:, None] * (0.5 + 2.0 ** -16))


def test_int8_norm_stands_for_the_norm():
    rng = np.random.default_rng(4)
    h, w = _bits(rng, 5, 64), f32_to_bf16_bits((1 + 0.1 * rng.standard_normal(64)).astype(np.float32))
    y, _ = norm.forward(h, w, 1e-5)
    q, s = norm.forward_int8(h, w, 1e-5)
    assert np.all(np.abs(q * s[:, None] - y) <= s[:, None] * (0.5 + 2.0 ** -16))
    assert np.allclose(np.abs(y).max(axis=1), 127 * s, rtol=1e-12)


def test_int8_linear_by_loops():
    rng = np.random.default_rng(5)
    x, w = rng.integers(-128, 128, (3, 16), dtype=np.int8), rng.integers(-128, 128, (4, 16), dtype=np.int8)
    xs, ws = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    y = int8.linear(x, xs, w, ws)
    for i in range(3):
        for j in range(4):
            acc = sum(int(a) * int(b) for a, b in zip(x[i], w[j]))
            assert y[i, j] == acc * float(xs[i]) * float(ws[j])


def test_grad_norm_matches_torch():
    rng = np.random.default_rng(6)
    gs = [rng.standard_normal(n).astype(np.float32) * 10.0 ** -i for i, n in enumerate((5, 1, 300, 64))]
    ps = [torch.nn.Parameter(torch.zeros(g.size, dtype=torch.float64)) for g in gs]
    for p, g in zip(ps, gs):
        p.grad = torch.tensor(g, dtype=torch.float64)
    total = torch.nn.utils.clip_grad_norm_(ps, 0.25)
    assert np.isclose(grads.norm(gs), float(total), rtol=1e-13)
    c = grads.coef(grads.norm(gs), 0.25)
    assert np.allclose(ps[2].grad.numpy(), gs[2].astype(np.float64) * c, rtol=1e-9)
    assert grads.coef(0.1, 0.25) == 1.0 and grads.coef(0.0, 0.0) == 0.0
