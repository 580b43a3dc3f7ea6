"""GPU parity of the global gradient norm, the clipping and the optimizer step
that takes the coefficient.

Squares and sums are fp64 (n 2^-53 of the sum, nothing at these sizes), so the
norm is within one fp32 rounding (2^-24) and 2^-40; the coefficient adds the
rounding of 1e-6's sum and of the quotient.  A clipped value is one product
rounded to its type: within 2^-24 (fp32) or 2^-8 and 2^-24 (bf16) of g coef."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_28_b200 as qn
from bit_nf4_quantized_28_b200 import grads
from oracle import grads as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def _make(sizes, dtypes, seed=0, offset=0):
    """Tensors of these sizes, cut out of buffers `offset` values past their start."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, (n, dt) in enumerate(zip(sizes, dtypes)):
        off = (offset * (i + 1)) % 8
        buf = torch.zeros(n + off, dtype=dt)
        buf[off:] = (torch.randn(n, generator=g) * 10.0 ** (-(i % 5))).to(dt)
        out.append(buf.cuda()[off:])
    return out


def _np(ts):
    return [t.cpu().double().numpy().ravel() for t in ts]


def _check(ts, max_norm, total, coef):
    ref = oracle.norm(_np(ts))
    assert abs(float(total) - ref) <= ref * (U + 2.0 ** -40)
    c = oracle.coef(ref, max_norm)
    assert abs(float(coef) - c) <= 5 * U * c
    return c


CASES = [([1], [F32]), ([5], [BF16]), ([4096], [F32]), ([4095, 4097, 1, 8191], [F32, BF16, F32, BF16]),
         ([100000, 3, 70000, 0, 12345], [F32, F32, BF16, F32, BF16]), ([16 * 4096, 16 * 11008] * 7, [F32] * 14),
         ([17] * 300, [F32, BF16] * 150), ([1234567], [BF16])]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("sizes,dtypes", CASES)
def test_norm_and_clip(sizes, dtypes, offset):
    ts = _make(sizes, dtypes, seed=len(sizes), offset=offset)
    for max_norm in (0.3, 1e9, 0.0):
        total, coef = grads.norm(ts, max_norm)
        _check(ts, max_norm, total, coef)
    total, coef = grads.norm(ts, 0.3)
    c = float(coef)
    before = _np(ts)
    # into other buffers, aligned differently, with what surrounds them kept
    bufs = [torch.full((t.numel() + 9,), 7.0, dtype=t.dtype, device="cuda") for t in ts]
    outs = [b[(i % 5):(i % 5) + t.numel()] for i, (b, t) in enumerate(zip(bufs, ts))]
    grads.clip(ts, coef, out=outs)
    for i, (b, o, t, g) in enumerate(zip(bufs, outs, ts, before)):
        tol = np.abs(g * c) * (U if t.dtype is F32 else 2.0 ** -8 + 2 * U) + 2.0 ** -149
        assert np.all(np.abs(o.cpu().double().numpy() - g * c) <= tol)
        assert bool((b[:i % 5] == 7).all()) and bool((b[i % 5 + t.numel():] == 7).all())
    for t, g in zip(ts, before):
        assert np.array_equal(t.cpu().double().numpy(), g)         # the gradients are inputs
    grads.clip(ts, coef)
    assert all(torch.equal(a, b) for a, b in zip(ts, outs))


def test_many_tensors():
    """More tensors than one launch takes, and a list with nothing in it."""
    ts = _make([33] * 2500, [F32] * 2500, seed=4)
    total, coef = grads.norm(ts, 0.5)
    c = _check(ts, 0.5, total, coef)
    want = [t * coef for t in ts]
    grads.clip(ts, coef)
    assert c < 1 and all(torch.equal(a, b) for a, b in zip(ts, want))
    none = [torch.empty(0, device="cuda"), torch.empty(0, dtype=BF16, device="cuda")]
    total, coef = grads.norm(none, 1.0)
    assert float(total) == 0 and float(coef) == 1
    grads.clip(none, coef)


@pytest.mark.parametrize("value", [1e25, 3e38, 1e-25, 1e-40])
def test_no_overflow_and_no_underflow(value):
    """Squares beyond fp32's range."""
    ts = [torch.full((1000,), value, device="cuda"), torch.full((24,), -value, device="cuda")]
    ref = oracle.norm(_np(ts))
    total, _ = grads.norm(ts)
    if ref < 3.4e38:
        assert abs(float(total) - ref) <= ref * (U + 2.0 ** -40) + 2.0 ** -149
    else:
        assert float(total) == float("inf")


def test_non_finite_gradients():
    ts = _make([5000, 300], [F32, BF16], seed=6)
    ts[0][4321] = float("inf")
    total, coef = grads.norm(ts, 1.0)
    assert float(total) == float("inf") and float(coef) == 0
    ts[1][7] = float("nan")
    total, coef = grads.norm(ts, 1.0)
    assert np.isnan(float(total)) and np.isnan(float(coef))


def test_nothing_to_clip_in_place_keeps_the_bits():
    ts = _make([9000, 77], [F32, BF16], seed=7)
    before = [t.clone() for t in ts]
    total, coef = grads.norm(ts, 1e6)
    assert float(coef) == 1
    grads.clip(ts, coef)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))


@pytest.mark.parametrize("n", [250, 4096 + 24, 1 << 18])
def test_step_with_coefficient(n):
    """adamw8_step(grad_scale=c) is the step on the products fl32(g c), bit
    for bit; without a coefficient, and with 1, it is the plain step."""
    g = torch.randn(n, generator=torch.Generator().manual_seed(n)).cuda()
    total, coef = grads.norm([g], 0.3)

    def run(grad, scale):
        p = torch.linspace(-1, 1, n, device="cuda")
        st = qn.AdamW8State.zeros(n)
        pb = torch.empty(n, dtype=BF16, device="cuda")
        for t in (1, 2, 3):
            qn.adamw8_step(p, grad, st, t, lr=1e-3, weight_decay=0.01, param_bf16=pb, grad_scale=scale)
        return p, pb, st.m_codes, st.m_scale, st.v_codes, st.v_scale

    for a, b in zip(run(g, coef), run(g * coef, None)):
        assert torch.equal(a, b)
    for a, b in zip(run(g, torch.ones((), device="cuda")), run(g, None)):
        assert torch.equal(a, b)


def test_equal_bits_each_time_streams_and_graph():
    ts = _make([100001, 4097, 65536], [F32, BF16, F32], seed=8)
    lst, ws = grads.TensorList(ts), None
    first = grads.norm(lst, 0.3)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(grads.norm(lst, 0.3), first))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = grads.norm(lst, 0.3, workspace=grads.make_workspace(lst))
    s.synchronize()
    assert torch.equal(side[0], first[0])
    ws = grads.make_workspace(lst)
    out = torch.empty(2, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        total, coef = grads.norm(lst, 0.3, out=out, workspace=ws)
        grads.clip(lst, coef)
    ts[0].mul_(3)
    want = grads.norm(lst, 0.3)
    expect = [t * want[1] if t.dtype is F32 else (t.float() * want[1]).to(BF16) for t in ts]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(total, want[0]) and torch.equal(coef, want[1])
    assert all(torch.equal(a, b) for a, b in zip(ts, expect))


def test_refusals():
    t = torch.ones(16, device="cuda")
    for bad in (t.double(), t.view(4, 4).t(), t.cpu()):
        with pytest.raises(ValueError):
            grads.norm([t, bad])
    for bad in (float("inf"), float("nan"), -1.0):
        with pytest.raises(qn.QNError):
            grads.norm([t], bad)
    with pytest.raises(qn.QNError):
        grads.norm([t], 1.0, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    c = torch.ones((), device="cuda")
    with pytest.raises(ValueError):
        grads.clip([t], t)
    with pytest.raises(qn.QNError):
        grads.clip([t], c, out=[t, t])
    with pytest.raises(qn.QNError):
        grads.clip([t], c, out=[torch.ones(15, device="cuda")])


def test_one_workspace_for_lists_of_any_length():
    """A workspace made for the longest list serves the others too, in any
    order: every call leaves its counter zero."""
    short, long = _make([500, 70000], [F32, BF16], seed=9), _make([3000] * 1500, [F32] * 1500, seed=10)
    ws = grads.make_workspace(long)
    for ts in (short, long, short, [torch.empty(0, device="cuda")], long, long, short):
        total, coef = grads.norm(ts, 0.3, workspace=ws)
        _check(ts, 0.3, total, coef)
