"""Refusals of the norm, 8-bit linear and gradient-norm entries, without a
GPU: bad arguments are rejected before the device is touched, by the C entries
with a status and by the Python calls with ValueError."""

import ctypes

import pytest
import torch

import bit_nf4_quantized_28_b200 as qn
from bit_nf4_quantized_28_b200 import build, grads, int8, norm

P, ODD, ODD4 = ctypes.c_void_p(4096), ctypes.c_void_p(4104), ctypes.c_void_p(4098)
F = ctypes.c_float


@pytest.fixture(scope="module")
def L():
    build.build()
    return qn.lib()


def test_norm_refusals(L):
    fwd = lambda x=P, r=None, w=P, m=4, d=64, eps=1e-5, h=None, y=P, rs=P: L.rmsnorm_fwd(x, r, w, m, d, eps, h, y, rs,
                                                                                        None)
    i8 = lambda x=P, r=None, w=P, m=4, d=64, eps=1e-5, h=None, q=P, s=P: L.rmsnorm_fwd_int8(x, r, w, m, d, eps, h, q,
                                                                                          s, None)
    for f in (fwd, i8):
        assert f(m=0) == 0 and f(m=0, x=None) == 0               # nothing to do
        assert f(m=-1) == 2 and f(d=0) == 2 and f(d=12) == 2 and f(d=32768 + 8) == 2
        assert f(eps=float("nan")) == 1 and f(eps=-1.0) == 1
        assert f(x=None) == 1 and f(w=None) == 1
        assert f(r=P) == 1                                        # a residual needs h
        assert f(x=ODD) == 3 and f(w=ODD) == 3 and f(r=ODD, h=P) == 3 and f(r=P, h=ODD) == 3
    assert fwd(y=None) == 1 and fwd(y=ODD) == 3 and fwd(rs=ODD4) == 3
    assert i8(q=None) == 1 and i8(s=None) == 1 and i8(q=ODD4) == 3 and i8(s=ODD4) == 3
    assert L.rmsnorm_bwd_workspace_bytes(0, 64) == 0
    need = L.rmsnorm_bwd_workspace_bytes(1000, 64)
    assert need >= 64 * 4
    bwd = lambda dy=P, h=P, w=P, rs=P, dh=None, m=1000, d=64, dx=P, dw=P, ws=P, nb=need: L.rmsnorm_bwd(
        dy, h, w, rs, dh, m, d, dx, dw, ws, nb, None)
    assert bwd(m=0, dw=None) == 0
    assert bwd(m=-1) == 2 and bwd(d=20) == 2
    for k in ("dy", "h", "w", "rs", "dx"):
        assert bwd(**{k: None}) == 1 and bwd(**{k: ODD4 if k == "rs" else ODD}) == 3
    assert bwd(dh=ODD) == 3 and bwd(dw=ODD) == 3
    assert bwd(ws=None) == 4 and bwd(nb=need - 1) == 4 and bwd(ws=ODD) == 3


def test_int8_refusals(L):
    q = lambda x=P, m=4, k=64, c=P, s=P: L.int8_quantize_rows(x, m, k, c, s, None)
    assert q(m=0) == 0 and q(m=-1) == 2 and q(k=12) == 2 and q(k=131072) == 2
    assert q(x=None) == 1 and q(c=None) == 1 and q(s=None) == 1 and q(x=ODD) == 3 and q(c=ODD4) == 3
    lin = lambda x=P, xs=P, m=4, w=P, ws=P, n=64, k=64, y=P: L.int8_linear_fwd(x, xs, m, w, ws, n, k, y, None)
    assert lin(m=0) == 0 and lin(m=-1) == 2
    assert lin(n=0) == 2 and lin(n=12) == 2 and lin(k=24) == 2 and lin(k=0) == 2
    assert lin(k=131072) == 2                                     # sums could pass 2^31
    for a in ("x", "xs", "w", "ws", "y"):
        assert lin(**{a: None}) == 1 and lin(**{a: ODD4 if a == "xs" else ODD}) == 3


def _list(data, n, dtype):
    c = len(n)
    return qn._TensorList(c, (ctypes.c_void_p * c)(*data), (ctypes.c_int64 * c)(*n), (ctypes.c_int * c)(*dtype))


def test_grad_norm_refusals(L):
    ok = _list([4096, 8192], [10, 0], [0, 1])
    need = L.qlora_grad_norm_workspace_bytes(2)
    assert need > 0 and L.qlora_grad_norm_workspace_bytes(-1) == 0
    assert L.qlora_grad_norm_workspace_bytes(5000) > need
    f = lambda lst=ok, mx=1.0, n=P, c=P, ws=P, nb=need: L.qlora_grad_norm(
        None if lst is None else ctypes.byref(lst), F(mx), n, c, ws, nb, None)
    assert f(lst=None) == 1 and f(n=None) == 1
    for bad in (float("nan"), float("inf"), -1.0):
        assert f(mx=bad) == 1
    assert f(lst=_list([4096], [10], [2])) == 1                   # not a type of the list
    assert f(lst=_list([4096], [-1], [0])) == 2
    assert f(lst=_list([None], [10], [0])) == 1
    assert f(lst=_list([4098], [10], [0])) == 3 and f(lst=_list([4097], [10], [1])) == 3
    assert f(n=ctypes.c_void_p(4098)) == 3 and f(ws=ODD) == 3
    assert f(ws=None) == 4 and f(nb=need - 1) == 4
    clip = lambda a, b, c=P: L.qlora_grad_clip(ctypes.byref(a), None if b is None else ctypes.byref(b), c, None)
    assert clip(ok, None, None) == 1
    assert clip(ok, _list([4096], [10], [0])) == 1
    assert clip(ok, _list([4096, 8192], [11, 0], [0, 1])) == 2
    assert clip(ok, _list([4096, 8192], [10, 0], [0, 0])) == 2
    assert clip(ok, None, ctypes.c_void_p(4098)) == 3


def test_scaled_step_refusals(L):
    s = lambda scale, n=100: L.qlora_adamw8_step_scaled(P, P, scale, n, P, P, P, P, None, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1,
                                                        None)
    assert s(ctypes.c_void_p(4098)) == 3 and s(P, 0) == 0 and s(P, -1) == 2


def test_no_gpu_reports_unsupported(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert L.rmsnorm_fwd(P, None, P, 4, 64, 1e-5, None, P, None, None) == 7
    assert L.int8_quantize_rows(P, 4, 64, P, P, None) == 7
    assert L.int8_linear_fwd(P, P, 4, P, P, 64, 64, P, None) == 7
    assert L.qlora_grad_clip(ctypes.byref(_list([4096], [10], [0])), None, P, None) == 7


def test_python_calls_refuse_what_they_cannot_take():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for call in (lambda: norm.forward(x, w), lambda: norm.forward_int8(x, w), lambda: norm.forward(x[0], w),
                 lambda: norm.backward(x, x, w, s), lambda: norm.backward(x, x[0], w, s),
                 lambda: int8.quantize(x), lambda: int8.quantize(x[0]), lambda: int8.linear(q[0], s, None),
                 lambda: int8.linear(q, s, int8.Weight(4, 64, q, s)),
                 lambda: grads.TensorList([]), lambda: grads.TensorList([x]), lambda: grads.norm([x.float()]),
                 lambda: qn.adamw8_step(s, s, None, 1, 1e-3, grad_scale=s)):
        with pytest.raises(ValueError):
            call()
