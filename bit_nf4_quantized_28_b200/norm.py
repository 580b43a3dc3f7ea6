"""RMS norm with the residual addition, between the linears of a block.

    y, h, rstd = forward(x, weight, residual)        # h = x + residual, y = norm(h) * weight
    dx, dw = backward(dy, h, weight, rstd, dh)       # dh: gradient of h from the residual stream
    codes, scale, h = forward_int8(x, weight, residual)   # y in 8 bits, for int8.linear

x, residual and the outputs are bf16 [m, d] (contiguous), weight bf16 [d];
d % 8 == 0 and d <= 32768.  The calls run on the tensors' device, on its
current stream.  Formulas and rounding: include/qlora_nf4.h.
"""

import torch

from . import _arg, _out, _run, lib

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(x, weight, residual, h):
    if x.dim() != 2:
        raise ValueError(f"x: [m, d] is needed, got {tuple(x.shape)}")
    dev = x.device
    px = _arg(x, "x", BF16, x.shape)
    pr = _arg(residual, "residual", BF16, x.shape, dev)
    pw = _arg(weight, "weight", BF16, x.shape[1:], dev)
    if residual is None:
        return px, None, pw, x, None
    return px, pr, pw, *_out(h, "h", BF16, x.shape, dev, x)


def forward(x, weight, residual=None, eps=1e-5, y=None, h=None, rstd=None):
    """(y, h, rstd): h = x + residual (x itself without a residual), rstd fp32
    [m] for the backward.  Outputs given are written in place; h may be x or
    residual."""
    px, pr, pw, h, ph = _inputs(x, weight, residual, h)
    m, d = x.shape
    dev = x.device
    y, py = _out(y, "y", BF16, x.shape, dev, x)
    rstd, ps = _out(rstd, "rstd", F32, (m,), dev)
    _run("rmsnorm_fwd", dev, px, pr, pw, m, d, eps, ph, py, ps)
    return y, h, rstd


def forward_int8(x, weight, residual=None, eps=1e-5, codes=None, scale=None, h=None):
    """(codes, scale, h): the norm's output as int8 codes [m, d] with one fp32
    scale per row; codes * scale stands for y."""
    px, pr, pw, h, ph = _inputs(x, weight, residual, h)
    m, d = x.shape
    dev = x.device
    codes, pc = _out(codes, "codes", torch.int8, x.shape, dev, x)
    scale, ps = _out(scale, "scale", F32, (m,), dev)
    _run("rmsnorm_fwd_int8", dev, px, pr, pw, m, d, eps, ph, pc, ps)
    return codes, scale, h


def backward_workspace_bytes(m, d):
    return lib().rmsnorm_bwd_workspace_bytes(m, d)


def backward(dy, h, weight, rstd, dh=None, need_dw=False, out=None, workspace=None):
    """(dx, dw) of forward: dx bf16 [m, d] is the gradient of x and of
    residual; dw fp32 [d] (None unless need_dw: QLoRA trains the adapters
    only).  dh: None or the gradient that reaches h from the residual stream.
    out: (dx, dw) to write into; dx may be dy or dh."""
    if h.dim() != 2:
        raise ValueError(f"h: [m, d] is needed, got {tuple(h.shape)}")
    dev = h.device
    m, d = shape = h.shape
    dx, dw = out if out is not None else (None, None)
    need_dw = dw is not None if out is not None else need_dw
    args = (_arg(dy, "dy", BF16, shape, dev), _arg(h, "h", BF16, shape), _arg(weight, "weight", BF16, (d,), dev),
            _arg(rstd, "rstd", F32, (m,), dev), _arg(dh, "dh", BF16, shape, dev))
    dx, px = _out(dx, "dx", BF16, shape, dev, h)
    dw, pw = _out(dw, "dw", F32, (d,), dev) if need_dw else (None, None)
    nbytes = 0
    if need_dw:
        nbytes = backward_workspace_bytes(m, d) if workspace is None else workspace.numel()
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        elif workspace.dtype is not torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous uint8 tensor on {dev} is needed")
    _run("rmsnorm_bwd", dev, *args, m, d, px, pw, workspace.data_ptr() if need_dw else None, nbytes)
    return dx, dw
