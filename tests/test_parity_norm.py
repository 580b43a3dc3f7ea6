"""GPU parity of the RMS norm (bf16, backward, 8-bit) and of 8-bit rows.

Bounds, with u = 2^-24 (fp32) and 2^-8 (half a step of bf16, relative):

* h and the codes are compared bit for bit: h is one fp32 sum and one
  rounding; the codes are rint of one fp32 quotient of exact values.
* rstd: the sum of squares has positive terms only, each thread adds at most
  64 of them and the tree adds 10 levels, so it is within 75 u; half of that
  after the root, plus the division by d, the addition of eps, the root and
  the quotient: under 48 u.  scale = amax rstd / 127: 2 u more.
* y: rstd's 48 u, two products, then the rounding to bf16.
* dx = dh + rstd (g - h c1), c1 = rstd^2 mean(g h): the mean's products and
  sum are within 80 u of the sum of magnitudes, the other roundings within
  8 u of their terms; then the rounding to bf16.
* dw: each term carries 3 u; a CTA adds at most ceil(m / 148) rows, the
  second kernel at most 2 * 148 / 8 + 8 sums: bounded in units of the sum of
  magnitudes."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_28_b200 as qn
from bit_nf4_quantized_28_b200 import int8, norm
from oracle import norm as oracle
from oracle.nf4 import bf16_bits_to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
EPS = 1e-5
SHAPES = [(1, 8), (3, 64), (1, 4096), (2, 11008), (77, 1032), (5, 8200), (3, 32768), (333, 264), (1200, 4096),
          (301, 16384), (700, 24)]


def _bf16(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _inputs(m, d, residual, seed=0):
    x = _bf16(seed, m, d)
    x[:, d // 3] *= 20                                    # a channel far larger than the others
    res = _bf16(seed + 1, m, d) if residual else None
    w = (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(seed + 2))).to(torch.bfloat16)
    if m > 2:
        x[1] = 0
        if residual:
            res[1] = 0                                    # a row of zeros
    return x, res, w


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _check_y(y, h_bits, w):
    ref, rstd = oracle.forward(h_bits, _bits(w), EPS)
    assert np.all(np.abs(_f64(y) - ref) <= np.abs(ref) * (BF + 52 * U) + 1e-38)
    return rstd


def _check_codes(codes, scale, h_bits, w):
    q, s = oracle.forward_int8(h_bits, _bits(w), EPS)
    assert np.array_equal(codes.cpu().numpy(), q)
    got = _f64(scale)
    assert np.array_equal(np.isnan(got), np.isnan(s))
    ok = ~np.isnan(s)
    assert np.all(np.abs(got[ok] - s[ok]) <= s[ok] * 52 * U + 2.0 ** -149)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,d", SHAPES)
def test_forward(m, d, residual):
    x, res, w = _inputs(m, d, residual)
    cx, cr, cw = _cuda(x, res, w)
    y, h, rstd = norm.forward(cx, cw, cr, EPS)
    hb = oracle.stream(_bits(x), _bits(res) if residual else None)
    assert np.array_equal(_bits(h), hb)
    ref = _check_y(y, hb, w)
    assert np.all(np.abs(_f64(rstd) - ref) <= ref * 48 * U)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m,d", SHAPES)
def test_forward_int8(m, d, residual):
    x, res, w = _inputs(m, d, residual, seed=5)
    cx, cr, cw = _cuda(x, res, w)
    codes, scale, h = norm.forward_int8(cx, cw, cr, EPS)
    hb = oracle.stream(_bits(x), _bits(res) if residual else None)
    assert np.array_equal(_bits(h), hb)
    _check_codes(codes, scale, hb, w)


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("need_dw", [False, True])
@pytest.mark.parametrize("m,d", SHAPES)
def test_backward(m, d, need_dw, with_dh):
    h, dh, w = _inputs(m, d, with_dh, seed=9)
    dy = _bf16(12, m, d, scale=0.01)
    ch, cdh, cw, cdy = _cuda(h, dh, w, dy)
    rstd = norm.forward(ch, cw, eps=EPS)[2]
    dx, dw = norm.backward(cdy, ch, cw, rstd, dh=cdh, need_dw=need_dw)
    hv, wv, dyv, r = _f64(h), _f64(w), _f64(dy), _f64(rstd)
    dhv = _f64(dh) if with_dh else np.zeros_like(hv)
    rx, rw = oracle.backward(dyv, hv, wv, r, dhv)
    g, rc = dyv * wv, r[:, None]
    mean_mag = np.abs(g * hv).sum(1, keepdims=True) / d
    tol = np.abs(rx) * BF + 8 * U * (np.abs(rc * g) + np.abs(dhv) + np.abs(rc ** 3 * hv) * mean_mag) \
        + 80 * U * np.abs(rc ** 3 * hv) * mean_mag
    assert np.all(np.abs(_f64(dx) - rx) <= tol * (1 + BF) + 1e-38)
    if not need_dw:
        assert dw is None
        return
    mag = np.abs(dyv * hv * rc).sum(0)
    adds = -(-m // 148) + 2 * 148 // 8 + 8 + 3
    assert np.all(np.abs(_f64(dw) - rw) <= adds * U * mag + 1e-38)


@pytest.mark.parametrize("m,d", [(5000, 64), (9600, 136), (1300, 8200)])
def test_more_rows_than_ctas(m, d):
    """More short rows than the SMs hold CTAs, and long rows enough for the
    backward's ring."""
    test_forward(m, d, True)
    test_forward_int8(m, d, False)
    test_backward(m, d, False, True)
    test_backward(m, d, False, False)
    test_backward(m, d, True, True)
    test_quantize_rows(m, d)
    assert qn.device_error() == 0


def test_backward_takes_no_workspace_without_dw():
    """A workspace passed without dw is left as it was."""
    m, d = 1300, 8200
    h, _, w = _inputs(m, d, False, seed=40)
    dy = _bf16(41, m, d)
    ch, cw, cdy = _cuda(h, w, dy)
    rstd = norm.forward(ch, cw, eps=EPS)[2]
    ws = torch.full((norm.backward_workspace_bytes(m, d),), 77, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(ch)
    stream = torch.cuda.current_stream().cuda_stream
    assert qn.lib().rmsnorm_bwd(cdy.data_ptr(), ch.data_ptr(), cw.data_ptr(), rstd.data_ptr(), None, m, d,
                                dx.data_ptr(), None, ws.data_ptr(), ws.numel(), stream) == 0
    assert torch.equal(dx, norm.backward(cdy, ch, cw, rstd)[0])
    assert bool((ws == 77).all())


@pytest.mark.parametrize("m,k", [(1, 8), (3, 64), (5, 11008), (300, 4096), (4096, 264), (2, 32776), (3, 131064)])
def test_quantize_rows(m, k):
    x, _, _ = _inputs(m, k, False, seed=20)
    codes, scale = int8.quantize(x.cuda())
    q, s = oracle.quantize(_bits(x))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.all(np.abs(_f64(scale) - s) <= s * U)


@pytest.mark.parametrize("scale", [2.0 ** -133, 1e-30, 1e-18, 1e18, 1e30, 2.0 ** 125])
def test_extreme_magnitudes(scale):
    """Rows at the ends of bf16's range: the codes do not depend on the
    magnitude's place in fp32 (rstd underflows or overflows on its own)."""
    x = (torch.randn(4, 256, generator=torch.Generator().manual_seed(3)).clamp(-3, 3) * scale).to(torch.bfloat16)
    codes, s = int8.quantize(x.cuda())
    q, ref = oracle.quantize(_bits(x))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert np.all(np.abs(_f64(s) - ref) <= ref * U + 2.0 ** -149)
    w = torch.ones(256, dtype=torch.bfloat16)
    codes, _, _ = norm.forward_int8(x.cuda(), w.cuda())
    assert np.array_equal(codes.cpu().numpy(), q)


def test_codes_at_half_integers():
    """Every half-integer code, and its neighbours in bf16 (a largest value of
    127 makes 127 t / amax the value itself)."""
    half = torch.arange(-126.5, 127, 1.0)
    ties = half.to(torch.bfloat16)
    assert torch.equal(ties.float(), half)
    step = ties.view(torch.int16)
    row = torch.cat([torch.tensor([127.0, -127.0]).to(torch.bfloat16), ties, (step + 1).view(torch.bfloat16),
                     (step - 1).view(torch.bfloat16)])
    x = torch.stack([row, row * 2.0 ** -20, row * 2.0 ** 30, row * 2.0 ** -110, row * 2.0 ** 110])
    assert x.shape[1] % 8 == 4
    x = torch.nn.functional.pad(x, (0, 4))
    q, _ = oracle.quantize(_bits(x))
    assert np.array_equal(int8.quantize(x.cuda())[0].cpu().numpy(), q)
    w = torch.ones(x.shape[1], dtype=torch.bfloat16)
    assert np.array_equal(norm.forward_int8(x.cuda(), w.cuda())[0].cpu().numpy(), q)


@pytest.mark.parametrize("a,b", [(255, 255), (129, 131), (251, 193), (181, 181), (255, 129), (128, 128)])
def test_codes_next_to_half_integers(a, b):
    """Products h w whose 127 t / amax comes closest to a half-integer, and
    those that are one: 16-bit significands, found among all pairs."""
    u, v = np.meshgrid(np.arange(128, 256), np.arange(128, 256), indexing="ij")
    t, top = (u * v).ravel(), a * b
    h, w = [a], [float(b)]
    for s in range(9):
        # 254 t against odd multiples of top 2^s: zero is a tie, small is close to one
        r = (254 * t + top * 2 ** s) % (2 * top * 2 ** s)
        gap = np.minimum(r, 2 * top * 2 ** s - r)
        for i in np.argsort(gap + 2.0 ** 40 * (t > top * 2 ** s), kind="stable")[:40]:
            if t[i] <= top * 2 ** s:
                h.append(int(u.ravel()[i]))
                w.append(float(v.ravel()[i]) * 2.0 ** -s)
    n = len(h) // 8 * 8
    x = torch.tensor([h[:n], [-c for c in h[:n]]], dtype=torch.float32).to(torch.bfloat16)
    weight = torch.tensor(w[:n], dtype=torch.float32).to(torch.bfloat16)
    assert weight.float().tolist() == w[:n] and x[0].float().tolist() == h[:n]
    codes, scale, _ = norm.forward_int8(x.cuda(), weight.cuda(), eps=EPS)
    _check_codes(codes, scale, _bits(x), weight)


def test_non_finite_rows_stay_alone():
    x, _, w = _inputs(6, 512, False, seed=30)
    x[0, 5] = float("nan")
    x[2, 0] = float("inf")
    x[4, 511] = float("-inf")
    x[5] = 0
    hb = _bits(x)
    codes, scale, _ = norm.forward_int8(x.cuda(), w.cuda(), eps=EPS)
    _check_codes(codes, scale, hb, w)
    q, s = int8.quantize(x.cuda())
    oq, os_ = oracle.quantize(hb)
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(np.isnan(_f64(s)), np.isnan(os_)) and _f64(s)[5] == 0
    y, _, rstd = norm.forward(x.cuda(), w.cuda(), eps=EPS)
    good = [1, 3, 5]
    ref, _ = oracle.forward(hb[good], _bits(w), EPS)
    got = _f64(y)
    assert np.all(np.abs(got[good] - ref) <= np.abs(ref) * (BF + 52 * U))
    assert np.isnan(got[0]).all() and np.isnan(got[2, 0]) and np.isnan(got[4, 511])


def test_aliased_outputs_and_rows_behind_the_last():
    """h over the residual, dx over dh, y over x; rows of the buffers behind
    the last row keep what they held."""
    m, d = 9, 1032
    x, res, w = _inputs(m, d, True, seed=40)
    cx, cr, cw = _cuda(x, res, w)
    y0, h0, rstd0 = norm.forward(cx, cw, cr)
    big = torch.full((m + 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((m + 3, d), 9, dtype=torch.int8, device="cuda")
    scale = torch.full((m + 3,), 5.0, device="cuda")
    big[:m] = cr
    norm.forward_int8(cx, cw, big[:m], h=big[:m], codes=codes[:m], scale=scale[:m])
    assert torch.equal(big[:m], h0) and bool((big[m:] == 7).all())
    assert bool((codes[m:] == 9).all()) and bool((scale[m:] == 5).all())
    x2 = cx.clone()
    y, h, rstd = norm.forward(x2, cw, cr, y=x2)
    assert y is x2 and torch.equal(y, y0) and torch.equal(h, h0) and torch.equal(rstd, rstd0)
    dy = _bf16(41, m, d).cuda()
    want, _ = norm.backward(dy, h0, cw, rstd0, dh=cr)
    big[:m] = cr
    got, _ = norm.backward(dy, h0, cw, rstd0, dh=big[:m], out=(big[:m], None))
    assert torch.equal(got, want) and bool((big[m:] == 7).all())


def test_zero_row_without_eps():
    """eps = 0: a row of zeros still has scale 0 and codes 0."""
    x, _, w = _inputs(4, 64, False, seed=60)
    codes, scale, _ = norm.forward_int8(x.cuda(), w.cuda(), eps=0.0)
    assert float(scale[1]) == 0 and not codes[1].any() and bool(torch.isfinite(scale).all())


def test_slices_of_a_batch():
    """Rows in the middle of larger buffers: codes and values stand on 16-byte
    boundaries there, one-per-row values on 4-byte ones."""
    x, res, w = _cuda(*_inputs(9, 72, True, seed=61))
    y, h, rstd = norm.forward(x, w, res)
    codes, scale, _ = norm.forward_int8(x, w, res)
    q, s = int8.quantize(x)
    dy = _bf16(62, 9, 72).cuda()
    dx, _ = norm.backward(dy, h, w, rstd, dh=res)
    big = [torch.zeros_like(t) for t in (y, h, rstd, codes, scale, q, s)]
    a, b = 3, 8
    cut = [t[a:b] for t in big]
    norm.forward(x[a:b], w, res[a:b], y=cut[0], h=cut[1], rstd=cut[2])
    norm.forward_int8(x[a:b], w, res[a:b], codes=cut[3], scale=cut[4], h=cut[1])
    int8.quantize(x[a:b], codes=cut[5], scale=cut[6])
    for t, want in zip(big, (y, h, rstd, codes, scale, q, s)):
        assert torch.equal(t[a:b], want[a:b]) and not t[:a].any() and not t[b:].any()
    got, _ = norm.backward(dy[a:b], h[a:b], w, rstd[a:b], dh=res[a:b])
    assert torch.equal(got, dx[a:b])


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = norm.forward(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    assert norm.forward_int8(x, w, residual=x)[0].shape == (0, 64)
    dx, dw = norm.backward(x, x, w, rstd, need_dw=True)
    assert dx.shape == (0, 64) and not dw.any()
    assert int8.quantize(x)[0].shape == (0, 64)


def test_other_stream_and_graph():
    """On a side stream, and captured once and replayed on new inputs."""
    x, res, w = _cuda(*_inputs(50, 4096, True, seed=50))
    want = norm.forward_int8(x, w, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = norm.forward_int8(x, w, res)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dy = _bf16(51, 50, 4096).cuda()
    ws = torch.empty(norm.backward_workspace_bytes(50, 4096), dtype=torch.uint8, device="cuda")
    xs = x.clone()

    def step():
        y, h, rstd = norm.forward(xs, w, res)
        return (y, h, rstd) + norm.backward(dy, h, w, rstd, dh=res, need_dw=True, workspace=ws)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    xs.copy_(res)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))
    assert qn.device_error() == 0


def test_workspace_too_small():
    x, _, w = _cuda(*_inputs(50, 64, False))
    rstd = norm.forward(x, w)[2]
    with pytest.raises(qn.QNError):
        norm.backward(x, x, w, rstd, need_dw=True, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for bad in (x[:, :32], x.float(), x.t()):
        with pytest.raises(ValueError):
            norm.forward(bad, w)
