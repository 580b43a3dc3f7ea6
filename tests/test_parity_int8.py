"""GPU parity of the linear in 8-bit integers.

The sums are exact integers; y carries the rounding of the sum to fp32, of
the scales' product and of their product (3 u, u = 2^-24) and half a step of
bf16 (2^-8 relative)."""

import numpy as np
import pytest
import torch

import bit_nf4_quantized_28_b200 as qn
from bit_nf4_quantized_28_b200 import int8
from oracle import int8 as oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8


def _operands(m, n, k, seed=0, extreme=False):
    g = torch.Generator().manual_seed(seed)
    if extreme:
        x, w = torch.full((m, k), -128, dtype=torch.int8), torch.full((n, k), -128, dtype=torch.int8)
        w[1::2] = 127
    else:
        x = torch.randint(-128, 128, (m, k), generator=g, dtype=torch.int8)
        w = torch.randint(-128, 128, (n, k), generator=g, dtype=torch.int8)
    return x, torch.rand(m, generator=g) + 0.1, w, torch.rand(n, generator=g) * 0.01 + 1e-4


def _weight(w, ws):
    return int8.Weight(w.shape[0], w.shape[1], w.cuda(), ws.cuda())


def _check(y, x, xs, w, ws):
    # exact: products of 8-bit values sum below 2^31, which fp64 holds
    ref = (x.cuda().double() @ w.cuda().double().T).cpu().numpy() * xs.double().numpy()[:, None] \
        * ws.double().numpy()[None, :]
    if ref.size <= 1 << 16:
        assert np.array_equal(ref, oracle.linear(x.numpy(), xs.numpy(), w.numpy(), ws.numpy()))
    got = y.cpu().double().numpy()
    assert np.all(np.abs(got - ref) <= np.abs(ref) * (BF + 4 * U))


MS = [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 100, 128, 129, 200, 256, 257, 300, 511, 700]


@pytest.mark.parametrize("m", MS)
@pytest.mark.parametrize("n,k", [(8, 16), (264, 144), (1000, 2064), (4096, 4096)])
def test_sizes(m, n, k):
    x, xs, w, ws = _operands(m, n, k, seed=m)
    _check(int8.linear(x.cuda(), xs.cuda(), _weight(w, ws)), x, xs, w, ws)
    assert qn.device_error() == 0


@pytest.mark.parametrize("k", [16, 32, 48, 64, 80, 112, 128, 144, 240, 256, 272, 400, 528, 1040, 11008])
@pytest.mark.parametrize("m,n", [(1, 40), (12, 136), (40, 520), (130, 264), (520, 776)])
def test_widths(m, n, k):
    x, xs, w, ws = _operands(m, n, k, seed=k)
    _check(int8.linear(x.cuda(), xs.cuda(), _weight(w, ws)), x, xs, w, ws)


@pytest.mark.parametrize("m", [1, 16, 64, 300])
def test_largest_sums(m):
    """Every product at its extreme and the longest k: sums of 2^31 - 262144."""
    x, xs, w, ws = _operands(m, 16, 131056, extreme=True)
    _check(int8.linear(x.cuda(), xs.cuda(), _weight(w, ws)), x, xs, w, ws)


@pytest.mark.parametrize("m,n,k", [(2048, 4096, 4096), (1, 11008, 4096), (16, 4096, 11008), (3000, 11008, 1024)])
def test_full_sizes(m, n, k):
    x, xs, w, ws = _operands(m, n, k, seed=1)
    _check(int8.linear(x.cuda(), xs.cuda(), _weight(w, ws)), x, xs, w, ws)


@pytest.mark.parametrize("m", [0, 1, 5, 16, 50, 130, 300])
def test_rows_behind_the_last_and_bad_scales(m):
    """Rows of y behind row m keep what they held; a NaN scale of a token (or
    of a channel) spoils its own row (or column) only."""
    n, k = 200, 272
    x, xs, w, ws = _operands(m, n, k, seed=3)
    y = torch.full((m + 4, n), 7.0, dtype=torch.bfloat16, device="cuda")
    if m > 1:
        xs[1] = float("nan")
    ws[5] = float("nan")
    int8.linear(x.cuda(), xs.cuda(), _weight(w, ws), y=y[:m])
    assert bool((y[m:] == 7).all())
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[:, 5] = True
    if m > 1:
        bad[1] = True
    assert torch.equal(torch.isnan(y[:m]).cpu(), bad)
    if m > 2:
        keep = [i for i in range(m) if i != 1]
        cols = [i for i in range(n) if i != 5]
        ref = oracle.linear(x[keep].numpy(), xs[keep].numpy(), w[cols].numpy(), ws[cols].numpy())
        got = y[:m].cpu().double().numpy()[np.ix_(keep, cols)]
        assert np.all(np.abs(got - ref) <= np.abs(ref) * (BF + 4 * U))


@pytest.mark.parametrize("m", [1, 12, 60, 400])
def test_streams_and_graph(m):
    """Two calls at once on two streams; captured and replayed on new tokens."""
    x, xs, w, ws = _operands(m, 520, 1040, seed=4)
    W = _weight(w, ws)
    x, xs = x.cuda(), xs.cuda()
    want = int8.linear(x, xs, W)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got += [int8.linear(x, xs, W) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)
    xc = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = int8.linear(xc, xs, W)
    xc.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, int8.linear(x.flip(0).contiguous(), xs, W))
    assert qn.device_error() == 0


@pytest.mark.parametrize("m", [3, 20, 300])
def test_slices_of_a_batch(m):
    """Tokens in the middle of a larger batch."""
    x, xs, w, ws = _operands(m + 9, 264, 528, seed=6)
    W = _weight(w, ws)
    x, xs = x.cuda(), xs.cuda()
    got = int8.linear(x[5:5 + m], xs[5:5 + m], W)
    assert torch.equal(got, int8.linear(x, xs, W)[5:5 + m])


def test_refusals():
    x, xs, w, ws = _operands(4, 16, 32)
    W = _weight(w, ws)
    for bad in (x.cuda()[:, :16], x.cuda().t(), x.cuda().float(), x):
        with pytest.raises(ValueError):
            int8.linear(bad, xs.cuda(), W)
    with pytest.raises(ValueError):
        int8.linear(x.cuda(), xs.cuda()[:3], W)
    with pytest.raises(qn.QNError):
        int8.linear(x.cuda(), xs.cuda(), _weight(w[:12], ws[:12]))
