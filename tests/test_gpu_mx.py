"""MXFP4 quantisation, reading back and the grouped product against fp64 on the CPU.

Quantisation is compared code for code: dividing by a power of two is exact and
the one rounding is to nearest even, so there is one right answer.  The product
of two 4-bit values and its scale are exact in fp32, so the product's error is
the accumulation's alone: at most one fp32 step (2^-23 of the sum of magnitudes)
for each of the K / 64 accumulating instructions plus what one instruction sums
inside, taken as as many steps again; a bf16 result adds half a step, 2^-8."""
import numpy as np
import pytest
import torch

import mx_ref
from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu
U8 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def randn(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def spread(rows, cols, seed):
    """Rows whose magnitudes reach from subnormal to the largest fp32 values."""
    v = randn(rows, cols, seed=seed).double()
    e = torch.linspace(-150, 125, rows, dtype=torch.float64)[:, None]
    return (v * torch.exp2(e)).clamp(-3.0e38, 3.0e38).float()


def quantised(src, up=None):
    *lead, cols = src.shape
    codes = torch.full((*lead, cols // 2), 0xAA, dtype=U8, device="cuda")
    scales = torch.full((*lead, cols // 32), 0xAA, dtype=U8, device="cuda")
    B.mx_quantise(src, codes, scales, up=up)
    return codes, scales


def assert_codes(codes, scales, v):
    code, byte = mx_ref.quantise(v)
    assert np.array_equal(scales.cpu().numpy(), byte)
    assert np.array_equal(codes.cpu().numpy(), mx_ref.pack(code))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (257, 352), (64, 2048)])
def test_rows(rows, cols, dtype):
    v = randn(rows, cols, seed=rows, dtype=dtype)
    v[0, :32] = 0
    assert_codes(*quantised(v.cuda()), v.double().numpy())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_every_magnitude_ties_and_non_finite_values(dtype):
    v = spread(276, 64, 5).to(dtype)
    # every midpoint of the grid, both signs, at several scales
    mid = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.5, 0.0, -0.0] * 3)[:32]
    for r in range(8):
        v[r, :32] = (mid * (-1) ** r * 2.0 ** (3 * r - 12)).to(dtype)
    v[20, 3], v[21, 40], v[22, 63] = float("inf"), float("nan"), float("-inf")
    codes, scales = quantised(v.cuda())
    assert_codes(codes, scales, v.double().numpy())
    back = torch.empty(276, 64, dtype=dtype, device="cuda")
    B.mx_dequantise(codes, scales, back)
    want = mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(back.cpu().double().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,ld", [(0, 96), (1, 96), (0, 97), (3, 101), (8, 104)])
def test_rows_with_strides_and_odd_addresses(dtype, offset, ld):
    base = randn(9 * ld + 16, seed=7, dtype=dtype).cuda()
    v = base[offset:offset + 9 * ld].view(9, ld)[:, :96]
    assert_codes(*quantised(v), v.double().cpu().numpy())


def test_no_rows():
    e = lambda *s: torch.empty(*s, dtype=U8, device="cuda")
    B.mx_quantise(torch.empty(0, 64, device="cuda"), e(0, 32), e(0, 2))
    B.mx_dequantise(e(0, 32), e(0, 2), torch.empty(0, 64, device="cuda"))
    B.mx_quantise_weights(torch.empty(0, 64, 5, device="cuda"), e(0, 5, 32), e(0, 5, 2))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gated_rows(dtype):
    g, u = randn(65, 256, seed=1, dtype=dtype) * 2, randn(65, 256, seed=2, dtype=dtype)
    codes, scales = quantised(g.cuda(), u.cuda())
    gd, ud = g.double().numpy(), u.double().numpy()
    h = gd / (1 + np.exp(-gd)) * ud
    # h is off by a few fp32 steps: a code may only differ where h lies that
    # near a border of the grid, so the values agree with those of h moved by
    # 8 steps down or up (the scale's borders included)
    got = mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy())
    sides = [mx_ref.quantise(h * (1 + s * 8 * 2.0 ** -24)) for s in (-1, 0, 1)]
    sides = [mx_ref.values(mx_ref.pack(c), b) for c, b in sides]
    assert np.all((got == sides[0]) | (got == sides[1]) | (got == sides[2]))
    assert np.mean(got == sides[1]) > 0.999


def test_gated_rows_whose_product_alone_overflows():
    # g u is -infinite in fp32.  silu(-120) = -120 e^-120 = -9e-51 is 0 in fp32;
    # silu(-80) 3e38 = -433164 is 6 of 2^16 (the border to the next code down, 5 of
    # 2^16, lies 24% away)
    g = torch.full((2, 32), -120.0)
    g[1, 3] = -80.0
    codes, scales = quantised(g.cuda(), torch.full((2, 32), 3e38).cuda())
    want = np.zeros((2, 32))
    want[1, 3] = -6 * 2.0 ** 16
    assert np.array_equal(mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy()), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,K,N", [(1, 32, 1), (2, 96, 7), (1, 256, 64), (3, 288, 66), (2, 1024, 129), (1, 7168, 10)])
def test_weights(E, K, N, dtype):
    W = randn(E, K, N, seed=N, dtype=dtype)
    W[0, :32, 0] = 0
    W[-1, 5, N - 1] = float("nan")
    codes = torch.full((E, N, K // 2), 0xAA, dtype=U8, device="cuda")
    scales = torch.full((E, N, K // 32), 0xAA, dtype=U8, device="cuda")
    B.mx_quantise_weights(W.cuda(), codes, scales)
    assert_codes(codes, scales, W.double().numpy().transpose(0, 2, 1))


def operands(counts, K, N, seed):
    rows, E = sum(counts), len(counts)
    rng = np.random.default_rng(seed)
    a = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    w = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    sa = rng.integers(118, 130, (rows, K // 32), dtype=np.uint8)
    sw = rng.integers(112, 132, (E, N, K // 32), dtype=np.uint8)
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    return a, sa, off, w, sw


def product(a, sa, off, w, sw, dtype=torch.float32, rows=None, fill=7.0):
    rows = a.shape[0] if rows is None else rows
    g = lambda t: torch.as_tensor(t).cuda()
    Y = torch.full((a.shape[0], w.shape[1]), fill, dtype=dtype, device="cuda")
    ws = B.alloc_mx_product_workspace(a.shape[0], w.shape[0])
    B.mx_grouped_product(g(a), g(sa), g(off), g(w), g(sw), Y, ws)
    rc, raw = B.check_device_status(ws)
    return Y, rc


def reference(a, sa, off, w, sw):
    """(the product, the sum of its terms' magnitudes) in fp64."""
    A = mx_ref.values(a, sa)
    y, m = np.zeros((a.shape[0], w.shape[1])), np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        W = mx_ref.values(w[e], sw[e])
        s = slice(off[e], off[e + 1])
        y[s], m[s] = A[s] @ W.T, np.abs(A[s]) @ np.abs(W).T
    return y, m


def assert_product(Y, y, m, K):
    got = Y.double().cpu().numpy()
    bound = m * 2 * (K / 64) * 2.0 ** -23
    if Y.dtype == torch.bfloat16:
        bound = bound + np.abs(y) * 2.0 ** -8
    assert np.all(np.abs(got - y) <= bound), (np.abs(got - y) / np.maximum(bound, 1e-300)).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,K,N", [
    ([1], 128, 128),
    ([16], 256, 128),
    ([0, 1, 0, 3, 0], 384, 256),
    ([17, 33, 48, 49, 64, 65], 512, 128),
    ([127, 128, 129], 640, 384),
    ([191, 192, 193, 385], 256, 128),
    ([5] * 64, 128, 256),
    ([300, 0, 2], 7168, 128),
])
def test_product(counts, K, N, dtype):
    args = operands(counts, K, N, seed=K + N)
    Y, rc = product(*args, dtype=dtype)
    assert rc == B.MOE_OK
    assert_product(Y, *reference(*args), K)


def test_product_leaves_rows_behind_the_last_segment():
    a, sa, off, w, sw = operands([3, 20, 41], 256, 128, 3)
    off = np.array([2, 10, 30], dtype=np.int32)
    Y, rc = product(a, sa, off, w[:2], sw[:2])
    assert rc == B.MOE_OK
    y, m = reference(a, sa, off, w[:2], sw[:2])
    assert torch.all(Y[:2] == 7.0) and torch.all(Y[30:] == 7.0)
    assert_product(Y[2:30], y[2:30], m[2:30], 256)


def test_product_skips_bad_offsets_and_reports_them():
    a, sa, _, w, sw = operands([8, 8, 8, 8], 128, 128, 4)
    off = np.array([0, 8, 4, 20, 900], dtype=np.int32)  # expert 1 descends, expert 3 ends past the rows
    Y, rc = product(a, sa, off, w, sw)
    assert rc == B.MOE_ERR_DEVICE_BOUNDS
    y, m = reference(a, sa, np.array([0, 8, 8, 8, 8]), w, sw)
    assert_product(Y[:4], y[:4], m[:4], 128)
    assert torch.all(Y[20:] == 7.0)


def test_product_keeps_extreme_scales_and_nan_to_their_rows():
    a, sa, off, w, sw = operands([40], 256, 128, 5)
    sa[3], sw[0, 9] = 0, 0            # 2^-127 on one side
    sa[7, 2] = 255                    # a NaN block: row 7 is NaN, no other
    Y, rc = product(a, sa, off, w, sw)
    y, m = reference(a, sa, off, w, sw)
    got = Y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(y)) and np.isnan(y[7]).all() and not np.isnan(y[:7]).any()
    ok = ~np.isnan(y)
    # products below 2^-126 may lose bits to fp32's subnormal spacing
    assert np.all(np.abs(got - y)[ok] <= (m * 2 * 4 * 2.0 ** -23 + 2.0 ** -126)[ok])


def test_product_is_deterministic_and_replays_in_a_graph():
    args = operands([100, 3, 250, 0, 31], 512, 256, 6)
    a, sa, off, w, sw = [torch.as_tensor(t).cuda() for t in args]
    Y = torch.empty(a.shape[0], 256, device="cuda")
    ws = B.alloc_mx_product_workspace(a.shape[0], 5)
    call = lambda: B.mx_grouped_product(a, sa, off, w, sw, Y, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    first = Y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    Y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, first)
    off.copy_(torch.tensor([0, 3, 103, 103, 353, 384], dtype=torch.int32))  # other loads, the same graph
    g.replay()
    torch.cuda.synchronize()
    y, m = reference(args[0], args[1], off.cpu().numpy(), args[3], args[4])
    assert_product(Y, y, m, 512)
    del g
