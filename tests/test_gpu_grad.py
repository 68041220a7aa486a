"""Gradient norm and clipping against fp64.

The squares of one 16-byte vector are summed in fp32 (at most 8 roundings of
2^-24, all terms positive) and everything else in fp64, so the norm is within
half of 9 * 2^-24 of the exact one plus its own rounding, 2^-24; a clipped value
is one fp32 product (factor and product: 2 * 2^-24) rounded to its type."""
import math

import numpy as np
import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu
NORM_TOL = 5.5 * 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def tensors(counts, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(dtype) for n in counts]


def exact_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def norm_of(ts):
    out = torch.full((1,), -1.0, device="cuda")
    B.grad_norm(ts, out, B.alloc_grad_workspace(len(ts)))
    return float(out)


def check_clip(ts, max_norm, out=None):
    src = [t.clone() for t in ts]
    norm = torch.full((1,), -1.0, device="cuda")
    B.grad_clip(ts, max_norm, norm, B.alloc_grad_workspace(len(ts)), out=out)
    torch.cuda.synchronize()
    n = exact_norm(src)
    assert abs(float(norm) - n) <= NORM_TOL * n
    factor = min(1.0, float(np.float32(max_norm)) / (n + 1e-6))
    for a, b, o in zip(src, ts, out or ts):
        want = a.double() * factor
        tol = (NORM_TOL + 2 * 2.0 ** -24 + HALF_STEP[a.dtype]) * want.abs() + 2.0 ** -133
        assert bool(((o.double() - want).abs() <= tol).all())
        if factor == 1.0:
            assert torch.equal(o, a)
        if out:
            assert torch.equal(a, b)


COUNTS = [[1], [7], [8191, 1, 0, 8193], [16384], [16385, 4097, 3], [100003, 5, 65536], [300000]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("place", ["in", "out"])
@pytest.mark.parametrize("clips", [True, False])
def test_clip(counts, dtype, place, clips):
    ts = tensors(counts, dtype, sum(counts))
    bound = exact_norm(ts) * (0.3 if clips else 1.5)
    check_clip(ts, bound, [torch.full_like(t, 9.0) for t in ts] if place == "out" else None)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 3), (1, 2), (5, 0), (7, 6)])
def test_views_at_odd_addresses(dtype, a, b):
    base, to = tensors([50000], dtype, 3)[0], torch.full((50016,), 9.0, dtype=dtype, device="cuda")
    v, o = base[a:a + 40001], to[b:b + 40001]
    check_clip([v], 1.0, [o])
    assert torch.all(to[:b] == 9.0) and torch.all(to[b + 40001:] == 9.0)
    keep = base.clone()
    check_clip([v], 1.0)
    assert torch.equal(base[:a], keep[:a]) and torch.equal(base[a + 40001:], keep[a + 40001:])


def test_mixed_types_and_more_tensors_than_a_launch_holds():
    ts = [t for i in range(301) for t in tensors([1 + 37 * i], torch.float32 if i % 2 else torch.bfloat16, i)]
    assert abs(norm_of(ts) - exact_norm(ts)) <= NORM_TOL * exact_norm(ts)
    check_clip(ts, 2.0)


def test_no_tensors_and_empty_tensors():
    assert norm_of([]) == 0.0
    assert norm_of([torch.empty(0, device="cuda")] * 3) == 0.0
    check_clip([torch.empty(0, device="cuda")], 1.0)


def test_all_zero():
    check_clip([torch.zeros(70000, device="cuda"), torch.zeros(5, dtype=torch.bfloat16, device="cuda")], 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-37, 1e-25, 1e-16, 1e-15, 1e14, 1e15, 1e30, 3e34])
def test_magnitudes_whose_squares_leave_fp32(dtype, scale):
    ts = tensors([70001, 12], dtype, 5, scale)
    n = exact_norm(ts)
    assert abs(norm_of(ts) - n) <= NORM_TOL * n


def test_magnitudes_far_apart_in_one_vector():
    t = torch.tensor([1e-30, 3e-16, 1e20, 2.0] * 4096, device="cuda")
    assert abs(norm_of([t]) - exact_norm([t])) <= NORM_TOL * exact_norm([t])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_gradients_show_in_the_norm(bad):
    t = tensors([50000], torch.float32, 6)[0]
    t[31234] = bad
    got = norm_of([t])
    assert math.isnan(got) if math.isnan(bad) else got == math.inf
    o = torch.empty_like(t)
    B.grad_clip([t], 1.0, None, B.alloc_grad_workspace(1), out=[o])
    if math.isnan(bad):
        assert torch.isnan(o).all()
    else:
        assert torch.isnan(o[31234]) and torch.all(torch.cat((o[:31234], o[31235:])) == 0)


def test_zero_bound():
    ts = tensors([5000], torch.bfloat16, 8)
    check_clip(ts, 0.0)
    assert torch.all(ts[0] == 0)


def test_same_bits_every_time_and_in_a_graph():
    ts = tensors([200001, 31, 70000], torch.bfloat16, 9)
    out = [torch.empty_like(t) for t in ts]
    norm, ws = torch.empty(1, device="cuda"), B.alloc_grad_workspace(3)
    call = lambda: B.grad_clip(ts, 1.0, norm, ws, out=out)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    first, n = [o.clone() for o in out], norm.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        norm.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, n) and all(torch.equal(a, b) for a, b in zip(first, out))
    ts[0].mul_(3)
    g.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - exact_norm(ts)) <= NORM_TOL * exact_norm(ts)
    del g


def test_calls_on_two_streams_with_workspaces_of_their_own():
    a, b = tensors([3000001], torch.float32, 10), tensors([2000003], torch.bfloat16, 11)
    norms = [torch.empty(1, device="cuda") for _ in range(2)]
    wss = [B.alloc_grad_workspace(1) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for ts, n, ws, st in zip((a, b), norms, wss, streams):
            B.grad_norm(ts, n, ws, stream=st)
    torch.cuda.synchronize()
    for ts, n in zip((a, b), norms):
        assert abs(float(n) - exact_norm(ts)) <= NORM_TOL * exact_norm(ts)
