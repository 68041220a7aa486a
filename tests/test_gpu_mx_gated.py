"""Quantisation of silu(g) * u where silu(g) is small: far below fp32's steps at 1, down to
its smallest numbers, with u large enough that the products matter."""
import numpy as np
import pytest
import torch

import mx_ref
from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def gated_values(g, u):
    rows, cols = g.shape
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    B.mx_quantise(g.cuda(), codes, scales, up=u.cuda())
    return mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy())


def check(g, u):
    got = gated_values(g, u)
    gd, ud = g.double().numpy(), u.double().numpy()
    h = gd / (1 + np.exp(-gd)) * ud
    # expf is good to 2 steps, of 2^-149 where the result is subnormal; the sum, the
    # reciprocal (2 steps) and the products: 8 steps of 2^-24 in all beside it.  A code may
    # differ only where h moved by so much down or up takes another one (a block's rows
    # share g, so that they move together).
    off = 8 * 2.0 ** -24 + np.where(gd < 0, 2 * 2.0 ** -149 / np.exp(gd), 0.0)
    sides = [mx_ref.quantise(h * (1 + s * off)) for s in (-1, 0, 1)]
    sides = [mx_ref.values(mx_ref.pack(c), b) for c, b in sides]
    assert np.all((got == sides[0]) | (got == sides[1]) | (got == sides[2]))
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_silu_times_large_u(dtype):
    # every quarter from -98 (e^-98 is 2^7.6 of fp32's smallest number) to -60
    g = torch.arange(-98, -60, 0.25)[:, None].repeat(1, 64).to(dtype)
    u = torch.randn(g.shape, generator=torch.Generator().manual_seed(1)).clamp(-4, 4) * 2.0 ** 124
    got = check(g, u.to(dtype))
    assert np.all(np.abs(got).max(1) > 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_where_the_exponential_of_minus_g_is_largest(dtype):
    # -88 3e38 silu'(...): about -160, where e^88 is above 2^126
    g = torch.full((2, 32), -88.0).to(dtype)
    g[1] = -87.5
    got = check(g, torch.full((2, 32), 3e38).to(dtype))
    assert np.all(got < -100)


def test_large_g_and_non_finite_values():
    g = torch.tensor([[100.0] * 32, [88.5] * 32, [float("nan")] * 32, [float("inf")] * 32])
    got = gated_values(g, torch.ones(4, 32))
    assert np.all(got[0] == 96) and np.all(got[1] == 96)  # 6 of 2^4 is nearest to both
    assert np.isnan(got[2:]).all()
