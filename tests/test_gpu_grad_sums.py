"""The norm's stated error, where its roundings add up instead of cancelling: equal
values in every place."""
import math

import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu

# of the exact norm: half of the roundings in a vector's sum of squares (fp32: the first
# product and three sums; bf16, whose squares are exact: seven sums), and the last one
BOUND = {torch.float32: 3 * 2.0 ** -24, torch.bfloat16: 4.5 * 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("values", [[0.1], [1 / 3], [0.7], [1e-3, 0.33], [0.99609375, 0.0123, 0.3, 0.77, 0.5, 0.21, 1.7, 0.9]])
@pytest.mark.parametrize("count", [8, 16384, 1000007])
def test_norm_of_repeated_values(values, dtype, count):
    t = torch.tensor(values, device="cuda").to(dtype).repeat(-(-count // len(values)))[:count].contiguous()
    norm = torch.empty(1, device="cuda")
    B.grad_norm([t], norm, B.alloc_grad_workspace(1))
    exact = math.sqrt(float(t.double().square().sum()))
    assert abs(float(norm) - exact) <= BOUND[dtype] * exact
