"""Calls of moe_forward_few that the batches of its other tests do not make."""
import threading

import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Layer:
    """bf16 experts, one token."""

    def __init__(self, E, d=128, inter=128):
        g = torch.Generator(device="cuda").manual_seed(E)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
        self.x, self.Wg = r(1, d), r(E, d)
        self.W = (r(E, d, inter), r(E, d, inter), r(E, inter, d))
        self.shape = B.make_shape(1, d, E, 2, inter, 0)
        self.ws, self.stream = B.alloc_few_workspace(self.shape), torch.cuda.Stream()
        self.y = torch.empty(1, d, device="cuda")

    def run(self, stream=None):
        B.forward_few(self.shape, self.x, self.Wg, None, *self.W, *[None] * 6, self.y, self.ws, stream=stream)


def run_threads(*calls):
    """Runs each call in a thread of its own; their exceptions."""
    errors = []

    def guarded(call):
        try:
            call()
        except Exception as e:  # noqa: BLE001 -- handed to the test's thread
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(call,)) for call in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_a_threads_first_cuda_call():
    layer = Layer(32)
    layer.run()
    torch.cuda.synchronize()
    want = layer.y.clone()
    layer.y.zero_()
    torch.cuda.synchronize()
    assert not run_threads(lambda: layer.run(layer.stream))
    torch.cuda.synchronize()
    assert torch.equal(layer.y, want)
