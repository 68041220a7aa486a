"""Calls of moe_forward_few that the batches of its other tests do not make."""
import os
import subprocess
import sys
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


@pytest.mark.parametrize("process", range(2))
def test_threads_with_layers_of_different_sizes(process):
    """A layer with more experts takes more shared memory, whatever another thread's
    layer takes at that moment.  In processes of their own, whose first launches these
    are: they take long, so that the threads' calls overlap (a limit on shared memory
    that each call sets for itself refused one or more of them in two of three runs)."""
    here = os.path.dirname(os.path.abspath(__file__))
    child = subprocess.run([sys.executable, "-c", "import test_gpu_few_calls as t; t.first_calls_of_threads()"],
                           cwd=here, env={**os.environ, "PYTHONPATH": os.path.dirname(here)}, timeout=120,
                           capture_output=True, text=True)
    assert child.returncode == 0, child.stdout + child.stderr


def first_calls_of_threads():
    layers = [Layer(E) for E in (32,) * 4 + (1024,) * 4]
    torch.cuda.synchronize()
    start = threading.Barrier(len(layers))

    def calls(layer):
        start.wait()
        for _ in range(100):
            layer.run(layer.stream)
        layer.stream.synchronize()

    errors = run_threads(*[lambda layer=layer: calls(layer) for layer in layers])
    assert not errors, errors
    for i in (0, 4):  # equal layers, equal results
        assert all(torch.equal(layer.y, layers[i].y) for layer in layers[i:i + 4])
