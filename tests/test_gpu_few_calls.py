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


def small_layer(kind, T=4, d=256, E=32, k=4, inter=256, shared=128):
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, Wg = r(T, d).bfloat16(), (r(E, d) * d ** -0.5).bfloat16()
    W = [(r(E, K, N) * K ** -0.5).bfloat16() for K, N in ((d, inter), (d, inter), (inter, d))]
    own = [(r(K, N) * K ** -0.5).bfloat16() for K, N in ((d, shared), (d, shared), (shared, d))]
    # h with few bits: its lower terms are zero
    W[0][:, :, 0] = W[1][:, :, 0] = 0
    S = [None] * 3
    if kind == "e4m3":
        W = [w.to(torch.float8_e4m3fn) for w in W]
        S = [torch.ones(E, w.shape[1] // 128, w.shape[2] // 128, device="cuda") for w in W]
    return B.make_shape(T, d, E, k, inter, shared, w_dtype=B.MOE_BF16 if kind == "bf16" else B.MOE_E4M3), x, Wg, W, S, own


def run_layer(shape, x, Wg, W, S, own):
    y = torch.empty(x.shape, device="cuda")
    idx = torch.empty(shape.T, shape.k, dtype=torch.int32, device="cuda")
    w, ws = torch.empty(shape.T, shape.k, device="cuda"), B.alloc_few_workspace(shape)
    B.forward_few(shape, x, Wg, None, *W, *S, *own, y, ws, idx, w)
    assert B.check_device_status(ws)[0] == B.MOE_OK
    return y, idx, w


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("kind,matrix", [("bf16", 0), ("bf16", 1), ("bf16", 2), ("bf16", "own 0"), ("bf16", "own 2"),
                                         ("e4m3", "own 2")])
def test_infinite_weights(kind, matrix, value):
    """An infinity or NaN stands where fp64 arithmetic has it, and the rest keeps its bits."""
    layer = small_layer(kind)
    shape, x, Wg, W, S, own = layer
    before, idx, w = run_layer(*layer)
    e, at = int(idx[1, 0]), (3, 5)
    if isinstance(matrix, int):
        W[matrix][e][at] = value
    else:
        own[int(matrix[-1])][at] = value
    y, idx2, _ = run_layer(*layer)
    assert torch.equal(idx, idx2)
    want = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    expert = lambda v, A, G, D: ((v @ A) / (1 + torch.exp(-(v @ A))) * (v @ G)) @ D
    for i in range(shape.E):
        t, j = torch.where(idx == i)
        if len(t):
            want.index_add_(0, t, w[t, j].double()[:, None] * expert(x[t].double(), *(m[i].double() for m in W)))
    want += expert(x.double(), *(m.double() for m in own))
    odd = ~torch.isfinite(want)
    assert odd.any()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(y[odd].nan_to_num(0.5), want[odd].float().nan_to_num(0.5))
    assert torch.equal(y[~odd], before[~odd])


def test_h_whose_lower_terms_are_zero():
    """h of one, a sum of one term: an infinite weight beside it is an infinite output."""
    shape, x, Wg, W, S, own = small_layer("bf16", T=1, E=32, k=1, shared=128)
    for A, G, D in (W, own):
        A.zero_(), G.zero_()
        # g = 32 and u = 1/32, both exact: silu(32) = 32 in fp32, so h = 1
        A[..., 0, :], G[..., 0, :] = 32.0, 1.0 / 32
        D[..., 2, 9] = float("inf")
    x.zero_()
    x[:, 0] = 1.0
    y, _, _ = run_layer(shape, x, Wg, W, S, own)
    assert y[0, 9] == float("inf") and torch.isfinite(y[0, :9]).all() and torch.isfinite(y[0, 10:]).all()
