"""The waits inside moe_forward_few and moe_mx_grouped_product: warps that come late,
and waits that run out.
Neither faults nor hangs: every wait is bounded, and debug switches of the library
hold a warp up or withhold loads."""
import time

import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

pytestmark = pytest.mark.gpu
# A wait's limit is 2 s.  A call that gives up waits twice: for what it was withheld,
# and for the copies that it may have under way; a second more for the host.
GIVEN_UP = 5.0


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Layer:
    """A layer of a kind of weights, its buffers and its call (codes and scales drawn as they are)."""

    def __init__(self, kind, T, d=1024, E=32, k=8, inter=512, shared=256):
        g = torch.Generator(device="cuda").manual_seed(T + d)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        u8 = lambda *s, lo=0, hi=256: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)
        self.x, self.Wg = r(T, d).bfloat16(), (r(E, d) * d ** -0.5).bfloat16()
        matrices = ((d, inter), (d, inter), (inter, d))
        if kind == "bf16":
            W, S = [(r(E, K, N) * K ** -0.5).bfloat16() for K, N in matrices], [None] * 3
        elif kind == "e4m3":
            W = [(r(E, K, N) * 64).to(torch.float8_e4m3fn).view(torch.uint8) for K, N in matrices]
            S = [torch.rand(E, K // 128, N // 128, generator=g, device="cuda") * K ** -0.5 / 32 for K, N in matrices]
        else:
            W = [u8(E, N, K // 2) for K, N in matrices]
            S = [u8(E, N, K // 32, lo=120, hi=122) for K, N in matrices]
        own = [(r(K, N) * K ** -0.5).bfloat16() if shared else None
               for K, N in ((d, shared), (d, shared), (shared, d))]
        self.weights = (*W, *S, *own)
        dtype = {"bf16": B.MOE_BF16, "e4m3": B.MOE_E4M3, "mxfp4": B.MOE_MXFP4}[kind]
        self.shape = B.make_shape(T, d, E, k, inter, shared, w_dtype=dtype)
        self.ws = B.alloc_few_workspace(self.shape)

    def run(self, fill=7.0):
        """y, which held `fill`, and the call's status."""
        y = torch.full(self.x.shape, fill, device="cuda")
        B.forward_few(self.shape, self.x, self.Wg, None, *self.weights, y, self.ws)
        return y, B.check_device_status(self.ws)[0]


@pytest.mark.parametrize("T,d,inter,shared", [(3, 1024, 512, 256), (1, 7168, 256, 0), (16, 7168, 2048, 0)])
def test_late_factors_are_waited_for(monkeypatch, T, d, inter, shared):
    """e4m3: the warp that brings a pass's factors comes a pass late.  The ring has to
    hold, and the sums to be the same."""
    layer = Layer("e4m3", T, d=d, inter=inter, shared=shared)
    want, rc = layer.run()
    assert rc == B.MOE_OK and torch.isfinite(want).all()
    monkeypatch.setenv("MOE_DEBUG_LATE_FACTORS", "1")
    got, rc = layer.run()
    assert rc == B.MOE_OK
    assert torch.equal(got, want)


@pytest.mark.parametrize("shared", [0, 256])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("withheld", ["1", "2"])
def test_waits_run_out_and_the_next_call_is_right(monkeypatch, kind, shared, withheld):
    """Tiles that never come, all of them or one CTA's of the down products: the call
    ends by itself with the status and leaves y as it was, and the next one, in the same
    workspace, is right."""
    layer = Layer(kind, 3, inter=1024, shared=shared)
    want, rc = layer.run()
    assert rc == B.MOE_OK and torch.isfinite(want).all()
    monkeypatch.setenv("MOE_DEBUG_WITHHOLD_LOADS", withheld)
    t0 = time.monotonic()
    y, rc = layer.run(fill=7.0)
    assert rc == B.MOE_ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < GIVEN_UP
    assert torch.all(y == 7.0)
    monkeypatch.delenv("MOE_DEBUG_WITHHOLD_LOADS")
    got, rc = layer.run()
    assert rc == B.MOE_OK
    assert torch.equal(got, want)


def test_a_cta_that_gave_up_is_missed(monkeypatch):
    """One CTA's down products fail at their start and the others go on for a while, so
    that they are still waiting for it when it has given up.  They must not take its
    sums, which were never written, for an answer."""
    layer = Layer("mxfp4", 16, d=7168, E=64, inter=8192, shared=0)
    monkeypatch.setenv("MOE_DEBUG_WITHHOLD_LOADS", "2")
    y, rc = layer.run(fill=7.0)
    assert rc == B.MOE_ERR_DEVICE_TIMEOUT
    assert torch.all(y == 7.0)


@pytest.mark.parametrize("rows", [3, 700])
def test_a_product_without_operands_gives_up(monkeypatch, rows):
    E, K, N = 3, 2048, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    u8 = lambda *s, lo=0, hi=256: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)
    args = (u8(rows, K // 2), u8(rows, K // 32, lo=120, hi=128),
            torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda"),
            u8(E, N, K // 2), u8(E, N, K // 32, lo=120, hi=128))
    ws = B.alloc_mx_product_workspace(rows, E)

    def product():
        Y = torch.full((rows, N), 7.0, device="cuda")
        B.mx_grouped_product(*args, Y, ws)
        return Y, B.check_device_status(ws)[0]

    want, rc = product()
    assert rc == B.MOE_OK
    monkeypatch.setenv("MOE_DEBUG_WITHHOLD_LOADS", "1")
    t0 = time.monotonic()
    Y, rc = product()
    assert rc == B.MOE_ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < GIVEN_UP
    assert torch.all(Y == 7.0)
    monkeypatch.delenv("MOE_DEBUG_WITHHOLD_LOADS")
    got, rc = product()
    assert rc == B.MOE_OK and torch.equal(got, want)
