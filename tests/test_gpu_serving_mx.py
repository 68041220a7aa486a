"""The MXFP4 operators together, as a serving program uses them: expert weights are
quantised once; a batch goes router, permutation, quantised rows, product, gated
quantisation, product, combine; and a few tokens go through moe_forward_few with
the same weights.  And a training step with its gradients clipped."""
import numpy as np
import pytest
import torch

import mx_ref
import oracle
from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild
from mixture_experts_ffn_17_b200 import workloads

from gpu_util import to_device
from parity import dec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    oracle.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def new(*shape, dtype=torch.uint8):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def quantised_weights(W):
    E, K, N = W.shape
    codes, scales = new(E, N, K // 2), new(E, N, K // 32)
    B.mx_quantise_weights(W, codes, scales)
    return codes, scales


def test_batch_through_quantised_experts():
    cfg = workloads.CONFIGS["prefill"].replace(T=100, d=512, E=32, k=4, inter=256, shared_inter=0, w_std=0.02)
    w = to_device(workloads.make(cfg))
    T, d, E, k, I = cfg.T, cfg.d, cfg.E, cfg.k, cfg.inter
    q1, q3, q2 = (quantised_weights(W) for W in (w.W1, w.W3, w.W2))
    shape = B.shape_of(cfg)
    ws, pws = B.alloc_workspace(shape), B.alloc_mx_product_workspace(T * k, E)
    idx, tw = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
    B.router_topk(shape, w.x, w.Wg, None, idx, tw, None, ws)
    counts, offsets = new(E, dtype=torch.int32), new(E + 1, dtype=torch.int32)
    perm, row_of, x_perm = new(T * k, dtype=torch.int32), new(T * k, dtype=torch.int32), new(T * k, d, dtype=torch.bfloat16)
    B.permute(shape, idx, counts, offsets, perm, row_of, w.x, x_perm, ws)

    R = T * k
    a, sa = new(R, d // 2), new(R, d // 32)
    B.mx_quantise(x_perm, a, sa)
    g, u = new(R, I, dtype=torch.float32), new(R, I, dtype=torch.float32)
    B.mx_grouped_product(a, sa, offsets, *q1, g, pws)
    B.mx_grouped_product(a, sa, offsets, *q3, u, pws)
    h, sh = new(R, I // 2), new(R, I // 32)
    B.mx_quantise(g, h, sh, up=u)
    o = new(R, d, dtype=torch.bfloat16)
    B.mx_grouped_product(h, sh, offsets, *q2, o, pws)
    y = new(T, d, dtype=torch.float32)
    B.combine(shape, o, None, row_of, tw, y)
    assert B.check_device_status(pws)[0] == B.MOE_OK

    # the same steps in fp64 from what each step was given: the codes of x and of
    # the weights, and the codes of h (whose rounding is tested on its own)
    val = lambda c, s: mx_ref.values(c.cpu().numpy(), s.cpu().numpy())
    A, H, off = val(a, sa), val(h, sh), offsets.cpu().numpy()
    gate = np.zeros((R, I))
    out = np.zeros((R, d))
    for e in range(E):
        s = slice(off[e], off[e + 1])
        ge, ue = A[s] @ val(q1[0][e], q1[1][e]).T, A[s] @ val(q3[0][e], q3[1][e]).T
        gate[s] = ge / (1 + np.exp(-ge)) * ue
        out[s] = H[s] @ val(q2[0][e], q2[1][e]).T
    # h's codes follow silu(g) * u: a quarter of a value at most, the grid's widest
    # half step (from 4 to 6 by 5, from below the smallest code to it by one half of
    # it), in its block's scale
    block = np.exp2(sh.cpu().numpy().astype(float) - 127).repeat(32, -1)
    assert np.all(np.abs(H - gate) <= np.maximum(0.25 * np.abs(gate), 0.25 * block) * (1 + 1e-5) + 2 * block * (np.abs(gate) > 6 * block))
    y_ref = np.zeros((T, d))
    np.add.at(y_ref, np.arange(R) // k, tw.cpu().numpy().reshape(-1, 1) * out[row_of.cpu().numpy()])
    err = np.abs(y.cpu().numpy() - y_ref)
    # one bf16 rounding of each expert's output (2^-8 of its weighted magnitude), then fp32 sums
    mag = np.zeros((T, d))
    np.add.at(mag, np.arange(R) // k, tw.cpu().numpy().reshape(-1, 1) * np.abs(out[row_of.cpu().numpy()]))
    assert np.all(err <= 2.0 ** -8 * mag + 1e-5 * np.abs(out).max())

    # a few of the tokens by moe_forward_few with the same weights: 16-bit
    # activations instead of 4-bit ones, so the two agree as far as 4 bits go
    few = cfg.replace(T=7)
    s7 = B.shape_of(few)
    s7.w_dtype = B.MOE_MXFP4
    y7, i7 = new(7, d, dtype=torch.float32), new(7, k, dtype=torch.int32)
    B.forward_few(s7, w.x[:7].contiguous(), w.Wg, None, q1[0], q3[0], q2[0], q1[1], q3[1], q2[1], None, None, None, y7,
                  B.alloc_few_workspace(s7), i7)
    assert torch.equal(i7, idx[:7])
    assert float((y7 - y[:7]).norm() / y7.norm()) < 0.5


@pytest.mark.parametrize("gdtype", [B.MOE_F32, B.MOE_BF16])
def test_training_step_with_clipped_gradients(gdtype):
    cfg = workloads.CONFIGS["prefill"].replace(T=64, d=256, E=32, k=4, inter=128, shared_inter=128, w_std=0.05)
    w = to_device(workloads.make(cfg))
    shape = B.shape_of(cfg, gdtype)
    dt = torch.float32 if gdtype == B.MOE_F32 else torch.bfloat16
    ws, gws = B.alloc_backward_workspace(shape), B.alloc_grad_workspace(8)
    y = new(cfg.T, cfg.d, dtype=dt)
    B.forward_train(shape, w.x, w.Wg, None, w.W1, w.W3, w.W2, w.W1s, w.W3s, w.W2s, y, ws)
    dx = new(cfg.T, cfg.d, dtype=dt)
    grads = [new(*t.shape, dtype=dt) for t in (w.Wg, w.W1, w.W3, w.W2, w.W1s, w.W3s, w.W2s)]
    dy = torch.randn(cfg.T, cfg.d, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    B.backward_saved(shape, w.x, w.Wg, w.W1, w.W3, w.W2, w.W1s, w.W3s, w.W2s, dy, dx, *grads, ws)
    before = [g.clone() for g in grads]
    norm = new(1, dtype=torch.float32)
    full = float(torch.stack([g.double().square().sum() for g in before]).sum().sqrt())
    B.grad_clip(grads, full / 4, norm, gws)
    torch.cuda.synchronize()
    assert abs(float(norm) - full) <= 1e-6 * full
    half = 2.0 ** -24 if dt == torch.float32 else 2.0 ** -8
    for a, b in zip(before, grads):
        want = a.double() / 4
        assert bool(((b.double() - want).abs() <= (half + 1e-6) * want.abs() + 2.0 ** -133).all())
    B.grad_norm(grads, norm, gws)
    assert abs(float(norm) - full / 4) <= (half + 1e-6) * full / 4
