"""Tensors that do not fit a call are refused by the binding, before the library sees
their addresses; and a norm that would land among the gradients, by the library."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

T, D, E, K, I, S = 3, 256, 32, 4, 128, 384
BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def few_arguments(kind):
    """Tensors of forward_few on the CPU, which it refuses last of all."""
    z = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)
    a = dict(x=z(T, D), Wg=z(E, D), bias=z(E, dtype=F32))
    for name, rows, cols in (("1", D, I), ("3", D, I), ("2", I, D)):
        if kind == B.MOE_BF16:
            W, s = z(E, rows, cols), None
        elif kind == B.MOE_E4M3:
            W, s = z(E, rows, cols, dtype=torch.float8_e4m3fn), z(E, rows // 128, cols // 128, dtype=F32)
        else:
            W, s = z(E, cols, rows // 2, dtype=U8), z(E, cols, rows // 32, dtype=U8)
        a["W" + name], a["s" + name] = W, s
    a.update(W1s=z(D, S), W3s=z(D, S), W2s=z(S, D), y=z(T, D, dtype=F32), topk_idx=z(T, K, dtype=I32),
             topk_w=z(T, K, dtype=F32), counts=z(E, dtype=I32), ws=z(1 << 20, dtype=U8))
    return a


def few(kind, y_dtype=B.MOE_F32, shape=None, **change):
    a = {**few_arguments(kind), **change}
    sh = dict(T=T, d=D, E=E, k=K, inter=I, shared_inter=S, route=1, n_group=8, topk_group=4, w_dtype=kind,
              y_dtype=y_dtype)
    B.forward_few(B.make_shape(**{**sh, **(shape or {})}), **a)


KINDS = [B.MOE_BF16, B.MOE_E4M3, B.MOE_MXFP4]


@pytest.mark.parametrize("kind", KINDS)
def test_few_takes_what_fits(kind):
    with pytest.raises(ValueError, match="CUDA"):  # all that is left to refuse
        few(kind)
    with pytest.raises(ValueError, match="CUDA"):  # more room than needed
        few(kind, y=torch.zeros(16, D), ws=torch.zeros(1 << 21, dtype=U8))
    with pytest.raises(ValueError, match="CUDA"):  # what is not needed is not looked at
        few(kind, shape=dict(shared_inter=0, route=0), bias=torch.zeros(1), W1s=None, W3s=torch.zeros(1), W2s=None,
            topk_idx=None, topk_w=None, counts=None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", "x Wg bias W1 W3 W2 s1 s3 s2 W1s W3s W2s y topk_idx topk_w counts".split())
def test_few_refuses_short_tensors_and_wrong_types(kind, name):
    t = few_arguments(kind)[name]
    if t is None:
        return
    with pytest.raises(ValueError, match=f"^{name} has"):
        few(kind, **{name: t.flatten()[:-1]})
    with pytest.raises(ValueError, match=f"^{name} has"):
        few(kind, **{name: t.to(torch.float64)})


def test_few_refuses_another_kinds_weights():
    for kind in KINDS:
        for other in KINDS:
            if kind != other:
                a = few_arguments(other)
                with pytest.raises(ValueError, match=" has "):
                    few(kind, **{n: a[n] for n in ("W1", "W3", "W2", "s1", "s3", "s2") if a[n] is not None})
    with pytest.raises(ValueError, match="^y has"):
        few(B.MOE_BF16, y_dtype=B.MOE_BF16)
    with pytest.raises(ValueError, match="^y has"):
        few(B.MOE_BF16, y=torch.zeros(T, D, dtype=BF16))


@pytest.mark.parametrize("bad", [torch.zeros(0), torch.zeros(1, dtype=BF16), torch.zeros(1, dtype=torch.float64)])
def test_norm_needs_room_for_an_fp32_number(bad):
    ws = torch.zeros(1 << 16, dtype=U8)
    with pytest.raises(ValueError, match="^norm has"):
        B.grad_norm([torch.zeros(4)], bad, ws)
    with pytest.raises(ValueError, match="^norm has"):
        B.grad_clip([torch.zeros(4)], 1.0, bad, ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.grad_clip([torch.zeros(4)], 1.0, None, ws)


def test_clip_refuses_a_norm_among_the_tensors():
    buf = ctypes.create_string_buffer((1 << 16) + 256)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 256
    size = B.lib().moe_grad_workspace_size(1)

    def clip(norm, data=p, out=None):
        arr = (B.MoeTensor * 1)()
        arr[0] = (data, out, 16, B.MOE_F32)
        return B.lib().moe_grad_clip(arr, 1, 1.0, norm, p + 8192, size - 1, None)

    for norm, out in ((p, None), (p + 60, None), (p + 4, p + 4096), (p + 4096 + 60, p + 4096)):
        assert clip(norm, out=out) == B.MOE_ERR_INVALID_ARG
    # beside them: the workspace that is a byte short is what is left to refuse
    for norm, out in ((p + 64, None), (p + 4096 + 64, p + 4096), (None, None)):
        assert clip(norm, out=out) == B.MOE_ERR_WORKSPACE
