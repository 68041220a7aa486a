"""Refusals of the few-token layer, the MXFP4 operators and the gradient calls:
host-side checks, before any CUDA call."""
import ctypes

import pytest
import torch

from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild

INVALID, UNSUPPORTED, WORKSPACE = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE
TINY = dict(T=4, d=256, E=32, k=2, inter=128, shared_inter=128)


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


@pytest.fixture(scope="module")
def p():
    """An aligned, non-null address for calls that must stop before a launch."""
    buf = ctypes.create_string_buffer((1 << 16) + 256)
    addr = ctypes.addressof(buf)
    yield addr + (-addr) % 256
    del buf


def test_tensor_struct_layout():
    assert ctypes.sizeof(B.MoeTensor) == 32
    assert [getattr(B.MoeTensor, f).offset for f, _ in B.MoeTensor._fields_] == [0, 8, 16, 24]


# ------------------------------------------------------------ few tokens
def few(p, shape=None, **change):
    s = B.make_shape(**{**TINY, **(shape or {})})
    names = "x Wg bias W1 W3 W2 s1 s3 s2 W1s W3s W2s y idx w counts ws".split()
    a = {n: p for n in names}
    a["bytes"] = B.few_workspace_size(s)
    a.update(change)
    return B.lib().moe_forward_few(ctypes.byref(s), *[a[n] for n in names], a["bytes"], None)


@pytest.mark.parametrize("name", "x Wg W1 W3 W2 W1s W3s W2s y".split())
def test_few_needs_its_pointers(p, name):
    assert few(p, **{name: None}) == INVALID
    assert few(p, **{name: p + 8}) == INVALID


@pytest.mark.parametrize("kind", [B.MOE_E4M3, B.MOE_MXFP4])
def test_few_needs_scales_with_coded_weights(p, kind):
    for name in ("s1", "s3", "s2"):
        assert few(p, dict(w_dtype=kind), **{name: None}) == INVALID


def test_few_workspace(p):
    n = B.few_workspace_size(B.make_shape(**TINY))
    assert n > 0
    assert few(p, bytes=n - 1) == WORKSPACE
    assert few(p, ws=None) == WORKSPACE
    assert few(p, ws=p + 16) == WORKSPACE


@pytest.mark.parametrize("bad,status", [
    (dict(T=17), UNSUPPORTED), (dict(T=-1), INVALID), (dict(d=200), UNSUPPORTED), (dict(E=48), UNSUPPORTED),
    (dict(k=33), INVALID), (dict(inter=0), INVALID), (dict(w_dtype=4), INVALID), (dict(w_dtype=2), INVALID),
    (dict(y_dtype=3), INVALID), (dict(route=1, n_group=3), INVALID),
    (dict(T=16, k=16, E=1024, d=1 << 20, inter=1 << 20), UNSUPPORTED),
    (dict(T=1, E=1024, inter=1 << 21), UNSUPPORTED),
])
def test_few_refuses_shapes(p, bad, status):
    assert few(p, bad, bytes=1 << 40) == status
    assert B.few_workspace_size(B.make_shape(**{**TINY, **bad})) == 0
    with pytest.raises(B.MoeError):
        B.alloc_few_workspace(B.make_shape(**{**TINY, **bad}), device="cpu")


def test_few_without_tokens_or_a_shared_expert(p):
    assert few(p, dict(T=0)) == B.MOE_OK
    assert few(p, dict(T=0, shared_inter=0), W1s=None, W3s=None, W2s=None) == B.MOE_OK
    assert B.lib().moe_forward_few(None, *[p] * 17, 1 << 30, None) == INVALID


def test_other_calls_still_refuse_mxfp4():
    assert B.workspace_size(B.make_shape(**TINY, w_dtype=B.MOE_MXFP4)) == 0
    assert B.backward_workspace_size(B.make_shape(**TINY, w_dtype=B.MOE_MXFP4)) == 0


# ------------------------------------------------------------ MXFP4
def test_quantise_refusals(p):
    q = B.lib().moe_mx_quantise
    ok = dict(src=p, up=None, dt=B.MOE_F32, rows=2, cols=64, ld=64, codes=p, scales=p)
    call = lambda **kw: q(*{**ok, **kw}.values(), None)
    for bad in (dict(src=None), dict(codes=None), dict(scales=None), dict(rows=-1), dict(cols=0), dict(ld=63),
                dict(dt=B.MOE_E4M3), dict(src=p + 2), dict(up=p + 2), dict(codes=p + 8), dict(scales=p + 1)):
        assert call(**bad) == INVALID, bad
    assert call(cols=48) == UNSUPPORTED
    assert call(rows=1 << 60) == UNSUPPORTED
    assert call(rows=0, src=None, codes=None, scales=None) == B.MOE_OK


def test_quantise_weights_refusals(p):
    q = B.lib().moe_mx_quantise_weights
    ok = dict(W=p, dt=B.MOE_BF16, E=1, K=64, N=3, codes=p, scales=p)
    call = lambda **kw: q(*{**ok, **kw}.values(), None)
    for bad in (dict(W=None), dict(codes=None), dict(scales=None), dict(E=-1), dict(K=0), dict(N=0), dict(dt=5),
                dict(W=p + 1), dict(codes=p + 4), dict(scales=p + 4)):
        assert call(**bad) == INVALID, bad
    assert call(K=40) == UNSUPPORTED
    assert call(E=65536) == UNSUPPORTED
    assert call(E=0, W=None) == B.MOE_OK


def test_dequantise_refusals(p):
    q = B.lib().moe_mx_dequantise
    ok = dict(codes=p, scales=p, rows=2, cols=64, dst=p, dt=B.MOE_F32)
    call = lambda **kw: q(*{**ok, **kw}.values(), None)
    for bad in (dict(codes=None), dict(scales=None), dict(dst=None), dict(rows=-1), dict(cols=0), dict(dt=1),
                dict(dst=p + 4)):
        assert call(**bad) == INVALID, bad
    assert call(cols=33) == UNSUPPORTED
    assert call(rows=0, codes=None) == B.MOE_OK


def test_product_refusals(p):
    q = B.lib().moe_mx_grouped_product
    n = B.lib().moe_mx_product_workspace_size(8, 2)
    assert n > 0
    ok = dict(rows=8, E=2, K=128, N=128, A=p, As=p, off=p, W=p, Ws=p, Y=p, dt=B.MOE_F32, ws=p, bytes=n)
    call = lambda **kw: q(*{**ok, **kw}.values(), None)
    for bad in (dict(A=None), dict(As=None), dict(off=None), dict(W=None), dict(Ws=None), dict(Y=None), dict(rows=-1),
                dict(E=0), dict(K=0), dict(N=0), dict(dt=B.MOE_MXFP4), dict(A=p + 8), dict(Y=p + 4), dict(off=p + 4)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(K=96), dict(N=64), dict(E=1025), dict(rows=1 << 31), dict(E=1024, N=1 << 22)):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=p + 128), dict(bytes=n - 1)):
        assert call(**bad) == WORKSPACE, bad
    assert B.lib().moe_mx_product_workspace_size(8, 1025) == 0
    assert B.lib().moe_mx_product_workspace_size(-1, 1) == 0


# ------------------------------------------------------------ gradients
def tensors(*rows):
    arr = (B.MoeTensor * max(1, len(rows)))()
    for i, r in enumerate(rows):
        arr[i] = r
    return arr


def clip(p, *rows, n=None, max_norm=1.0, norm=None, ws=True, size=None):
    size = B.lib().moe_grad_workspace_size(len(rows)) if size is None else size
    return B.lib().moe_grad_clip(tensors(*rows), len(rows) if n is None else n, max_norm, norm, p if ws else None, size,
                                 None)


def test_clip_refuses_tensors(p):
    f, h = B.MOE_F32, B.MOE_BF16
    for row in ((None, None, 4, f), (p + 2, None, 4, f), (p + 1, None, 4, h), (p, None, -1, f), (p, None, 4, 1),
                (p, p + 4098, 4, f)):
        assert clip(p, row) == INVALID, row
    assert clip(p, (p, None, 4, f), n=-1) == INVALID
    assert clip(p, (p, None, 1 << 41, f)) == UNSUPPORTED
    assert clip(p, (p, None, 4, f), max_norm=-1.0) == INVALID
    assert clip(p, (p, None, 4, f), max_norm=float("nan")) == INVALID
    assert clip(p, (p, None, 4, f), norm=p + 2) == INVALID
    assert clip(p, (p, None, 4, f), ws=False) == WORKSPACE
    assert clip(p, (p, None, 4, f), size=8) == WORKSPACE


def test_clip_refuses_overlaps(p):
    f, h = B.MOE_F32, B.MOE_BF16
    for rows in (((p, None, 16, f), (p, None, 16, f)),                   # the same tensor twice
                 ((p, None, 16, f), (p + 60, None, 16, f)),              # one element shared
                 ((p, p + 32, 16, f),),                                  # a shifted copy over itself
                 ((p, p + 4096, 16, f), (p + 4096, p + 8192, 16, f)),    # one's output is another's source
                 ((p, p + 4096, 16, f), (p + 64, p + 4098, 16, h)),      # two outputs overlap
                 ((p, p + 8192, 2048, f), (p + 64, None, 4, h))):        # written inside another's source
        assert clip(p, *rows) == INVALID, rows


def test_too_many_tensors(p):
    assert B.lib().moe_grad_workspace_size(1025) == 0
    assert B.lib().moe_grad_workspace_size(-1) == 0
    assert B.lib().moe_grad_workspace_size(0) > 0
    assert clip(p, n=1025, size=1 << 30) == UNSUPPORTED
    assert B.lib().moe_grad_norm(tensors(), 1025, p, p, 1 << 30, None) == UNSUPPORTED


def test_norm_refusals(p):
    q, arr = B.lib().moe_grad_norm, tensors((p, None, 4, B.MOE_F32))
    size = B.lib().moe_grad_workspace_size(1)
    assert q(arr, 1, None, p, size, None) == INVALID
    assert q(arr, 1, p + 2, p, size, None) == INVALID
    assert q(None, 1, p, p, size, None) == INVALID
    assert q(arr, 1, p, p + 8, size, None) == WORKSPACE


# ------------------------------------------------------------ binding
def test_binding_refusals():
    u8, z = torch.uint8, torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        B.mx_quantise(z(2, 64), z(2, 32, dtype=u8), z(2, 2, dtype=u8))
    with pytest.raises(ValueError, match="codes"):
        B.mx_quantise(z(2, 64), z(2, 31, dtype=u8), z(2, 2, dtype=u8))
    with pytest.raises(ValueError, match="scales"):
        B.mx_dequantise(z(2, 32, dtype=u8), z(2, 1, dtype=u8), z(2, 64))
    with pytest.raises(ValueError, match="fp32 or bf16"):
        B.mx_quantise(z(2, 64, dtype=torch.float16), z(2, 32, dtype=u8), z(2, 2, dtype=u8))
    with pytest.raises(ValueError, match="contiguous"):
        B.mx_quantise(z(64, 2).T, z(2, 32, dtype=u8), z(2, 2, dtype=u8))
    with pytest.raises(ValueError, match="evenly"):
        B.mx_quantise(z(1, 64).expand(2, 64), z(2, 32, dtype=u8), z(2, 2, dtype=u8))
    with pytest.raises(ValueError, match="up"):
        B.mx_quantise(z(2, 64), z(2, 32, dtype=u8), z(2, 2, dtype=u8), up=z(2, 65)[:, :64])
    with pytest.raises(ValueError, match="fit"):
        B.mx_grouped_product(z(4, 64, dtype=u8), z(4, 4, dtype=u8), z(2, dtype=torch.int32), z(1, 128, 32, dtype=u8),
                             z(1, 128, 2, dtype=u8), z(4, 128), z(256, dtype=u8))
    with pytest.raises(ValueError, match="outputs"):
        B.grad_clip([z(4)], 1.0, None, z(8), out=[])
    with pytest.raises(ValueError, match="type or shape"):
        B.grad_clip([z(4)], 1.0, None, z(8), out=[z(5)])
