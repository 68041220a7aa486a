"""moe_forward_few against the fp64 oracle: every weight type, both routings,
batches of 1 to 16 tokens, forced and skewed routings, odd layer shapes.

Error of an output, relative to the sum of the magnitudes it is made of: each of
the three products sums its contraction in fp32, split over at least 8 warps in
chains of MMAs of 16 steps, each adding at most 2^-23; h, the weights and the
joins add a few steps more.  With d and I the contractions (in units of 128):
  tol = (2 d/128 + I/128 + 24) 2^-23
taken on the 2-norm (the magnitudes' sum exceeds the norm of a product of
independent terms by about the square root of its length, which the single
steps, of either sign, give back); bf16 outputs add half a step, 2^-8."""
import dataclasses

import numpy as np
import pytest
import torch

import mx_ref
import oracle
from mixture_experts_ffn_17_b200 import binding as B
from mixture_experts_ffn_17_b200 import build as libbuild
from mixture_experts_ffn_17_b200 import workloads

from gpu_util import oracle_full, run_forward, to_device
from parity import compare_indices, dec, oracle_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()
    oracle.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@dataclasses.dataclass
class Case:
    """A workload with the weights as the call takes them, and as fp64 reads them."""
    w: workloads.Workload      # on the device; W1, W3, W2 (and scales) of the call
    ref: workloads.Workload    # bf16 or e4m3 weights of the same values, for the oracle
    dtype: int


def make(kind, seed=None, **kw):
    name = "fp8" if kind == "e4m3" else "prefill"
    cfg = workloads.CONFIGS[name].replace(w_std=0.02, **kw)
    if seed is not None:
        cfg = cfg.replace(seed=seed)
    w = to_device(workloads.make(cfg))
    if kind != "mxfp4":
        return Case(w, w, B.MOE_E4M3 if kind == "e4m3" else B.MOE_BF16)
    packed, plain = {}, {}
    for m in ("W1", "W3", "W2"):
        W = getattr(w, m)
        E, K, N = W.shape
        codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
        B.mx_quantise_weights(W, codes, scales)
        packed[m], packed["s" + m[1]] = codes, scales
        v = mx_ref.values(codes.cpu().numpy(), scales.cpu().numpy()).transpose(0, 2, 1)
        plain[m] = torch.as_tensor(np.ascontiguousarray(v)).to(torch.bfloat16)  # exact: 2 significant bits
        assert np.array_equal(plain[m].double().numpy(), v)
    return Case(dataclasses.replace(w, **packed), dataclasses.replace(w, **plain), B.MOE_MXFP4)


def shape_of(case, y_dtype=B.MOE_F32):
    s = B.shape_of(case.w.cfg, y_dtype)
    s.w_dtype = case.dtype
    return s


def run(case, y_dtype=B.MOE_F32, ws=None, stream=None):
    cfg, w = case.w.cfg, case.w
    shape = shape_of(case, y_dtype)
    ws = B.alloc_few_workspace(shape) if ws is None else ws
    ws.fill_(0xA5)  # nothing may depend on what a workspace held
    y = torch.full((cfg.T, cfg.d), 7.0, dtype=torch.float32 if y_dtype == B.MOE_F32 else torch.bfloat16, device="cuda")
    idx = torch.full((cfg.T, cfg.k), -1, dtype=torch.int32, device="cuda")
    tw = torch.full((cfg.T, cfg.k), -1.0, device="cuda")
    counts = torch.full((cfg.E,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    B.forward_few(shape, w.x, w.Wg, w.bias, w.W1, w.W3, w.W2, w.s1, w.s3, w.s2, w.W1s, w.W3s, w.W2s, y, ws, idx, tw,
                  counts, stream=stream)
    rc, raw = B.check_device_status(ws, stream)
    assert rc == B.MOE_OK, (rc, raw)
    return y, idx, tw, counts


def tolerance(cfg):
    wide = max(cfg.inter, cfg.shared_inter)
    return (2 * cfg.d / 128 + wide / 128 + 24) * 2.0 ** -23


def check(case, y_dtype=B.MOE_F32):
    cfg = case.w.cfg
    y, idx, tw, counts = run(case, y_dtype)
    bias = None if case.w.bias is None else dec(case.w.bias)
    lg = oracle.logits(dec(case.w.x), dec(case.w.Wg))
    idx_o, w_o, scores, gaps, ggap = oracle_route(cfg, lg, bias)
    idx_d = idx.cpu().numpy()
    group = (cfg.n_group, cfg.topk_group, cfg.group_topn) if cfg.route == 1 else None
    compare_indices(idx_d, idx_o, scores, gaps, ggap, cfg.E, group=group)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(idx_d.ravel(), minlength=cfg.E))
    w_o = oracle.weights_for(lg, idx_d, cfg.route, cfg.route_scale)
    # a logit of size up to 8 is off by 2^-22 after its rounding, and so, relatively, is its exponential
    assert np.all(np.abs(tw.cpu().numpy() - w_o) <= 2.0 ** -20 * w_o)
    y_o = oracle_full(case.ref, force_idx=idx_d)[0]
    err = y.double().cpu().numpy() - y_o
    tol = tolerance(cfg) + 2.0 ** -20
    if y_dtype == B.MOE_F32:
        assert np.linalg.norm(err) <= tol * np.linalg.norm(y_o), np.linalg.norm(err) / np.linalg.norm(y_o)
    rms = np.sqrt(np.mean(y_o ** 2))
    step = 2.0 ** -8 if y_dtype == B.MOE_BF16 else 0.0
    assert np.all(np.abs(err) <= step * np.abs(y_o) + 8 * tol * rms), np.abs(err).max() / rms
    return y


GROUP = dict(route=1, n_group=8, topk_group=4, group_topn=2, route_scale=2.5, bias_std=0.01)
PLAIN = dict(route=0, bias_std=0.0)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 11, 16])
def test_batches(kind, T):
    check(make(kind, T=T, d=512, E=32, k=4, inter=256, shared_inter=256, **(GROUP if kind == "e4m3" else PLAIN)))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
@pytest.mark.parametrize("shape", [
    dict(T=1, d=128, E=32, k=1, inter=128, shared_inter=0),
    dict(T=16, d=128, E=32, k=32, inter=128, shared_inter=128),     # every expert for every token
    dict(T=7, d=1152, E=96, k=6, inter=640, shared_inter=384),      # odd numbers of 128-column blocks
    dict(T=4, d=2048, E=64, k=8, inter=128, shared_inter=1024),     # shared wider than the routed experts
    dict(T=16, d=640, E=1024, k=2, inter=256, shared_inter=0),
    dict(T=9, d=384, E=32, k=8, inter=1408, shared_inter=128),
])
def test_layer_shapes(kind, shape):
    check(make(kind, **shape, **PLAIN))


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 13])
def test_group_routing(kind, T):
    check(make(kind, T=T, d=512, E=64, k=6, inter=256, shared_inter=128, **GROUP))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
def test_bf16_output(kind):
    check(make(kind, T=6, d=512, E=32, k=4, inter=256, shared_inter=256, **PLAIN), B.MOE_BF16)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mxfp4"])
def test_all_tokens_on_the_same_experts(kind):
    c = make(kind, T=16, d=512, E=32, k=4, inter=384, shared_inter=0, **PLAIN)
    c.w.x[1:] = c.w.x[0]
    c.ref.x[1:] = c.w.x[0]
    y = check(c)
    assert torch.equal(y, y[:1].expand_as(y))


def test_equal_scores_take_the_lowest_index():
    c = make("bf16", T=3, d=256, E=64, k=5, inter=128, shared_inter=0, **PLAIN)
    c.w.Wg[:] = 0
    c.w.Wg[40] = c.w.x[0].to(c.w.Wg.dtype)
    _, idx, tw, _ = run(c)
    assert idx[0].tolist() == [40, 0, 1, 2, 3]
    c.w.Wg[:] = 0
    _, idx, tw, _ = run(c)
    assert idx.tolist() == [[0, 1, 2, 3, 4]] * 3
    assert torch.allclose(tw, torch.full_like(tw, 0.2), rtol=2 ** -22, atol=0)


def test_large_and_small_magnitudes():
    # h runs over many binades: its three bf16 terms follow it
    c = make("bf16", T=4, d=256, E=32, k=2, inter=128, shared_inter=128, **PLAIN)
    for W in (c.w.W1, c.w.W3, c.w.W1s, c.w.W3s):
        W *= torch.exp2(torch.linspace(-20, 3, W.shape[-1], device="cuda")).to(W.dtype)
    check(c)


def test_a_nan_token_stays_alone():
    c = make("mxfp4", T=5, d=256, E=32, k=4, inter=128, shared_inter=128, **PLAIN)
    y0 = run(c)[0]
    c.w.x[2, 17] = float("nan")
    y1, idx, _, _ = run(c)
    keep = [0, 1, 3, 4]
    assert torch.equal(y0[keep], y1[keep]) and torch.isnan(y1[2]).all()
    assert int(idx.min()) >= 0 and int(idx.max()) < 32


def test_nan_codes_and_scales_show():
    c = make("e4m3", T=1, d=256, E=32, k=32, inter=128, shared_inter=0, **PLAIN)
    c.w.W2[3, 5, 77] = 0x7F
    y = run(c)[0]
    assert torch.isnan(y[0, 77]) and not torch.isnan(y[0, :77]).any() and not torch.isnan(y[0, 78:]).any()
    c = make("mxfp4", T=1, d=256, E=32, k=32, inter=128, shared_inter=0, **PLAIN)
    c.w.s2[3, 77, 2] = 255
    y = run(c)[0]
    assert torch.isnan(y[0, 77]) and not torch.isnan(y[0, :77]).any() and not torch.isnan(y[0, 78:]).any()


def test_scales_over_one_and_tiny_scales():
    # scale bytes over 128 leave bf16's range in one multiplication
    c = make("mxfp4", T=2, d=256, E=32, k=3, inter=256, shared_inter=0, **PLAIN)
    for name in ("s1", "s3", "s2"):
        s = getattr(c.w, name)
        s += torch.randint(-20, 16, s.shape, generator=torch.Generator().manual_seed(1)).to(torch.uint8).cuda()
    c.w.x *= 2.0 ** -6
    for m in ("W1", "W3", "W2"):
        v = mx_ref.values(getattr(c.w, m).cpu().numpy(), getattr(c.w, "s" + m[1]).cpu().numpy())
        setattr(c.ref, m, torch.as_tensor(np.ascontiguousarray(v.transpose(0, 2, 1))).to(torch.bfloat16))
    assert int(c.w.s1.max()) > 130
    c.ref.x = c.w.x
    check(c)


def test_agrees_with_the_whole_batch_call():
    c = make("bf16", T=12, d=512, E=32, k=4, inter=256, shared_inter=256, **PLAIN)
    y, idx, tw, counts = run(c)
    y2, idx2, tw2, counts2, _ = run_forward(c.w)
    assert torch.equal(idx, idx2) and torch.equal(counts, counts2)
    # moe_forward rounds h and each expert's output to bf16
    assert float((y - y2).norm() / y2.norm()) < 2.0 ** -7


def test_no_tokens():
    s = B.make_shape(T=0, d=256, E=32, k=2, inter=128, shared_inter=128)
    e = lambda *sz: torch.empty(*sz, dtype=torch.bfloat16, device="cuda")
    W1, W2, W1s = e(32, 256, 128), e(32, 128, 256), e(256, 128)
    y = torch.empty(16, 256, device="cuda")
    B.forward_few(s, W1, e(32, 256), None, W1, W1, W2, None, None, None, W1s, W1s, W1s, y, B.alloc_few_workspace(s))


def test_same_bits_every_time():
    c = make("e4m3", T=9, d=1024, E=64, k=6, inter=512, shared_inter=256, **GROUP)
    a, b = run(c), run(c)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_graph_replays_follow_the_input():
    c = make("mxfp4", T=6, d=512, E=64, k=4, inter=256, shared_inter=256, **PLAIN)
    cfg, w, shape = c.w.cfg, c.w, shape_of(c)
    ws, y = B.alloc_few_workspace(shape), torch.empty(cfg.T, cfg.d, device="cuda")
    x = w.x.clone()
    call = lambda x, y: B.forward_few(shape, x, w.Wg, w.bias, w.W1, w.W3, w.W2, w.s1, w.s3, w.s2, w.W1s, w.W3s, w.W2s,
                                      y, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(x, y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(x, y)
    for rep in range(3):
        x.copy_(w.x.roll(rep + 1, 0) * (1.0 + 0.25 * rep))
        g.replay()
        torch.cuda.synchronize()
        got, eager = y.clone(), torch.empty_like(y)
        call(x, eager)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
    del g


def test_two_streams_with_workspaces_of_their_own():
    cs = [make("bf16", T=5, d=1024, E=32, k=4, inter=512, shared_inter=256, **PLAIN),
          make("mxfp4", T=16, d=512, E=64, k=4, inter=256, shared_inter=128, **PLAIN)]
    want = [run(c)[0] for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [B.alloc_few_workspace(shape_of(c)) for c in cs]
    ys = [torch.empty_like(y) for y in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, st, ws, y in zip(cs, streams, wss, ys):
            w = c.w
            B.forward_few(shape_of(c), w.x, w.Wg, w.bias, w.W1, w.W3, w.W2, w.s1, w.s3, w.s2, w.W1s, w.W3s, w.W2s, y,
                          ws, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, ys))


def test_long_sums_keep_their_bits():
    """The tensor core cuts off (2^-24 of its accumulator on average) at every MMA.
    Four MMAs of a tile, whose sum is 1/sqrt(d/64) of the whole, cut 4 2^-24 of it in
    norm over all d/64 tiles: 2.4e-7 in each of g, u and the down product.  Adding the
    tiles up to nearest, h and the joins add some 4 roundings of 2^-24 at random
    signs, 1.2e-7.  Together sqrt(3) (2.4e-7 + 1.2e-7) = 6.2e-7; cutting in one
    accumulator over 64 MMAs would cost about 64^(1/2) / 2 as much."""
    d, inter, E, k, T = 7168, 2048, 32, 2, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, Wg = r(T, d).bfloat16(), (r(E, d) * d ** -0.5).bfloat16()
    W = [(r(E, K, N) * K ** -0.5).bfloat16() for K, N in ((d, inter), (d, inter), (inter, d))]
    shape = B.make_shape(T, d, E, k, inter, 0, 0, 1, 1, 2, 1.0, B.MOE_BF16, B.MOE_F32)
    y, ws = torch.empty(T, d, device="cuda"), B.alloc_few_workspace(shape)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    B.forward_few(shape, x, Wg, None, *W, None, None, None, None, None, None, y, ws, idx, w)
    assert B.check_device_status(ws) == (0, 0)
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.where(idx == e)
        if len(t):
            v = x[t].double()
            h = torch.nn.functional.silu(v @ W[0][e].double()) * (v @ W[1][e].double())
            want.index_add_(0, t, w[t, j].double()[:, None] * (h @ W[2][e].double()))
    error = ((y.double() - want).norm() / want.norm()).item()
    assert error < 6.2e-7, error


GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


def coded(kind, E, K, N, generator):
    """Weights of a kind and their values [K, N] of expert e in fp64."""
    w = (torch.randn(E, K, N, generator=generator, device="cuda") * K ** -0.5).bfloat16()
    if kind == "e4m3":
        b = w.float().view(E, K // 128, 128, N // 128, 128)
        s = b.abs().amax((2, 4)) / 448
        q = (b / s[:, :, None, :, None]).to(torch.float8_e4m3fn).view(E, K, N)
        spread = lambda e: s[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return q.view(torch.uint8), s, lambda e: q[e].double() * spread(e)
    c = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N, K // 32, dtype=torch.uint8, device="cuda")
    B.mx_quantise_weights(w, c, s)
    grid = torch.tensor(GRID + [-v for v in GRID], dtype=torch.float64, device="cuda")

    def values(e):
        codes = torch.stack((c[e] & 15, c[e] >> 4), -1).flatten(1).long()
        return (grid[codes] * torch.exp2(s[e].double() - 127).repeat_interleave(32, 1)).t()
    return c, s, values


@pytest.mark.parametrize("kind", ["e4m3", "mxfp4"])
@pytest.mark.parametrize("T,k,inter,shared", [(16, 8, 2048, 0), (3, 8, 2048, 256), (16, 32, 256, 0)])
def test_many_chunks_of_codes(kind, T, k, inter, shared):
    """Dozens of chunks a CTA, of one to 32 stages: every ring turns many times.  Sums
    as in test_long_sums_keep_their_bits, 6.2e-7; the terms of x and of h are good
    to 2^-24 of the largest of a block, 4 times its rms, at random signs: 2.4e-7 /
    sqrt(3) each.  Together below 6.6e-7."""
    d, E = 7168, 32
    g = torch.Generator(device="cuda").manual_seed(T * inter)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, Wg = r(T, d).bfloat16(), (r(E, d) * d ** -0.5).bfloat16()
    W, S, values = zip(*(coded(kind, E, K, N, g) for K, N in ((d, inter), (d, inter), (inter, d))))
    own = [(r(K, N) * K ** -0.5).bfloat16() for K, N in ((d, shared), (d, shared), (shared, d))] if shared else [None] * 3
    dtype = B.MOE_E4M3 if kind == "e4m3" else B.MOE_MXFP4
    shape = B.make_shape(T, d, E, k, inter, shared, 0, 1, 1, 2, 1.0, dtype, B.MOE_F32)
    y, ws = torch.empty(T, d, device="cuda"), B.alloc_few_workspace(shape)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    B.forward_few(shape, x, Wg, None, *W, *S, *own, y, ws, idx, w)
    assert B.check_device_status(ws) == (0, 0)
    want = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    expert = lambda v, A, G, D: (torch.nn.functional.silu(v @ A) * (v @ G)) @ D
    for e in range(E):
        t, j = torch.where(idx == e)
        if len(t):
            want.index_add_(0, t, w[t, j].double()[:, None] * expert(x[t].double(), *(f(e) for f in values)))
    if shared:
        want += expert(x.double(), *(m.double() for m in own))
    error = ((y.double() - want).norm() / want.norm()).item()
    assert error < 6.6e-7, error
