"""Cases of four operators: the layer for a few tokens, MXFP4 quantisation, the grouped product of MXFP4
operands, and the clipping of a set of gradients by their global norm.

`run` computes them in plain torch, or with `own` set through the package's binding.

MXFP4 is the microscaled format of the OCP MX specification: blocks of 32 consecutive values share a power of two
2^(s - 127) held in one byte s, and every value is a 4-bit code (sign, two exponent bits, one mantissa bit) of
magnitude 0, 0.5, 1, 1.5, 2, 3, 4 or 6; two codes to a byte, the even index in the low half.
"""
import math

import torch

own = False

BLOCK = 32
F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)

# a layer of 256 experts of which 8 work for each token, as the decode and prefill workloads have it
WIDE = dict(d=7168, E=256, k=8, inter=2048, shared=2048)
TINY = dict(d=512, E=32, k=4, inter=256, shared=256)
PLAIN_ROUTE = dict(route=0, n_group=1, topk_group=1, group_topn=2, route_scale=1.0)
GROUP_ROUTE = dict(route=1, n_group=8, topk_group=4, group_topn=2, route_scale=2.5)


def listed():
    return [
        # one token through a small layer that stays in the L2 cache: the call's latency
        dict(name="few-tiny-1", op="few", T=1, **TINY, **PLAIN_ROUTE, weights="bf16", out="f32"),
        # one sequence being answered, bf16 experts: every chosen expert's weights once
        dict(name="few-bf16-1", op="few", T=1, **WIDE, **PLAIN_ROUTE, weights="bf16", out="bf16"),
        # the largest batch of the few-token form, about a hundred distinct experts
        dict(name="few-bf16-16", op="few", T=16, **WIDE, **PLAIN_ROUTE, weights="bf16", out="f32"),
        # four sequences, e4m3 experts with block scales and group-limited routing
        dict(name="few-e4m3-4", op="few", T=4, **WIDE, **GROUP_ROUTE, weights="e4m3", out="f32"),
        # an odd batch on MXFP4 experts
        dict(name="few-mxfp4-5", op="few", T=5, **WIDE, **GROUP_ROUTE, weights="mxfp4", out="bf16"),
        # a decode batch's hidden states on their way into MXFP4 experts
        dict(name="mx-rows-64", op="quantise", layout="rows", E=1, K=7168, N=64, src="bf16"),
        # loading time: one matrix of an expert-parallel rank's 32 experts, read back to see what the format leaves
        dict(name="mx-weights-32", op="quantise", layout="weights", E=32, K=7168, N=2048, src="bf16"),
        # the small layer's routed rows (128 tokens, 4 experts each)
        dict(name="product-tiny", op="product", rows=512, E=32, K=512, N=256, skew=0.0, out="bf16"),
        # a decode batch's routed rows (64 tokens, 8 experts each): one or two rows an expert, the weights' bytes
        dict(name="product-decode", op="product", rows=512, E=256, K=7168, N=2048, skew=0.0, out="bf16"),
        # a prefill batch's routed rows (4096 tokens) through the down projection, expert loads uneven
        dict(name="product-prefill", op="product", rows=32768, E=256, K=2048, N=7168, skew=0.5, out="bf16"),
        # every gradient of the small layer in fp32, above the bound
        dict(name="clip-tiny", op="clip", **TINY, experts=32, grads="f32", clips=True),
        # a rank's share of the wide layer's gradients: 32 experts' weights in bf16
        dict(name="clip-share", op="clip", **WIDE, experts=32, grads="bf16", clips=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "quantise", "product", "product", "clip"])
    if op == "few":
        E = 32 * rng.randint(1, 8)
        route = dict(GROUP_ROUTE) if rng.random() < 0.5 else dict(PLAIN_ROUTE)
        return dict(op="few", T=rng.randint(1, 16), d=128 * _log_uniform(rng, 2, 56), E=E, k=rng.randint(1, 8),
                    inter=128 * _log_uniform(rng, 1, 16), shared=128 * rng.randint(0, 16), **route,
                    weights=rng.choice(["bf16", "e4m3", "mxfp4"]), out=rng.choice(["f32", "bf16"]))
    if op == "quantise":
        if rng.random() < 0.5:
            return dict(op="quantise", layout="rows", E=1, K=BLOCK * _log_uniform(rng, 1, 224),
                        N=_log_uniform(rng, 1, 20000), src=rng.choice(["f32", "bf16"]))
        return dict(op="quantise", layout="weights", E=rng.randint(1, 16), K=BLOCK * _log_uniform(rng, 1, 224),
                    N=_log_uniform(rng, 1, 4096), src=rng.choice(["f32", "bf16"]))
    if op == "product":
        return dict(op="product", rows=_log_uniform(rng, 1, 16384), E=rng.randint(1, 128),
                    K=128 * _log_uniform(rng, 1, 56), N=128 * _log_uniform(rng, 1, 56),
                    skew=rng.choice([0.0, 0.5, 1.0]), out=rng.choice(["f32", "bf16"]))
    return dict(op="clip", d=128 * rng.randint(1, 32), E=32 * rng.randint(1, 8), k=4,
                inter=128 * _log_uniform(rng, 1, 8), shared=128 * rng.randint(0, 8), experts=rng.randint(1, 24),
                grads=rng.choice(["f32", "bf16"]), clips=rng.random() < 0.5)


def work(case):
    op = case["op"]
    if op == "few":
        T, d, E, k, I, S = (case[n] for n in ("T", "d", "E", "k", "inter", "shared"))
        touched = E * (1.0 - (1.0 - k / E) ** T)  # distinct experts, choices independent
        width = {"bf16": 2.0, "e4m3": 1.0 + 4.0 / 16384, "mxfp4": 0.5 + 1.0 / 32}[case["weights"]]
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": touched * 3 * d * I * width + 3 * d * S * 2 + E * d * 2 + T * d * (2 + size) + T * k * 8,
                "flops": 2.0 * T * (E * d + k * 3 * d * I + 3 * d * S)}
    if op == "quantise":
        n = case["E"] * case["K"] * case["N"]
        size = 4 if case["src"] == "f32" else 2
        return {"bytes": n * (size + 2 * (0.5 + 1.0 / 32) + size), "flops": 4.0 * n}
    if op == "product":
        R, E, K, N = (case[n] for n in ("rows", "E", "K", "N"))
        used = int((_segments(case)[1:] > _segments(case)[:-1]).sum())
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": R * K * (2 + 2 * (0.5 + 1.0 / 32)) + used * N * K * (0.5 + 1.0 / 32) + R * N * size,
                "flops": 2.0 * R * N * K}
    n = sum(math.prod(s) for s in _gradient_shapes(case)) * (4 if case["grads"] == "f32" else 2)
    return {"bytes": 2.0 * n, "flops": 3.0 * n}


# ---------------------------------------------------------------- inputs
def _generator(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(1000003 * (seed + 1) % (1 << 62))
    return g


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _hidden(g, T, d):
    z = _normal(g, T, d)
    return (z / z.square().mean(1, keepdim=True).sqrt()).to(BF16)


def _e4m3(w):
    """e4m3 codes of [n, rows, cols] with a scale amax / 448 for each block of 128 x 128."""
    n, r, c = w.shape
    b = w.view(n, r // 128, 128, c // 128, 128)
    scale = b.abs().amax(dim=(2, 4)) / 448.0
    q = (b / scale[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(n, r, c)
    return q.view(torch.uint8), scale


def _power(s):
    """2^(s - 127) of the scale bytes; the byte 255 stands for NaN."""
    s = s.to(torch.int32)
    p = torch.where(s == 0, 1 << 22, s << 23).to(torch.int32).view(F32)
    return torch.where(s == 255, torch.full_like(p, math.nan), p)


def _mxfp4(v):
    """(codes [..., K / 2], scale bytes [..., K / 32]) of fp32 values [..., K]: the block's scale is the power of two
    floor(log2(max)) - 2 (1 where all are zero), every value then the nearest code, ties to the even one, at most 6."""
    b = v.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    byte = (torch.frexp(top).exponent - 3 + 127).clamp(0, 254)
    byte = torch.where(top == 0, 127, byte)
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    byte = torch.where(bad, 255, byte).to(torch.int32)
    # dividing by the scale in two exact steps: the inverse of 2^-127 and of 2^127 are no normal numbers
    half = torch.where(bad, 127, byte) - 127
    a = b * _power((127 - half // 2)) * _power(127 - (half - half // 2))
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    code = code + (torch.signbit(b).to(torch.uint8) << 3)
    code = torch.where(bad, torch.zeros_like(code), code).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.squeeze(-1).to(torch.uint8)


def _values(codes, scales):
    """fp32 values that codes [..., K / 2] with scale bytes [..., K / 32] stand for."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, BLOCK)) * _power(scales)[..., None]).flatten(-2)


def _segments(case):
    """offsets [E + 1] of the experts' rows: loads as e^(skew z) for normal z, at skew 0 as chance has it."""
    g = torch.Generator().manual_seed(case["rows"] * 131 + case["E"])
    load = torch.exp(case["skew"] * torch.randn(case["E"], generator=g))
    who = torch.multinomial(load, case["rows"], replacement=True, generator=g)
    count = torch.bincount(who, minlength=case["E"])
    return torch.cat((torch.zeros(1, dtype=torch.int64), count.cumsum(0)))


def _gradient_shapes(case):
    d, E, I, S, n = (case[k] for k in ("d", "E", "inter", "shared", "experts"))
    shapes = [(E, d), (n, d, I), (n, d, I), (n, I, d)]
    return shapes + ([(d, S), (d, S), (S, d)] if S else [])


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": case}
    if op == "few":
        T, d, E, k, I, S = (case[n] for n in ("T", "d", "E", "k", "inter", "shared"))
        st["x"] = _hidden(g, T, d)
        st["Wg"] = _normal(g, E, d, std=d ** -0.5).to(BF16)
        st["bias"] = _normal(g, E, std=0.01) if case["route"] == 1 else None
        kind = case["weights"]
        for name, rows, cols in (("1", d, I), ("3", d, I), ("2", I, d)):
            shape = {"bf16": (E, rows, cols), "e4m3": (E, rows, cols), "mxfp4": (E, cols, rows // 2)}[kind]
            W = torch.empty(shape, dtype=BF16 if kind == "bf16" else torch.uint8, device="cuda")
            s = None
            if kind == "e4m3":
                s = torch.empty(E, rows // 128, cols // 128, device="cuda")
            elif kind == "mxfp4":
                s = torch.empty(E, cols, rows // BLOCK, dtype=torch.uint8, device="cuda")
            std = 0.5 * rows ** -0.5
            for e in range(0, E, 16):
                m = min(16, E - e)
                if kind == "bf16":
                    W[e:e + m] = _normal(g, m, rows, cols, std=std)
                elif kind == "e4m3":
                    W[e:e + m], s[e:e + m] = _e4m3(_normal(g, m, rows, cols, std=std))
                else:
                    W[e:e + m], s[e:e + m] = _mxfp4(_normal(g, m, cols, rows, std=std))
            st["W" + name], st["s" + name] = W, s
            st["W%ss" % name] = None
            if S:
                r, c = (S, cols) if name == "2" else (rows, S)
                st["W%ss" % name] = _normal(g, r, c, std=0.5 * r ** -0.5).to(BF16)
    elif op == "quantise":
        E, K, N = case["E"], case["K"], case["N"]
        shape = (N, K) if case["layout"] == "rows" else (E, K, N)
        std = 1.0 if case["layout"] == "rows" else 0.5 * K ** -0.5
        st["src"] = _normal(g, *shape, std=std).to(DTYPES[case["src"]])
    elif op == "product":
        E, K, N = case["E"], case["K"], case["N"]
        off = _segments(case)
        st["offsets"] = off.to(device="cuda", dtype=torch.int32)
        st["most"] = int((off[1:] - off[:-1]).max())
        st["x"] = _hidden(g, case["rows"], K)
        st["W"] = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        st["s"] = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device="cuda")
        for e in range(0, E, 16):
            m = min(16, E - e)
            st["W"][e:e + m], st["s"][e:e + m] = _mxfp4(_normal(g, m, N, K, std=0.5 * K ** -0.5))
    else:
        shapes = _gradient_shapes(case)
        st["grads"] = []
        for s in shapes:
            t = _normal(g, *s, std=1e-3).to(DTYPES[case["grads"]])
            if len(s) == 3 and s[0] > 2:
                t[s[0] // 2] = 0  # an expert that no token chose
            st["grads"].append(t)
        n = sum(t.numel() for t in st["grads"])
        st["max_norm"] = (0.5 if case["clips"] else 2.0) * 1e-3 * math.sqrt(n)
    if own:
        _keep(st)
    return st


def _keep(st):
    """The buffers and workspaces that a program keeps for its calls."""
    from mixture_experts_ffn_17_b200 import binding as B
    case, op, new = st["case"], st["case"]["op"], lambda *s, **kw: torch.empty(*s, device="cuda", **kw)
    u8 = torch.uint8
    if op == "few":
        T, d, k = case["T"], case["d"], case["k"]
        kind = {"bf16": B.MOE_BF16, "e4m3": B.MOE_E4M3, "mxfp4": B.MOE_MXFP4}[case["weights"]]
        st["shape"] = B.make_shape(T, d, case["E"], k, case["inter"], case["shared"], case["route"], case["n_group"],
                                   case["topk_group"], case["group_topn"], case["route_scale"], kind,
                                   B.MOE_F32 if case["out"] == "f32" else B.MOE_BF16)
        st["ws"] = B.alloc_few_workspace(st["shape"])
        st["y"] = new(T, d, dtype=DTYPES[case["out"]])
        st["idx"], st["w"] = new(T, k, dtype=torch.int32), new(T, k)
    elif op == "quantise":
        lead = () if case["layout"] == "rows" else (case["E"],)
        N, K = case["N"], case["K"]
        st["codes"], st["scales"] = new(*lead, N, K // 2, dtype=u8), new(*lead, N, K // BLOCK, dtype=u8)
        st["back"] = new(*lead, N, K, dtype=DTYPES[case["src"]])
    elif op == "product":
        R, K, N = case["rows"], case["K"], case["N"]
        st["codes"], st["scales"] = new(R, K // 2, dtype=u8), new(R, K // BLOCK, dtype=u8)
        st["Y"] = new(R, N, dtype=DTYPES[case["out"]])
        st["ws"] = B.alloc_mx_product_workspace(R, case["E"])
    else:
        st["to"] = [torch.empty_like(t) for t in st["grads"]]
        st["norm"] = new(1)
        st["ws"] = B.alloc_grad_workspace(len(st["grads"]))


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"few": _few, "quantise": _quantise, "product": _product, "clip": _clip}[case["op"]](st, case)


def _run_own(st, case):
    from mixture_experts_ffn_17_b200 import binding as B
    op = case["op"]
    if op == "few":
        B.forward_few(st["shape"], st["x"], st["Wg"], st["bias"], st["W1"], st["W3"], st["W2"], st["s1"], st["s3"],
                      st["s2"], st["W1s"], st["W3s"], st["W2s"], st["y"], st["ws"], st["idx"], st["w"])
        return {"y": st["y"], "idx": st["idx"], "w": st["w"]}
    if op == "quantise":
        if case["layout"] == "rows":
            B.mx_quantise(st["src"], st["codes"], st["scales"])
        else:
            B.mx_quantise_weights(st["src"], st["codes"], st["scales"])
        B.mx_dequantise(st["codes"], st["scales"], st["back"])
        return {"values": st["back"]}
    if op == "product":
        B.mx_quantise(st["x"], st["codes"], st["scales"])
        B.mx_grouped_product(st["codes"], st["scales"], st["offsets"], st["W"], st["s"], st["Y"], st["ws"])
        return {"Y": st["Y"]}
    B.grad_clip(st["grads"], st["max_norm"], st["norm"], st["ws"], out=st["to"])
    return {"norm": st["norm"], "grads": st["to"]}


def _choose(key, k):
    """The k largest of each row, in descending order, the lower index first where two are equal."""
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :k]


def _route(x, Wg, bias, case):
    """Indices and weights of the k experts of each token, from logits summed in 64 bits and rounded to 32."""
    logits = (x.double() @ Wg.double().T).float()
    k = case["k"]
    if case["route"] == 0:
        idx = _choose(logits, k)
        return idx, torch.softmax(logits.gather(1, idx), 1)
    s = torch.sigmoid(logits.double())
    sel = s + bias.double()
    groups = sel.unflatten(1, (case["n_group"], -1))
    best = groups.sort(dim=-1, descending=True).values[..., :case["group_topn"]].sum(-1)
    kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, _choose(best, case["topk_group"]), True)
    idx = _choose(torch.where(kept[..., None], groups, -math.inf).flatten(1), k)
    w = s.gather(1, idx)
    return idx, (case["route_scale"] * w / w.sum(1, keepdim=True)).float()


def _gathered(st, name, idx):
    """fp32 weights [len(idx), K, N] of the chosen experts."""
    W, s, kind = st["W" + name][idx], st["s" + name], st["case"]["weights"]
    if kind == "bf16":
        return W.float()
    if kind == "mxfp4":
        return _values(W, s[idx]).transpose(1, 2)
    w = W.view(torch.float8_e4m3fn).float()
    n, r, c = w.shape
    return (w.view(n, r // 128, 128, c // 128, 128) * s[idx][:, :, None, :, None]).view(n, r, c)


def _few(st, case):
    x = st["x"]
    idx, w = _route(x, st["Wg"], st["bias"], case)
    flat = idx.flatten()
    rows = x.float().repeat_interleave(case["k"], 0)[:, None, :]
    g = torch.bmm(rows, _gathered(st, "1", flat))
    u = torch.bmm(rows, _gathered(st, "3", flat))
    o = torch.bmm(g * torch.sigmoid(g) * u, _gathered(st, "2", flat)).view(case["T"], case["k"], -1)
    y = (w[..., None] * o).sum(1)
    if case["shared"]:
        g, u = x.float() @ st["W1s"].float(), x.float() @ st["W3s"].float()
        y = y + (g * torch.sigmoid(g) * u) @ st["W2s"].float()
    return {"y": y.to(DTYPES[case["out"]]), "idx": idx.int(), "w": w}


def _quantise(st, case):
    v = st["src"].float()
    return {"values": _values(*_mxfp4(v if case["layout"] == "rows" else v.transpose(1, 2))).to(st["src"].dtype)}


def _product(st, case):
    a = _values(*_mxfp4(st["x"].float()))
    off = st["offsets"].long()
    # every expert's rows at the head of a block of its own, the rest of the block zero
    who = torch.bucketize(torch.arange(case["rows"], device="cuda"), off[1:], right=True)
    place = torch.arange(case["rows"], device="cuda") - off[who]
    blocks = torch.zeros(case["E"], st["most"], case["K"], device="cuda")
    blocks[who, place] = a
    out = torch.bmm(blocks, _values(st["W"], st["s"]).transpose(1, 2))
    return {"Y": out[who, place].to(DTYPES[case["out"]])}


def _clip(st, case):
    norm = torch.stack([t.double().square().sum() for t in st["grads"]]).sum().sqrt()
    factor = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(t.float() * factor).to(t.dtype) for t in st["grads"]]}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"few": _exact_few, "quantise": _exact_quantise, "product": _exact_product,
            "clip": _exact_clip}[case["op"]](st, case)


def _exact_values(codes, scales):
    """MXFP4 values in 64 bits from the code's fields: (-1)^s 2^(e - 1) (1 + m / 2), and m / 2 where e is 0."""
    c = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        q = ((codes >> (4 * half)) & 15).double()
        sign, q = torch.where(q >= 8, -1.0, 1.0), q % 8
        e, m = torch.floor(q / 2), q % 2
        c[..., half::2] = sign * torch.where(e > 0, torch.exp2(e - 1) * (1 + m / 2), m / 2)
    p = torch.exp2(scales.double() - 127)
    p[scales == 255] = math.nan
    return c * p.repeat_interleave(BLOCK, -1)


def _exact_weight(st, name, e):
    W, s, kind = st["W" + name][e], st["s" + name], st["case"]["weights"]
    if kind == "bf16":
        return W.double()
    if kind == "mxfp4":
        return _exact_values(W, s[e]).T
    return W.view(torch.float8_e4m3fn).double() * s[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def _exact_few(st, case):
    x = st["x"].double()
    logits = torch.einsum("td,ed->te", x, st["Wg"].double()).float().double().cpu()
    bias = st["bias"].double().cpu() if st["bias"] is not None else None
    idx, w = [], []
    for t in range(case["T"]):
        l = logits[t].tolist()
        if case["route"] == 0:
            pick = sorted(range(case["E"]), key=lambda e: (-l[e], e))[:case["k"]]
            part = [math.exp(l[e] - l[pick[0]]) for e in pick]
            scale = 1.0
        else:
            s = [1.0 / (1.0 + math.exp(-v)) for v in l]
            sel = [a + b for a, b in zip(s, bias.tolist())]
            size = case["E"] // case["n_group"]
            score = [sum(sorted(sel[i * size:(i + 1) * size], reverse=True)[:case["group_topn"]])
                     for i in range(case["n_group"])]
            kept = sorted(range(case["n_group"]), key=lambda i: (-score[i], i))[:case["topk_group"]]
            pick = sorted((e for e in range(case["E"]) if e // size in kept), key=lambda e: (-sel[e], e))[:case["k"]]
            part = [s[e] for e in pick]
            scale = case["route_scale"]
        idx.append(pick)
        w.append([scale * p / sum(part) for p in part])
    w = torch.tensor(w, dtype=torch.float64, device="cuda")
    y = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")

    def expert(rows, W1, W3, W2):
        g = rows @ W1
        return (g / (1 + torch.exp(-g)) * (rows @ W3)) @ W2

    for e in sorted({e for row in idx for e in row}):
        at = [(t, j) for t in range(case["T"]) for j in range(case["k"]) if idx[t][j] == e]
        t, j = [a[0] for a in at], [a[1] for a in at]
        y[t] += w[t, j][:, None] * expert(x[t], *(_exact_weight(st, n, e) for n in "132"))
    if case["shared"]:
        y += expert(x, *(st["W%ss" % n].double() for n in "132"))
    return {"y": y, "idx": torch.tensor(idx, dtype=torch.int32), "w": w}


def _exact_quantise(st, case):
    if case["layout"] == "rows":
        return {"values": _exact_rounded(st["src"])}
    return {"values": torch.stack([_exact_rounded(p.T) for p in st["src"]])}


def _exact_rounded(v):
    """Values [..., K] as MXFP4 leaves them, by the grid's spacing around each: half a step of the value's binade."""
    b = v.double().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -149))).clamp(min=-125) - 2)
    unit = torch.where(top == 0, 1.0, unit)
    a = b / unit
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp(-6, 6).mul(unit).flatten(-2)


def _exact_product(st, case):
    a = _exact_rounded(st["x"])
    off = st["offsets"].tolist()
    out = torch.empty(case["rows"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        if off[e + 1] > off[e]:
            out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _exact_values(st["W"][e], st["s"][e]).T
    return {"Y": out}


def _exact_clip(st, case):
    total = sum(float(p.double().pow(2).sum()) for t in st["grads"] for p in t.flatten().split(1 << 26))
    norm = math.sqrt(total)
    factor = min(1.0, st["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64),
            "grads": [t.double() * factor for t in st["grads"]]}
