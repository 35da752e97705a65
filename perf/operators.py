"""The operators around the FP8 linear layer, as they are measured: the norm in front of it (as a tensor, as the codes
and scales its products read, and backward), the product of those codes for any number of rows, and the clipping of its
gradients by their global norm.

`run` computes each in its plain form (elementary torch operations in 32 bits, sums of squares in 64), or, where `own`
is true, by the framework's entry points.  `exact` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -96
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# The weight shapes [out, in] of one layer of the framework's layer sweep: qkv, o, gate + up, down.
LAYER = ((4096, 2048), (2048, 2048), (12288, 2048), (2048, 6144))


def listed():
    return [
        # decoding one sequence: the norm of one token, latency only
        {"name": "norm_token", "op": "norm", "kind": "layer", "T": 1, "C": 2048, "dtype": "bf16"},
        # a training micro-batch of the layer sweep (4 sequences of 4096 tokens)
        {"name": "norm_train", "op": "norm", "kind": "layer", "T": 16384, "C": 2048, "dtype": "bf16"},
        # a small decode batch in front of an FP8 linear layer: the codes, no tensor in between
        {"name": "norm_quant_rows", "op": "quant", "kind": "rms", "T": 7, "C": 2048, "dtype": "bf16", "dual": False},
        # the training step's form: codes for the forward product and, transposed, for the weight gradient
        {"name": "norm_quant_train", "op": "quant", "kind": "rms", "T": 16384, "C": 2048, "dtype": "bf16", "dual": True},
        # the backward pass of the same micro-batch
        {"name": "norm_backward_train", "op": "backward", "kind": "layer", "T": 16384, "C": 2048, "dtype": "bf16"},
        # a ragged batch of a model whose width is no power of two, in fp32
        {"name": "norm_backward_odd", "op": "backward", "kind": "layer", "T": 1027, "C": 1000, "dtype": "fp32"},
        # the gradients of a small test model: many short tensors, views of one flat bucket at odd offsets
        {"name": "clip_small", "op": "clip", "layers": 3, "div": 16, "dtype": "fp32", "flat": True, "max_norm": 1.0},
        # one layer's gradients in bf16, below the bound (no clipping that step)
        {"name": "clip_layer", "op": "clip", "layers": 1, "div": 1, "dtype": "bf16", "flat": False, "max_norm": 1e4},
        # the fp32 main gradients of eight layers of the sweep, clipped
        {"name": "clip_model", "op": "clip", "layers": 8, "div": 1, "dtype": "fp32", "flat": False, "max_norm": 1.0},
        # one token through the qkv projection
        {"name": "rows_token", "op": "rows", "M": 1, "N": 4096, "K": 2048, "out": "bf16"},
        # a decode batch through the gate + up projection
        {"name": "rows_batch", "op": "rows", "M": 37, "N": 12288, "K": 2048, "out": "bf16"},
        # a short ragged prompt through the down projection, fp32 out
        {"name": "rows_prompt", "op": "rows", "M": 200, "N": 2048, "K": 6144, "out": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "quant", "backward", "clip", "rows"))
    if op == "rows":
        return {"op": op, "M": _log(rng, 1, 256), "N": 128 * _log(rng, 4, 96), "K": 128 * _log(rng, 2, 48),
                "out": rng.choice(("bf16", "bf16", "fp32"))}
    if op == "clip":
        return {"op": op, "layers": rng.randint(1, 6), "div": rng.choice((1, 1, 2, 4, 8, 16)),
                "dtype": rng.choice(("fp32", "bf16")), "flat": rng.random() < 0.5, "max_norm": rng.choice((0.1, 1.0, 1e4))}
    case = {"op": op, "kind": rng.choice(("layer", "rms")), "dtype": rng.choice(("bf16", "bf16", "fp32"))}
    most = 16384 * 2048                                   # elements: the largest listed norm
    if op == "quant":
        case["dual"] = rng.random() < 0.5
        case["C"] = 128 * _log(rng, 1, 64)
        rows = min(16384, most // case["C"])
        case["T"] = 128 * _log(rng, 1, max(1, rows // 128)) if case["dual"] else _log(rng, 1, rows)
    else:
        case["C"] = _log(rng, 64, 8192)
        case["T"] = _log(rng, 1, min(16384, most // case["C"]))
    return case


def _heavy(shape, g):
    """Student-t with 3 degrees of freedom: the heavy tails of activations and their gradients."""
    z = torch.randn(shape, generator=g, device=DEV)
    chi = torch.zeros(shape, device=DEV)
    for _ in range(3):
        chi += torch.randn(shape, generator=g, device=DEV).square_()
    return z / (chi / 3).sqrt_()


def _grad_shapes(case):
    """The gradients of `layers` layers, each dimension divided by `div`: the weights, two norm weights, and a bias of
    odd length per layer."""
    d = case["div"]
    return [s for _ in range(case["layers"])
            for s in [(n // d, k // d) for n, k in LAYER] + [(2048 // d,), (2048 // d,), (2048 // d - 1,)]]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "rows":
        M, N, K = case["M"], case["N"], case["K"]
        # codes as the quantizers leave them: heavy-tailed activations, normal weights, scales of the groups' maxima
        x = _heavy((M, K), g).view(M, K // 128, 128)
        w = (torch.randn((N, K), generator=g, device=DEV) * 0.02).view(N // 128, 128, K // 128, 128)
        ax, aw = x.abs().amax(2), w.abs().amax((1, 3))
        A = (x * (E4M3_MAX / ax)[:, :, None]).view(M, K).to(torch.float8_e4m3fn).view(torch.uint8)
        B = (w * (E4M3_MAX / aw)[:, None, :, None]).view(N, K).to(torch.float8_e4m3fn).view(torch.uint8)
        return {"case": case, "A": A, "sA": (ax / E4M3_MAX).t().contiguous(), "B": B, "sB": aw / E4M3_MAX}
    dtype = DTYPES[case["dtype"]]
    if op == "clip":
        shapes = _grad_shapes(case)
        sizes = [math.prod(s) for s in shapes]
        if case["flat"]:                                  # one bucket, the tensors behind each other
            flat = (torch.randn(sum(sizes), generator=g, device=DEV) * 1e-3).to(dtype)
            grads = [v.view(s) for v, s in zip(flat.split(sizes), shapes)]
            outs = [v.view(s) for v, s in zip(torch.zeros_like(flat).split(sizes), shapes)]
        else:
            grads = [(torch.randn(s, generator=g, device=DEV) * 1e-3).to(dtype) for s in shapes]
            outs = [torch.zeros_like(t) for t in grads]
        return {"case": case, "grads": grads, "outs": outs}
    T, C = case["T"], case["C"]
    state = {"case": case, "x": (_heavy((T, C), g) + 0.25).to(dtype),
             "weight": (1 + 0.1 * torch.randn(C, generator=g, device=DEV)).to(dtype)}
    if case["kind"] == "layer":
        state["bias"] = (0.1 * torch.randn(C, generator=g, device=DEV)).to(dtype)
    if op == "backward":
        state["dy"] = (_heavy((T, C), g) * 1e-3).to(dtype)
        # what the forward pass keeps: each row's mean (layer norm only) and reciprocal deviation
        x = state["x"].double()
        mean = x.mean(1, keepdim=True) if case["kind"] == "layer" else torch.zeros((T, 1), dtype=x.dtype, device=DEV)
        state["mean"] = mean[:, 0].float() if case["kind"] == "layer" else None
        state["rstd"] = ((x - mean).square().mean(1) + EPS).rsqrt().float()
    return state


def _normed(state):
    """The plain norm in 32 bits: (y, mean, rstd)."""
    x = state["x"].float()
    layer = state["case"]["kind"] == "layer"
    mean = x.mean(1, keepdim=True) if layer else None
    d = x - mean if layer else x
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd * state["weight"].float()
    if layer:
        y = y + state["bias"].float()
    return y, mean[:, 0] if layer else None, rstd[:, 0]


def _coded(y):
    """Codes and scales of the groups of 128 along the last axis of y [R, K]: codes [R, K], scales [K/128, R]."""
    R, K = y.shape
    v = y.view(R, K // 128, 128)
    amax = v.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (v * (E4M3_MAX / amax)[:, :, None]).view(R, K).to(torch.float8_e4m3fn)
    return q, (amax / E4M3_MAX).t().contiguous()


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        y, mean, rstd = _normed(state)
        return y.to(state["x"].dtype), mean, rstd
    if op == "quant":
        y, mean, rstd = _normed(state)
        q, s = _coded(y)
        if not case["dual"]:
            return q, s
        qT, sT = _coded(y.t().contiguous())
        return q, s, qT, sT, mean, rstd
    if op == "backward":
        x, dy = state["x"].float(), state["dy"].float()
        layer = case["kind"] == "layer"
        rstd = state["rstd"][:, None]
        xh = (x - state["mean"][:, None]) * rstd if layer else x * rstd
        u = dy * state["weight"].float()
        t = u - xh * (u * xh).mean(1, keepdim=True)
        if layer:
            t = t - u.mean(1, keepdim=True)
        dx = (rstd * t).to(state["x"].dtype)
        return dx, (dy * xh).sum(0), dy.sum(0) if layer else None
    if op == "clip":
        squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in state["grads"]])
        norm = squares.sum().sqrt().float()
        coef = (case["max_norm"] / (norm + 1e-6)).clamp_max(1.0)
        outs = [o.copy_(g.float() * coef) for g, o in zip(state["grads"], state["outs"])]
        return norm, outs
    M, K = state["A"].shape
    N = state["B"].shape[0]
    A = state["A"].view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * state["sA"].t()[:, :, None]
    B = state["B"].view(torch.float8_e4m3fn).float().view(N // 128, 128, K // 128, 128) * state["sB"][:, None, :, None]
    return (A.view(M, K) @ B.view(N, K).t()).to(DTYPES[case["out"]])


def _run_own(state):
    import blockwise_scaled_fp8_quant_amd as P
    case = state["case"]
    op = case["op"]
    f8 = torch.float8_e4m3fn
    if op == "rows":
        return P.puro_gemm_rows(state["A"], state["sA"], state["B"], state["sB"],
                                out_dtype=P.OUT_BF16 if case["out"] == "bf16" else P.OUT_FP32)
    if op == "clip":
        return P.puro_clip_grad_norm(state["grads"], case["max_norm"], outs=state["outs"])
    kind = P.LAYER_NORM if case["kind"] == "layer" else P.RMS_NORM
    if op == "backward":
        return P.puro_layer_norm_backward(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"],
                                          kind=kind, with_bias=case["kind"] == "layer")
    x, weight, bias = state["x"], state["weight"], state.get("bias")
    if op == "norm":
        return P.puro_layer_norm(x, weight, bias, eps=EPS, kind=kind)
    if case["dual"]:
        q, s, qT, sT, mean, rstd = P.puro_layer_norm_quant_dual(x, weight, bias, eps=EPS, kind=kind)
        return q.view(f8), s, qT.view(f8), sT, mean, rstd
    q, s = P.puro_layer_norm_quant(x, weight, bias, eps=EPS, kind=kind)
    return q.view(f8), s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "rows":
        M, N, K = case["M"], case["N"], case["K"]
        eo = 2 if case["out"] == "bf16" else 4
        return {"bytes": M * K + N * K + M * N * eo + 4 * (M * K // 128 + N * K // 16384), "flops": 2 * M * N * K}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "clip":
        n = sum(math.prod(s) for s in _grad_shapes(case))
        return {"bytes": 2 * n * e, "flops": 3 * n}
    T, C = case["T"], case["C"]
    layer = case["kind"] == "layer"
    n, vec, stats = T * C, (2 if layer else 1) * C, (8 if layer else 4) * T
    if op == "norm":
        return {"bytes": 2 * n * e + vec * e + stats, "flops": 8 * n}
    if op == "backward":
        return {"bytes": 3 * n * e + C * e + vec * 4 + stats, "flops": 14 * n}
    ways = 2 if case["dual"] else 1
    return {"bytes": n * e + ways * (n + n // 32) + vec * e + (stats if case["dual"] else 0), "flops": (8 + 2 * ways) * n}


# ---- in 64 bits, from the definitions ---------------------------------------------------------------------------------

def _e4m3(v):
    """The E4M3 value nearest to v, ties to the even code, at most 448 in magnitude: 3 mantissa bits, smallest normal
    exponent -6."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))
    step = torch.ldexp(torch.ones_like(v), e - 1 - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_codes(y):
    groups = torch.stack(y.split(128, dim=1), dim=0)                       # [K/128, R, 128]
    scale = groups.abs().max(dim=2).values.clamp_min(AMAX_FLOOR) / E4M3_MAX
    return torch.cat(list(_e4m3(groups / scale[:, :, None])), dim=1), scale


def _exact_value(code):
    """What an E4M3 code byte stands for, by its bits."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, torch.ldexp(1 + m / 8, e - 7))
    return torch.where(c >= 128, -mag, mag)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        (M, K), N = state["A"].shape, state["B"].shape[0]
        sa, sb = state["sA"].double(), state["sB"].double()
        total = torch.zeros((M, N), dtype=torch.float64, device=DEV)
        for kb in range(K // 128):
            part = slice(128 * kb, 128 * kb + 128)
            product = _exact_value(state["A"][:, part]) @ _exact_value(state["B"][:, part]).t()
            total += product * sa[kb][:, None] * sb[:, kb].repeat_interleave(128)[None, :]
        return total
    if op == "clip":
        square = torch.zeros((), dtype=torch.float64, device=DEV)
        for g in state["grads"]:
            d = g.double().reshape(-1)
            square += torch.dot(d, d)
        norm = torch.sqrt(square)
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return norm, [g.double() * factor for g in state["grads"]]
    x, w = state["x"].double(), state["weight"].double()
    T, C = x.shape
    layer = case["kind"] == "layer"
    if op == "backward":
        mean = state["mean"].double() if layer else torch.zeros(T, dtype=torch.float64, device=DEV)
        rstd = state["rstd"].double()
        dy = state["dy"].double()
        xh = (x - mean[:, None]) * rstd[:, None]
        g = dy * w[None, :]
        first = g.sum(1) / C if layer else torch.zeros_like(rstd)
        second = (g * xh).sum(1) / C
        dx = (g - first[:, None] - xh * second[:, None]) * rstd[:, None]
        return dx, torch.einsum("tc,tc->c", dy, xh), dy.sum(0) if layer else None
    mean = x.sum(1) / C if layer else torch.zeros(T, dtype=torch.float64, device=DEV)
    rstd = 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / C + EPS)
    y = (x - mean[:, None]) * rstd[:, None] * w[None, :]
    if layer:
        y = y + state["bias"].double()[None, :]
    kept = mean if layer else None
    if op == "norm":
        return y, kept, rstd
    q, s = _exact_codes(y)
    if not case["dual"]:
        return q, s
    qT, sT = _exact_codes(y.t().contiguous())
    return q, s, qT, sT, kept, rstd
