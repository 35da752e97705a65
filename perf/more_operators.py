"""The operators around the FP8 linear layer's blocks, as they are measured: the residual sum behind a block together with
the norm in front of the next one (as a tensor, as the codes and scales its products read, and backward; with a gate, a
scale and a norm of the block's output where a model has them), rotary positions and their backward pass, and the AdamW
step over all tensors of a model, with states in 32 bits or in 8.

`run` computes each in its plain form (elementary torch operations in 32 bits, angles in 64), or, where `own` is true, by
the framework's entry points.  `exact` computes it in 64 bits from the definition.

The AdamW step holds 8-bit states as E4M3 codes with one fp32 scale for 128 consecutive elements of a tensor: the first
moment, and the root of the second.  They are rounded to the three bits of a code's mantissa with 16 random bits
(the low half of a number for the moment, the high half for the root); values below the codes' normal range go to
the nearest code, and a root that is not zero never becomes zero.  The random numbers are a function of the seed, the
step, the tensor's place in the list and the element.
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

ADAM = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
STEP, SEED = 100, 20240607
M32 = 0xFFFFFFFF


def listed():
    return [
        # decoding one sequence: behind the attention of one token, latency only
        {"name": "residual_token", "op": "residual", "form": "tensor", "kind": "rms", "T": 1, "C": 2048, "dtype": "bf16",
         "gate": False, "post": False, "scale": 1.0},
        # a ragged batch of a model with norms on both sides of a block and a gate per channel, of a width that is no
        # power of two
        {"name": "residual_gated_odd", "op": "residual", "form": "tensor", "kind": "layer", "T": 1027, "C": 1000,
         "dtype": "fp32", "gate": True, "post": True, "scale": 0.5},
        # a training micro-batch of the layer sweep (4 sequences of 4096 tokens): the next FP8 layer's codes
        {"name": "residual_codes_train", "op": "residual", "form": "dual", "kind": "rms", "T": 16384, "C": 2048,
         "dtype": "bf16", "gate": False, "post": False, "scale": 1.0},
        # its backward pass
        {"name": "residual_backward_train", "op": "residual_backward", "kind": "rms", "T": 16384, "C": 2048,
         "dtype": "bf16", "gate": False, "post": False, "scale": 1.0},
        # the same with a gate and a norm behind the block
        {"name": "residual_backward_gated", "op": "residual_backward", "kind": "rms", "T": 16384, "C": 2048,
         "dtype": "bf16", "gate": True, "post": True, "scale": 0.5},
        # decoding one sequence: 16 query and 8 key heads of one token, far into a long context
        {"name": "rotary_token", "op": "rotary", "T": 1, "H": 24, "of": 32, "D": 128, "rot": 128, "layout": "half",
         "dtype": "bf16", "start": 100000, "scale": 1.0, "inverse": False},
        # the micro-batch's query and key heads, in the rows that the qkv projection left
        {"name": "rotary_train", "op": "rotary", "T": 16384, "H": 24, "of": 32, "D": 128, "rot": 128, "layout": "half",
         "dtype": "bf16", "start": 0, "scale": 1.0, "inverse": False},
        # the gradient of a ragged batch in fp32: part of an odd-sized head, pairs side by side, a scaled long context
        {"name": "rotary_backward_part", "op": "rotary", "T": 3001, "H": 20, "of": 20, "D": 80, "rot": 32,
         "layout": "interleaved", "dtype": "fp32", "start": 1000000, "scale": 1.1, "inverse": True},
        # a small test model: many short tensors, views of flat buckets at odd offsets
        {"name": "adamw_small", "op": "adamw", "layers": 3, "div": 16, "bits": 32, "param": "fp32", "grad": "fp32",
         "odd": True, "clip": False},
        # eight layers of the sweep, fp32 throughout, the gradients clipped by their global norm on the way
        {"name": "adamw_model", "op": "adamw", "layers": 8, "div": 1, "bits": 32, "param": "fp32", "grad": "fp32",
         "odd": False, "clip": True},
        # one layer with bf16 weights and gradients, an fp32 master copy and 8-bit states
        {"name": "adamw8_layer", "op": "adamw", "layers": 1, "div": 1, "bits": 8, "param": "bf16", "grad": "bf16",
         "odd": False, "clip": False},
        # eight layers with 8-bit states
        {"name": "adamw8_model", "op": "adamw", "layers": 8, "div": 1, "bits": 8, "param": "fp32", "grad": "fp32",
         "odd": False, "clip": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("residual", "residual_backward", "rotary", "adamw"))
    if op == "adamw":
        return {"op": op, "layers": rng.randint(1, 6), "div": rng.choice((1, 1, 2, 4, 8, 16)), "bits": rng.choice((8, 32)),
                "param": rng.choice(("fp32", "bf16")), "grad": rng.choice(("fp32", "bf16")), "odd": rng.random() < 0.5,
                "clip": rng.random() < 0.5}
    if op == "rotary":
        D = 2 * _log(rng, 16, 128)
        H = _log(rng, 1, 40)
        most = 16384 * 24 * 128                           # elements: the largest listed case
        return {"op": op, "T": _log(rng, 1, min(16384, most // (H * D))), "H": H, "of": H + rng.choice((0, 0, 8)), "D": D,
                "rot": D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2), "layout": rng.choice(("half", "interleaved")),
                "dtype": rng.choice(("bf16", "bf16", "fp32")), "start": rng.choice((0, 0, 5000, 1000000)),
                "scale": rng.choice((1.0, 1.0, 1.1)), "inverse": rng.random() < 0.4}
    case = {"op": op, "kind": rng.choice(("layer", "rms")), "dtype": rng.choice(("bf16", "bf16", "fp32"))}
    most = 16384 * 2048                                   # elements: the largest listed case
    if op == "residual":
        case["form"] = rng.choice(("tensor", "codes", "dual"))
    if case.get("form", "tensor") == "tensor":
        case["C"] = _log(rng, 64, 8192)
        case["T"] = _log(rng, 1, min(16384, most // case["C"]))
    else:
        case["C"] = 128 * _log(rng, 1, 64)
        rows = min(16384, most // case["C"])
        case["T"] = 128 * _log(rng, 1, max(1, rows // 128)) if case["form"] == "dual" else _log(rng, 1, rows)
    case["gate"], case["post"] = rng.random() < 0.5, rng.random() < 0.5
    case["scale"] = rng.choice((1.0, 0.5, 0.22))
    return case


def _heavy(shape, g):
    """Student-t with 3 degrees of freedom: the heavy tails of activations and their gradients."""
    z = torch.randn(shape, generator=g, device=DEV)
    chi = torch.zeros(shape, device=DEV)
    for _ in range(3):
        chi += torch.randn(shape, generator=g, device=DEV).square_()
    return z / (chi / 3).sqrt_()


def _adam_shapes(case):
    """The tensors of `layers` layers, each dimension divided by `div`: the weights, two norm weights, and a bias of odd
    length per layer."""
    d = case["div"]
    return [s for _ in range(case["layers"])
            for s in [(n // d, k // d) for n, k in LAYER] + [(2048 // d,), (2048 // d,), (2048 // d - 1,)]]


def _prepare_adamw(case, g):
    shapes = _adam_shapes(case)
    sizes = [math.prod(s) for s in shapes]
    # one flat buffer for each kind of tensor, the tensors behind each other or each from a multiple of 128 elements
    room = [n if case["odd"] else -(-n // 128) * 128 for n in sizes]
    total, eight = sum(room), case["bits"] == 8

    def views(flat):
        return [v[:n].view(s) for v, n, s in zip(flat.split(room), sizes, shapes)]

    state = {"case": case, "flat": {}}

    def keep(name, flat):
        state["flat"][name] = flat
        state[name] = views(flat)

    grad = torch.randn(total, generator=g, device=DEV) * 1e-3
    keep("grads", grad.to(DTYPES[case["grad"]]))
    full = torch.randn(total, generator=g, device=DEV) * 0.02
    keep("params", full.to(DTYPES[case["param"]]))
    if case["param"] == "bf16":
        keep("masters", full)
    avg = torch.randn(total, generator=g, device=DEV) * 3e-4
    root = (torch.randn(total, generator=g, device=DEV).square_() + 0.25).sqrt_().mul_(1e-3)
    if not eight:
        keep("avg", avg)
        keep("sq", root.square_())
    else:
        blocks = [-(-n // 128) for n in sizes]
        for name, flat in (("avg", avg), ("sq", root)):
            coded = [_code_blocks(v) for v in views(flat)]
            state["flat"][name + "_scale"] = torch.cat([s for _, s in coded])
            state[name + "_scale"] = list(state["flat"][name + "_scale"].split(blocks))
            codes = torch.zeros(total, dtype=torch.uint8, device=DEV)
            for v, (q, _) in zip(views(codes), coded):
                v.view(-1).copy_(q)
            keep(name, codes)
    state["norm"] = None
    if case["clip"]:
        state["norm"] = sum(v.double().square().sum() for v in state["grads"]).sqrt().float()
    return state


def _code_blocks(v):
    """Codes (nearest) and scales of the blocks of 128 elements of a tensor, as an earlier step left them."""
    flat = v.reshape(-1)
    n = flat.numel()
    blocks = torch.nn.functional.pad(flat, (0, -n % 128)).view(-1, 128)
    amax = blocks.abs().amax(1).clamp_min(AMAX_FLOOR)
    q = (blocks * (E4M3_MAX / amax)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(-1)[:n], amax / E4M3_MAX


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, g)
    dtype = DTYPES[case["dtype"]]
    T = case["T"]
    if op == "rotary":
        rows = _heavy((T, case["of"], case["D"]), g).to(dtype)
        half = case["rot"] // 2
        freqs = 1000000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        # the positions of a batch of sequences of different lengths, each counted from `start`
        at = torch.arange(T, device=DEV)
        length = max(1, (3 * T + 4) // 7)
        return {"case": case, "x": rows[:, : case["H"]], "freqs": freqs, "positions": case["start"] + at % length}
    C = case["C"]

    def vector(mean, dev):
        return (mean + dev * torch.randn(C, generator=g, device=DEV)).to(dtype)

    state = {"case": case, "x": (_heavy((T, C), g) + 0.1).to(dtype), "weight": vector(1.0, 0.1), "bias": None, "gate": None,
             "post_weight": None}
    if case["kind"] == "layer":
        state["bias"] = vector(0.0, 0.1)
    if case["gate"]:
        state["gate"] = vector(0.3, 0.2)
    if case["post"]:
        state["post_weight"] = vector(1.0, 0.1)
    h = (_heavy((T, C), g) * 2).to(dtype)
    if op == "residual":
        state["h"] = h
        return state
    # what the forward pass keeps: the sum as written, and each norm's statistics
    state["h_out"] = h
    state["dy"] = (_heavy((T, C), g) * 1e-3).to(dtype)
    state["dh_out"] = (_heavy((T, C), g) * 1e-3).to(dtype)
    state["mean"], state["rstd"] = _stats64(h, case["kind"])
    state["post_mean"], state["post_rstd"] = _stats64(state["x"], case["kind"]) if case["post"] else (None, None)
    return state


def _stats64(x, kind):
    x = x.double()
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=x.dtype, device=DEV)
    rstd = ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()
    return mean.float() if kind == "layer" else None, rstd.float()


# ---- the plain forms ---------------------------------------------------------------------------------------------------

def _normed(x, layer, weight, bias):
    """The plain norm of fp32 rows: (y, mean, rstd)."""
    mean = x.mean(1, keepdim=True) if layer else None
    d = x - mean if layer else x
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd * weight.float()
    if bias is not None:
        y = y + bias.float()
    return y, mean[:, 0] if layer else None, rstd[:, 0]


def _coded(y):
    """Codes and scales of the groups of 128 along the last axis of y [R, K]: codes [R, K], scales [K/128, R]."""
    R, K = y.shape
    v = y.view(R, K // 128, 128)
    amax = v.abs().amax(2).clamp_min(AMAX_FLOOR)
    q = (v * (E4M3_MAX / amax)[:, :, None]).view(R, K).to(torch.float8_e4m3fn)
    return q, (amax / E4M3_MAX).t().contiguous()


def _plain_residual(state):
    case = state["case"]
    layer = case["kind"] == "layer"
    p, post_mean, post_rstd = state["x"].float(), None, None
    if case["post"]:
        p, post_mean, post_rstd = _normed(p, layer, state["post_weight"], None)
    factor = case["scale"] * state["gate"].float() if case["gate"] else case["scale"]
    h_out = (state["h"].float() + factor * p).to(state["h"].dtype)
    # the norm is that of the sum as it is written
    y, mean, rstd = _normed(h_out.float(), layer, state["weight"], state["bias"])
    if case["form"] == "tensor":
        return y.to(h_out.dtype), h_out, mean, rstd, post_mean, post_rstd
    q, s = _coded(y)
    if case["form"] == "codes":
        return q, s, h_out
    qT, sT = _coded(y.t().contiguous())
    return q, s, qT, sT, h_out, mean, rstd, post_mean, post_rstd


def _norm_back(dy, x, layer, weight, mean, rstd):
    """(dx, x normalised) of the plain norm's backward pass, in fp32."""
    xh = (x - mean[:, None]) * rstd[:, None] if layer else x * rstd[:, None]
    u = dy * weight.float()
    d = u - xh * (u * xh).mean(1, keepdim=True)
    if layer:
        d = d - u.mean(1, keepdim=True)
    return d * rstd[:, None], xh


def _plain_residual_backward(state):
    case = state["case"]
    layer = case["kind"] == "layer"
    dtype = state["x"].dtype
    dy, x = state["dy"].float(), state["x"].float()
    d, xh = _norm_back(dy, state["h_out"].float(), layer, state["weight"], state["mean"], state["rstd"])
    d = d + state["dh_out"].float()
    dweight, dbias = (dy * xh).sum(0), dy.sum(0) if layer else None
    dp = d * (case["scale"] * state["gate"].float()) if case["gate"] else d * case["scale"]
    dgate = dpost = None
    p, dx = x, dp
    if case["post"]:
        dx, ph = _norm_back(dp, x, layer, state["post_weight"], state["post_mean"], state["post_rstd"])
        dpost = (dp * ph).sum(0)
        p = ph * state["post_weight"].float()
    if case["gate"]:
        dgate = case["scale"] * (d * p).sum(0)
    return d.to(dtype), dx.to(dtype), dweight, dbias, dgate, dpost


def _plain_rotary(state):
    case = state["case"]
    x, rot = state["x"], case["rot"]
    angle = state["positions"].double()[:, None] * state["freqs"][None, :]
    c, s = (f(angle).float()[:, None, :] * case["scale"] for f in (torch.cos, torch.sin))
    if case["inverse"]:
        s = -s
    v = x.float()
    if case["layout"] == "half":
        a, b = v[..., : rot // 2], v[..., rot // 2: rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    else:
        a, b = v[..., 0:rot:2], v[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    return torch.cat([turned, v[..., rot:]], dim=-1).to(x.dtype)


def _mix(h):
    """Murmur3's 32-bit finalizer, of numbers held in 64 bits."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & M32
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def _shift(x):
    """One step of the 32-bit xorshift generator (13, 17, 5)."""
    x = (x ^ (x << 13)) & M32
    x = x ^ (x >> 17)
    return (x ^ (x << 5)) & M32


def _randoms(place, blocks):
    """The random numbers of the blocks of 128 elements of the list's tensor `place`: [blocks, 128], 32 bits each."""
    key = _mix(_mix(_mix(_mix(SEED & M32) ^ (SEED >> 32)) ^ (STEP & M32)) ^ place)
    k = torch.arange(16 * blocks, device=DEV)
    x = _mix(((key ^ (k >> 32)) + (k & M32) * 0x9E3779B9) & M32) | 1
    steps = [x := _shift(x) for _ in range(8)]
    return torch.stack(steps, dim=-1).view(blocks, 128)


def _rounded_codes(v, bits, root):
    """Codes [blocks, 128] of fp32 values with 16 random bits each, and the blocks' scales."""
    amax = v.abs().amax(1).clamp_min(AMAX_FLOOR)
    y = v * (E4M3_MAX / amax)[:, None]
    r = ((y.view(torch.int32) + (bits << 4).to(torch.int32)) & -0x100000).view(torch.float32)
    if root:
        r = torch.where(v > 0, r.clamp_min(2.0 ** -9), r)
    return r.to(torch.float8_e4m3fn).view(torch.uint8), amax / E4M3_MAX


def _plain_adamw_tensor(state, place, coef):
    a, eight = ADAM, state["case"]["bits"] == 8
    held = state["masters"][place] if "masters" in state else state["params"][place]
    n = held.numel()
    g = state["grads"][place].reshape(-1).float()
    if coef is not None:
        g = g * coef
    if eight:
        pad, blocks = -n % 128, -(-n // 128)
        g = torch.nn.functional.pad(g, (0, pad)).view(blocks, 128)

        def value(name):
            q = torch.nn.functional.pad(state[name][place].view(-1), (0, pad)).view(torch.float8_e4m3fn)
            return q.float().view(blocks, 128) * state[name + "_scale"][place][:, None]
        m, v = value("avg"), value("sq").square()
    else:
        m, v = state["avg"][place].view(-1), state["sq"][place].view(-1)
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g * g
    root = v.sqrt()
    den = root * (1 - a["beta2"] ** STEP) ** -0.5 + a["eps"]
    update = (a["lr"] / (1 - a["beta1"] ** STEP)) * (m / den)
    if eight:
        update = update.view(-1)[:n]
        bits = _randoms(place, blocks)
        for name, x, r in (("avg", m, bits & 0xFFFF), ("sq", root, bits >> 16)):
            q, s = _rounded_codes(x, r, name == "sq")
            state[name][place].view(-1).copy_(q.view(-1)[:n])
            state[name + "_scale"][place].copy_(s)
    else:
        state["avg"][place].view(-1).copy_(m)
        state["sq"][place].view(-1).copy_(v)
    p = held.view(-1).float() * (1 - a["lr"] * a["weight_decay"]) - update
    held.view(-1).copy_(p)
    if "masters" in state:
        state["params"][place].view(-1).copy_(p)


def _adamw_outputs(state):
    flat, eight = state["flat"], state["case"]["bits"] == 8
    out = [flat["params"], flat.get("masters")]
    if not eight:
        return out + [flat["avg"], flat["sq"]]
    return out + [flat[k].view(torch.float8_e4m3fn) for k in ("avg", "sq")] + [flat["avg_scale"], flat["sq_scale"]]


def _run_plain(state):
    op = state["case"]["op"]
    if op == "residual":
        return _plain_residual(state)
    if op == "residual_backward":
        return _plain_residual_backward(state)
    if op == "rotary":
        return _plain_rotary(state)
    coef = None if state["norm"] is None else (1.0 / (state["norm"] + 1e-6)).clamp_max(1.0)
    for place in range(len(state["params"])):
        _plain_adamw_tensor(state, place, coef)
    return _adamw_outputs(state)


# ---- the framework's calls ---------------------------------------------------------------------------------------------

def _run_own(state):
    import blockwise_scaled_fp8_quant_amd as P
    case = state["case"]
    op = case["op"]
    f8 = torch.float8_e4m3fn
    if op == "rotary":
        return P.puro_rotary(state["x"], state["freqs"], state["positions"], scale=case["scale"], inverse=case["inverse"],
                             layout=P.ROTARY_HALF if case["layout"] == "half" else P.ROTARY_INTERLEAVED)
    if op == "adamw":
        P.puro_adamw(state["params"], state["grads"], state["avg"], state["sq"], STEP, masters=state.get("masters"),
                     avg_scales=state.get("avg_scale"), sq_scales=state.get("sq_scale"), norm=state["norm"], max_norm=1.0,
                     seed=SEED, **ADAM)
        return _adamw_outputs(state)
    kind = P.LAYER_NORM if case["kind"] == "layer" else P.RMS_NORM
    how = {"kind": kind, "gate": state["gate"], "post_weight": state["post_weight"], "scale": case["scale"]}
    if op == "residual_backward":
        return P.puro_residual_norm_backward(state["dy"], state["h_out"], state["weight"], state["mean"], state["rstd"],
                                             x=state["x"], post_mean=state["post_mean"], post_rstd=state["post_rstd"],
                                             dh_out=state["dh_out"], with_bias=case["kind"] == "layer", **how)
    h, x, weight, bias = state["h"], state["x"], state["weight"], state["bias"]
    if case["form"] == "tensor":
        return P.puro_residual_norm(h, x, weight, bias, eps=EPS, **how)
    if case["form"] == "codes":
        q, s, h_out = P.puro_residual_norm_quant(h, x, weight, bias, eps=EPS, **how)
        return q.view(f8), s, h_out
    q, s, qT, sT, *rest = P.puro_residual_norm_quant_dual(h, x, weight, bias, eps=EPS, **how)
    return q.view(f8), s, qT.view(f8), sT, *rest


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op = case["op"]
    if op == "adamw":
        sizes = [math.prod(s) for s in _adam_shapes(case)]
        n, blocks = sum(sizes), sum(-(-s // 128) for s in sizes)
        each = 8 + (2 if case["param"] == "bf16" else 0) + (2 if case["grad"] == "bf16" else 4)
        states = 16 * n if case["bits"] == 32 else 4 * n + 16 * blocks
        return {"bytes": each * n + states, "flops": (16 if case["bits"] == 32 else 24) * n}
    e = 2 if case["dtype"] == "bf16" else 4
    T = case["T"]
    if op == "rotary":
        n = T * case["H"] * case["D"]
        return {"bytes": 2 * n * e + 8 * T + 4 * case["rot"], "flops": 3 * T * case["H"] * case["rot"] + 20 * T * case["rot"]}
    C, layer = case["C"], case["kind"] == "layer"
    n = T * C
    stats = (8 if layer else 4) * T * (2 if case["post"] else 1)
    vectors = 1 + layer + case["gate"] + case["post"]
    if op == "residual_backward":
        # read dy, the sum, its gradient, and the block's output where a norm or gate needs it; write one or two gradients
        one = not case["gate"] and not case["post"]
        moved = 4 * n if one and case["scale"] == 1.0 else 5 * n if one else 6 * n
        return {"bytes": moved * e + stats + (vectors - layer) * C * e + vectors * C * 4,
                "flops": (30 if case["post"] else 18) * n}
    out = {"tensor": n * e, "codes": n + n // 32, "dual": 2 * (n + n // 32)}[case["form"]]
    kept = 0 if case["form"] == "codes" else stats
    return {"bytes": 3 * n * e + out + kept + vectors * C * e, "flops": (20 if case["post"] else 12) * n}


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


def _exact_norm(x, layer, w, b):
    n = x.shape[1]
    mean = x.sum(1) / n if layer else torch.zeros(x.shape[0], dtype=torch.float64, device=DEV)
    rstd = 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / n + EPS)
    y = (x - mean[:, None]) * rstd[:, None] * w[None, :]
    if b is not None:
        y = y + b.double()[None, :]
    return y, mean if layer else None, rstd


def _exact_residual(state):
    case = state["case"]
    layer = case["kind"] == "layer"
    branch, pm, pr = state["x"].double(), None, None
    if case["post"]:
        branch, pm, pr = _exact_norm(branch, layer, state["post_weight"].double(), None)
    if case["gate"]:
        branch = branch * state["gate"].double()[None, :]
    total = state["h"].double() + case["scale"] * branch
    stored = total.to(state["h"].dtype).double()
    y, mean, rstd = _exact_norm(stored, layer, state["weight"].double(), state["bias"])
    if case["form"] == "tensor":
        return y, total, mean, rstd, pm, pr
    q, s = _exact_codes(y)
    if case["form"] == "codes":
        return q, s, total
    qT, sT = _exact_codes(y.t().contiguous())
    return q, s, qT, sT, total, mean, rstd, pm, pr


def _exact_residual_backward(state):
    case = state["case"]
    layer = case["kind"] == "layer"

    def back(grad, x, w, mean, rstd):
        r = rstd.double()[:, None]
        xh = (x - (mean.double()[:, None] if layer else 0.0)) * r
        u = grad * w.double()[None, :]
        first = u.sum(1, keepdim=True) / u.shape[1] if layer else 0.0
        second = (u * xh).sum(1, keepdim=True) / u.shape[1]
        return (u - first - xh * second) * r, xh

    dy, x = state["dy"].double(), state["x"].double()
    d, xh = back(dy, state["h_out"].double(), state["weight"], state["mean"], state["rstd"])
    d = d + state["dh_out"].double()
    gate = state["gate"].double() if case["gate"] else torch.ones(x.shape[1], dtype=torch.float64, device=DEV)
    dp = d * gate[None, :] * case["scale"]
    if case["post"]:
        dx, ph = back(dp, x, state["post_weight"], state["post_mean"], state["post_rstd"])
        branch = ph * state["post_weight"].double()[None, :]
        dpost = torch.einsum("tc,tc->c", dp, ph)
    else:
        dx, branch, dpost = dp, x, None
    dgate = case["scale"] * torch.einsum("tc,tc->c", d, branch) if case["gate"] else None
    return d, dx, torch.einsum("tc,tc->c", dy, xh), dy.sum(0) if layer else None, dgate, dpost


def _exact_rotary(state):
    case = state["case"]
    out = state["x"].double().clone()
    half = case["rot"] // 2
    first = torch.arange(half, device=DEV)
    second = first + half
    if case["layout"] == "interleaved":
        first, second = 2 * first, 2 * first + 1
    angle = torch.outer(state["positions"].double(), state["freqs"]) * (-1.0 if case["inverse"] else 1.0)
    turn = torch.polar(torch.full_like(angle, case["scale"]), angle)[:, None, :]
    z = torch.complex(out[..., first], out[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_random(place, elements):
    """The random numbers of a tensor's elements, from the generator's definition: each of the group of eight's steps is
    taken by those elements that are behind it."""
    def finish(h):
        h = torch.bitwise_xor(h, torch.div(h, 65536, rounding_mode="floor"))
        h = torch.remainder(h * 2246822507, 2 ** 32)
        h = torch.bitwise_xor(h, torch.div(h, 8192, rounding_mode="floor"))
        h = torch.remainder(h * 3266489909, 2 ** 32)
        return torch.bitwise_xor(h, torch.div(h, 65536, rounding_mode="floor"))

    key = torch.zeros((), dtype=torch.int64, device=DEV)
    for word in (SEED % 2 ** 32, SEED // 2 ** 32, STEP % 2 ** 32, place):
        key = finish(torch.bitwise_xor(key, torch.tensor(word, device=DEV)))
    i = torch.arange(elements, device=DEV)
    group, lane = i // 8, i % 8
    x = torch.bitwise_xor(key, group // 2 ** 32)
    x = finish(torch.remainder(x + torch.remainder(group, 2 ** 32) * 2654435769, 2 ** 32))
    x = torch.bitwise_or(x, torch.ones_like(x))
    for k in range(8):
        y = torch.bitwise_xor(x, torch.remainder(x * 8192, 2 ** 32))
        y = torch.bitwise_xor(y, y // 131072)
        y = torch.bitwise_xor(y, torch.remainder(y * 32, 2 ** 32))
        x = torch.where(lane >= k, y, x)
    return x


def _exact_rounded(v, chance, root):
    """The value of each element's code, with `chance` in [0, 1) added to the last place before it is cut, and the scales."""
    n = v.numel()
    padded = torch.zeros(-(-n // 128) * 128, dtype=torch.float64, device=DEV)
    padded[:n] = v
    scale = padded.view(-1, 128).abs().max(dim=1).values.clamp_min(AMAX_FLOOR) / E4M3_MAX
    y = v / scale.repeat_interleave(128)[:n]
    mag, e = torch.frexp(y.abs())                                          # mag in [0.5, 1)
    cut = torch.ldexp(torch.floor(mag * 16 + chance) / 16, e)
    if root:
        cut = torch.where(v > 0, torch.maximum(cut, torch.full_like(cut, 2.0 ** -9)), cut)
    return torch.copysign(_e4m3(cut), v), scale


def _exact_adamw(state):
    case, a = state["case"], ADAM
    eight = case["bits"] == 8
    factor = 1.0 if state["norm"] is None else min(1.0, 1.0 / (float(state["norm"]) + 1e-6))
    flat = {k: v.double() for k, v in state["flat"].items() if v.dtype != torch.uint8}
    if eight:
        flat.update({k: _exact_value(state["flat"][k]) for k in ("avg", "sq")})
    done = {k: 0 for k in flat}

    def part(name, n, room):
        at = done[name]
        done[name] = at + room
        return flat[name][at: at + n]

    for place, shape in enumerate(_adam_shapes(case)):
        n = math.prod(shape)
        room = n if case["odd"] else -(-n // 128) * 128
        g = part("grads", n, room) * factor
        p = part("params", n, room)
        held = part("masters", n, room) if "masters" in flat else p
        m, v = part("avg", n, room), part("sq", n, room)
        scales = [part(k + "_scale", -(-n // 128), -(-n // 128)) for k in ("avg", "sq")] if eight else None
        before_m, before_v = (m, v) if not eight else (m * scales[0].repeat_interleave(128)[:n],
                                                       (v * scales[1].repeat_interleave(128)[:n]) ** 2)
        new_m = a["beta1"] * before_m + (1 - a["beta1"]) * g
        new_v = a["beta2"] * before_v + (1 - a["beta2"]) * g ** 2
        mean = new_m / (1 - a["beta1"] ** STEP)
        deviation = torch.sqrt(new_v / (1 - a["beta2"] ** STEP))
        new_p = held - a["lr"] * (a["weight_decay"] * held + mean / (deviation + a["eps"]))
        held.copy_(new_p)
        p.copy_(new_p)
        if eight:
            number = _exact_random(place, n)
            for old, new, s, r, root in ((m, new_m, scales[0], number % 65536, False),
                                         (v, torch.sqrt(new_v), scales[1], number // 65536, True)):
                values, scale = _exact_rounded(new, r.double() / 65536, root)
                old.copy_(values)
                s.copy_(scale)
        else:
            m.copy_(new_m)
            v.copy_(new_v)
    out = [flat["params"], flat.get("masters"), flat["avg"], flat["sq"]]
    return out + [flat["avg_scale"], flat["sq_scale"]] if eight else out


def exact(case, seed):
    state = prepare(case, seed)
    return {"residual": _exact_residual, "residual_backward": _exact_residual_backward, "rotary": _exact_rotary,
            "adamw": _exact_adamw}[case["op"]](state)
