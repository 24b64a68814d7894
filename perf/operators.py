"""Cases of the 8-bit linear layer: what runs, trains and records a pruned, quantized layer.

A layer comes as the joint sparse + quantized sweep leaves it: codes [m, n] in
uint8, a scale and an integer zero point for each output channel (W_hat =
scale * (codes - zero)) and the mask of pruned positions.  Activations X are
token-major [T, n].

    checkpoint   codes of X with one scale a token, and the tensor read back
    linear       the product in 8-bit integers, Y = X_hat W_hat^T
    grad_input   dX = dY W_hat
    grad_weight  dW = kept * (dY^T X_hat), from the 8-bit checkpoint
    step         one training step of the layer: forward, dX and dW

Where ``own`` is false every operator runs in plain torch operations, where it
is true through the package's calls.
"""

import torch

own = False

PAD = 64  # rows of codes are stored with a pitch that is a multiple of this

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


def _case(name, op, T, n, m=0, x="bf16", out="bf16", bits=8, pattern="half"):
    return {"name": name, "op": op, "T": T, "n": n, "m": m, "x": x, "out": out, "bits": bits, "pattern": pattern}


def listed():
    return [
        # a chunk of calibration inputs of a 4096-channel layer, recorded in 8 bits
        _case("checkpoint_calib", "checkpoint", 32768, 4096),
        # a short, odd batch of fp32 activations
        _case("checkpoint_odd_f32", "checkpoint", 203, 1001, x="f32", out="f32"),
        # generating one token with an attention projection: latency counts
        _case("linear_one_token", "linear", 1, 4096, 4096),
        # sixteen sequences generating side by side, the widest layer: the weights are streamed
        _case("linear_decode_wide", "linear", 16, 28672, 8192, pattern="2:4"),
        # a short prompt, sizes off every tile
        _case("linear_prompt_odd", "linear", 300, 1000, 1130, out="f32", bits=4),
        # a batch of prompts through an up projection: the matrix cores count
        _case("linear_prefill", "linear", 8192, 4096, 11008),
        # the input gradient of a small ragged batch
        _case("grad_input_odd", "grad_input", 129, 1000, 2050, out="f32"),
        # the input gradient of a training batch through an up projection
        _case("grad_input_batch", "grad_input", 8192, 4096, 11008),
        # the weight gradient of a small ragged batch
        _case("grad_weight_odd", "grad_weight", 515, 1000, 770, out="bf16", pattern="2:4"),
        # the weight gradient of a training batch, kept in fp32 for accumulation
        _case("grad_weight_batch", "grad_weight", 8192, 4096, 11008, out="f32"),
        # sparse fine-tuning of an attention projection, a few short sequences
        _case("step_short", "step", 512, 4096, 4096),
        # the same on a full batch
        _case("step_batch", "step", 8192, 4096, 4096, pattern="2:4"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["checkpoint", "linear", "linear", "grad_input", "grad_weight", "step"])
    case = {"op": op, "x": "bf16", "bits": rng.choice([8, 8, 4, 3]), "pattern": rng.choice(["half", "2:4", "dense"])}
    case["T"] = _between(rng, 1, 8192)
    case["n"] = _between(rng, 64, 11008)
    case["m"] = _between(rng, 64, 11008)
    if rng.random() < 0.5:  # a model's widths are mostly whole tiles
        case["n"] = (case["n"] + 127) // 128 * 128
        case["m"] = (case["m"] + 127) // 128 * 128
    if case["pattern"] == "2:4":
        case["n"] = (case["n"] + 3) // 4 * 4
    # no drawn case costs more than the largest listed one
    while case["T"] * case["n"] * case["m"] > 4096 * 4096 * 8192:
        case["T"] = (case["T"] + 1) // 2
    case["out"] = "bf16"
    if op == "checkpoint":
        case["m"] = 0
        case["x"] = case["out"] = rng.choice(["bf16", "f32"])
    elif op != "step":
        case["out"] = rng.choice(["bf16", "f32"])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    """Activations, the layer and the gradient, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, n, m = case["T"], case["n"], case["m"]
    f32 = torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=f32)

    d = {}
    # channels of different sizes, a few of them much larger
    size = torch.exp(0.5 * normal(n))
    far = torch.randperm(n, generator=g, device="cuda")[: max(1, n // 512)]
    size[far] *= 20.0
    d["X"] = (normal(T, n) * size).to(_TYPES[case["x"]])
    if not m:
        return d
    W = 0.02 * normal(m, n)
    if case["pattern"] == "2:4":
        low = W.abs().view(m, n // 4, 4).argsort(dim=2)[:, :, :2]
        mask = torch.zeros(m, n // 4, 4, dtype=torch.bool, device="cuda").scatter_(2, low, True).view(m, n)
    elif case["pattern"] == "half":
        mask = W.abs() < 0.02 * 0.6745
    else:
        mask = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    top = 2 ** case["bits"] - 1
    lo, hi = W.amin(1).clamp(max=0.0), W.amax(1).clamp(min=0.0)
    scale = (hi - lo) / top
    zero = torch.round(-lo / scale)
    codes = torch.clamp(torch.round(W / scale[:, None]) + zero[:, None], 0, top)
    d["codes"] = torch.where(mask, zero[:, None].expand(m, n), codes).to(torch.uint8)
    d["scale"], d["zero"] = scale, zero
    d["mask"] = mask.to(torch.uint8)
    d["dY"] = (0.01 * normal(T, m)).to(torch.bfloat16)
    return d


def _quantized(X):
    """(codes int8, scale fp32, sum of codes int32) of each row of X: nearest
    code of 127 x / max|x|, halves to even, taken in 64 bits so that values
    next to a border fall on its right side."""
    a = X.abs().amax(1).float()
    ok = a > 0
    scale = torch.where(ok, a / 127.0, torch.ones_like(a))
    d = torch.where(ok, a, torch.ones_like(a)).double()
    q = torch.round(X.double() * 127.0 / d[:, None])
    return q.to(torch.int8), scale, q.sum(1).to(torch.int32)


def prepare(case, seed):
    d = _inputs(case, seed)
    op, T, n, m = case["op"], case["T"], case["n"], case["m"]
    s = {"op": op, "out": _TYPES[case["out"]], "n": n}
    if op in ("checkpoint", "step"):
        s["X"] = d["X"]
    else:
        # the codes as the forward pass left them: rows padded to the pitch
        q, s["x_scale"], s["x_sum"] = _quantized(d["X"])
        store = torch.zeros(T, (n + PAD - 1) // PAD * PAD, dtype=torch.int8, device="cuda")
        s["q"] = store[:, :n]
        s["q"].copy_(q)
    if m:
        s["codes"], s["scale"], s["zero"] = d["codes"], d["scale"], d["zero"]
        s["mask"], s["dY"] = d["mask"], d["dY"]
    if op == "step":
        s["X"].requires_grad_(True)
        # the trained weights: the gradient takes their shape and type
        s["W"] = (s["scale"][:, None] * (s["codes"].float() - s["zero"][:, None])).to(torch.bfloat16).requires_grad_(True)
    if own and m:
        # a program lays a layer's codes out once
        import post_pruning_amd as sg
        s["layer"] = sg.sg_pack_w8(s["codes"], s["scale"], s["zero"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _w_hat(s):
    return s["scale"][:, None] * (s["codes"].float() - s["zero"][:, None])


def _plain_checkpoint(X, out):
    q, scale, total = _quantized(X)
    return (q.float() * scale[:, None]).to(out), scale, total


def _plain_linear(q, x_scale, s, out):
    return ((q.float() * x_scale[:, None]) @ _w_hat(s).t()).to(out)


def _plain_grad_input(s, out):
    # the layer's weights stand in bf16 in the backward pass
    return (s["dY"].float() @ _w_hat(s).bfloat16().float()).to(out)


def _plain_grad_weight(q, x_scale, s, out):
    # the checkpoint reads back as a bf16 tensor
    x_hat = (q.float() * x_scale[:, None]).bfloat16().float()
    g = s["dY"].float().t() @ x_hat
    return torch.where(s["mask"].bool(), torch.zeros_like(g), g).to(out)


def run(s):
    op = s["op"]
    if own:
        import post_pruning_amd as sg
        if op == "checkpoint":
            q, scale, total = sg.sg_quantize_tokens(s["X"])
            return sg.sg_dequantize_tokens(q, scale, dtype=s["out"]), scale, total
        if op == "linear":
            return sg.sg_linear_w8a8(s["q"], s["x_scale"], s["x_sum"], s["layer"], dtype=s["out"])
        if op == "grad_input":
            return sg.sg_linear_w8_grad_input(s["dY"], s["layer"], dtype=s["out"])
        if op == "grad_weight":
            return sg.sg_linear_w8_grad_weight(s["dY"], s["q"], s["x_scale"], mask=s["mask"], dtype=s["out"])
        Y = sg.linear_w8(s["X"], s["W"], s["layer"], mask=s["mask"])
        dX, dW = torch.autograd.grad(Y, (s["X"], s["W"]), s["dY"])
        return Y.detach(), dX, dW
    if op == "checkpoint":
        return _plain_checkpoint(s["X"], s["out"])
    if op == "linear":
        return _plain_linear(s["q"], s["x_scale"], s, s["out"])
    if op == "grad_input":
        return _plain_grad_input(s, s["out"])
    if op == "grad_weight":
        return _plain_grad_weight(s["q"], s["x_scale"], s, s["out"])
    q, x_scale, _ = _quantized(s["X"].detach())
    return (_plain_linear(q, x_scale, s, s["out"]), _plain_grad_input(s, s["out"]),
            _plain_grad_weight(q, x_scale, s, s["out"]))


def work(case):
    T, n, m, e = case["T"], case["n"], case["m"], _SIZE[case["out"]]
    mul = 2.0 * T * n * m
    linear = T * n + m * n + T * m * e + 8 * (T + m)
    grad_x = 2 * T * m + m * n + T * n * e + 8 * m
    grad_w = 2 * T * m + T * n + m * n + m * n * e + 4 * T
    if case["op"] == "checkpoint":
        return {"bytes": T * n * (_SIZE[case["x"]] + 1 + 1 + e) + 12 * T, "flops": 0}
    if case["op"] == "linear":
        return {"bytes": linear, "flops": mul}
    if case["op"] == "grad_input":
        return {"bytes": grad_x, "flops": mul}
    if case["op"] == "grad_weight":
        return {"bytes": grad_w, "flops": mul}
    return {"bytes": T * n * 3 + linear + grad_x + grad_w, "flops": 3 * mul}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    """The same outputs from the definition, in 64 bits."""
    d = _inputs(case, seed)
    f64 = torch.float64
    X = d["X"].to(f64)
    T, n, m = case["T"], case["n"], case["m"]
    peak = X.abs().max(dim=1, keepdim=True).values
    filled = peak != 0
    code = (X * 127 / peak.masked_fill(~filled, 1.0)).round()
    # the scale and the values read back are kept in fp32 and bf16: these
    # roundings are part of the definition
    unit = torch.where(filled, peak / 127, torch.ones_like(peak)).float().to(f64)
    value = code * unit
    if case["op"] == "checkpoint":
        return value, unit[:, 0], code.sum(1).to(torch.int32)
    weight = (d["codes"].to(f64) - d["zero"].to(f64).unsqueeze(1)) * d["scale"].to(f64).unsqueeze(1)
    grad = d["dY"].to(f64)
    got = []
    if case["op"] in ("linear", "step"):
        got.append(torch.matmul(value, weight.T))
    if case["op"] in ("grad_input", "step"):
        got.append(torch.matmul(grad, weight.float().bfloat16().to(f64)))
    if case["op"] in ("grad_weight", "step"):
        full = torch.matmul(grad.T, value.float().bfloat16().to(f64))
        got.append(full.masked_fill(d["mask"] != 0, 0.0))
    return got[0] if len(got) == 1 else tuple(got)
