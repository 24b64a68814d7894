"""Cases of the layer in 8-bit floating point and of dropout: what runs and fine-tunes a pruned layer.

Numbers are held in 8 bits (e4m3, gradients also e5m2) with one scale, a power
of two, for every block of 128: 128 neighbours along the contraction for
activations X [T, n] and gradients dY [T, m], 128 x 128 for weights W [m, n].
Dropout draws its numbers from a counter (Philox4x32-10), so that its mask is
made anew wherever it is needed.

    checkpoint  codes of X (after dropout, if there is one) and the tensor they stand for; for training along both directions
    linear      Y = X_hat W_hat^T
    backward    a layer's backward pass: dY in 8 bits, dX = drop(dY_hat W_hat), dW = kept * (dY_hat^T X_hat)
    dropout     residual + drop(X), and the gradient with respect to X
    step        one training step of the layer from its weights: pack W, drop and quantize X, Y, dX and dW

Where ``own`` is false every operator runs in plain torch operations, where it
is true through the package's calls.
"""

import torch

own = False

BLOCK = 128

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_SIZE = {"bf16": 2, "f32": 4}


def _case(name, op, T, n, m=0, x="bf16", out="bf16", p=0.0, fmt="e4m3", both=False, residual=False, pattern="half"):
    return {"name": name, "op": op, "T": T, "n": n, "m": m, "x": x, "out": out, "p": p, "fmt": fmt, "both": both,
            "residual": residual, "pattern": pattern}


def listed():
    return [
        # one generated token's activation: latency counts
        _case("checkpoint_token", "checkpoint", 1, 4096),
        # a training batch, dropped and quantized for the forward and for the backward pass
        _case("checkpoint_train", "checkpoint", 8192, 4096, p=0.1, both=True),
        # generating one token with an attention projection: latency counts
        _case("linear_one_token", "linear", 1, 4096, 4096),
        # sixteen sequences generating side by side, the widest layer: the weights are streamed
        _case("linear_decode_wide", "linear", 16, 28672, 8192, pattern="2:4"),
        # a short prompt, sizes off every tile and block
        _case("linear_prompt_odd", "linear", 300, 1000, 1130, out="f32"),
        # a batch of prompts through an up projection: the matrix cores count
        _case("linear_prefill", "linear", 8192, 4096, 11008),
        # the backward pass of a small ragged batch, gradients in the wide-range format
        _case("backward_odd", "backward", 515, 1000, 770, out="f32", p=0.25, fmt="e5m2", pattern="2:4"),
        # the backward pass of a training batch through an up projection
        _case("backward_batch", "backward", 8192, 4096, 11008),
        # dropout of a short odd fp32 activation
        _case("dropout_odd_f32", "dropout", 203, 1001, x="f32", out="f32", p=0.1),
        # dropout of a block's output with its residual, a training batch of a wide model
        _case("dropout_residual_batch", "dropout", 8192, 8192, p=0.1, residual=True),
        # sparse fine-tuning of an attention projection, a few short sequences
        _case("step_short", "step", 512, 4096, 4096, p=0.1),
        # the same on a full batch
        _case("step_batch", "step", 8192, 4096, 4096, p=0.05, pattern="2:4"),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["checkpoint", "linear", "linear", "backward", "backward", "dropout", "step"])
    case = {"op": op, "x": "bf16", "out": "bf16", "pattern": rng.choice(["half", "2:4", "dense"])}
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
    case["p"] = 0.0
    if op != "linear":
        case["p"] = round(0.01 + 0.5 * rng.random(), 3) if op == "dropout" or rng.random() < 0.5 else 0.0
    case["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"]) if op in ("checkpoint", "backward", "step") else "e4m3"
    case["both"] = op == "checkpoint" and rng.random() < 0.5
    case["residual"] = op == "dropout" and rng.random() < 0.5
    if op in ("checkpoint", "dropout"):
        case["m"] = 0
        case["pattern"] = "half"
        case["x"] = case["out"] = rng.choice(["bf16", "f32"])
    elif op != "step":
        case["out"] = rng.choice(["bf16", "f32"])
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _inputs(case, seed):
    """Activations, the weights, the gradient and the random numbers' key, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T, n, m = case["T"], case["n"], case["m"]
    f32 = torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=f32)

    d = {"key": (int(seed) * 0x9E3779B97F4A7C15 + 0x632BE59BD9B4E019) % (1 << 64), "offset": (int(seed) << 33) + 7}
    # channels of different sizes, a few of them much larger
    size = torch.exp(0.5 * normal(n))
    far = torch.randperm(n, generator=g, device="cuda")[: max(1, n // 512)]
    size[far] *= 20.0
    d["X"] = (normal(T, n) * size).to(_TYPES[case["x"]])
    if case["op"] == "dropout":
        d["R"] = normal(T, n).to(_TYPES[case["x"]]) if case["residual"] else None
        d["dY"] = (0.01 * normal(T, n)).to(_TYPES[case["x"]])
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
    d["W"] = W.masked_fill_(mask, 0.0).bfloat16()
    d["mask"] = mask.to(torch.uint8)
    # gradients differ in size from token to token
    d["dY"] = (0.01 * normal(T, m) * torch.exp(normal(T, 1))).to(torch.bfloat16)
    return d


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
_TOP = {torch.float8_e4m3fn: 8, torch.float8_e5m2: 15}  # the largest value is 1.75 * 2^TOP


def _exponent(peak, fmt):
    """The least whole e >= -127 with peak <= 1.75 * 2^(TOP + e); 0 for a peak of 0."""
    f, e = torch.frexp(peak)
    e = e - _TOP[fmt] - 1 + (f > 0.875).to(e.dtype)
    return torch.where(peak > 0, e.clamp(min=-127), torch.zeros_like(e))


def _power(e):
    """2^e in fp32 for whole e from -127 on, from its bits."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _padded(X, rows, cols):
    return torch.nn.functional.pad(X, (0, -X.shape[1] % cols, 0, -X.shape[0] % rows))


def _codes(X, fmt, rows=1, cols=BLOCK):
    """(codes, exponents) of blocks of rows x cols of a fp32 X; the exponents
    [blocks along a row, rows of X] as whole numbers from 0 (2^-127) on."""
    h, w = X.shape
    P = _padded(X, rows, cols)
    H, V = P.shape[0] // rows, P.shape[1] // cols
    P = P.view(H, rows, V, cols)
    e = _exponent(P.abs().amax((1, 3)), fmt)  # [H, V]
    q = (P * _power(-e)[:, None, :, None]).view(H * rows, V * cols).to(fmt)
    scale = (e + 127).to(torch.uint8).repeat_interleave(rows, 0)[:h].t().contiguous()
    return q[:h, :w], scale


def _values(q, scale, cols=BLOCK):
    e = (scale.t().to(torch.int32) - 127).repeat_interleave(cols, 1)[:, : q.shape[1]]
    return q.float() * _power(e)


def _keep(T, n, d, p):
    """Truth values [T, n]: element (t, c) takes word c % 4 of the Philox4x32-10
    numbers of the counter (c / 4, t, offset) and is kept where that is at
    least p 2^32."""
    low = 0xFFFFFFFF
    c0 = torch.arange((n + 3) // 4, device="cuda").expand(T, -1)
    c1 = torch.arange(T, device="cuda")[:, None].expand_as(c0)
    c2 = torch.full_like(c0, d["offset"] & low)
    c3 = torch.full_like(c0, d["offset"] >> 32)
    k0, k1 = d["key"] & low, d["key"] >> 32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64, as whole numbers with a sign
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return (torch.stack((c0, c1, c2, c3), 2) >= round(p * 2.0**32)).view(T, -1)[:, :n]


def _drop(X, keep, p):
    """fp32: the kept elements times 1 / (1 - p), which is rounded to fp32."""
    grow = torch.tensor(1.0 / (1.0 - p), dtype=torch.float32, device="cuda")
    return torch.where(keep, X.float() * grow, 0.0)


def _dropped(s):
    if s["p"] == 0.0:
        return s["X"].detach().float()
    return _drop(s["X"].detach(), _keep(*s["X"].shape, s, s["p"]), s["p"])


def _plain_checkpoint(X, s):
    q, scale = _codes(X, s["fmt"])
    got = (_values(q, scale).to(s["out"]), scale)
    if s["both"]:
        q, scale = _codes(X.t().contiguous(), s["fmt"])
        got += (_values(q, scale).to(s["out"]), scale)
    return got


def _plain_backward(w_hat, xt_hat, s):
    dY = s["dY"].float()
    dX = _values(*_codes(dY, s["fmt"])) @ w_hat
    if s["p"] != 0.0:
        dX = _drop(dX, _keep(*dX.shape, s, s["p"]), s["p"])
    dW = _values(*_codes(dY.t().contiguous(), s["fmt"])) @ xt_hat.t()
    return dX.to(s["out"]), torch.where(s["mask"].bool(), torch.zeros_like(dW), dW).to(s["out"])


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------
def _stored(q):
    """Codes in rows of whole blocks, as the package keeps them."""
    wide = torch.zeros(q.shape[0], (q.shape[1] + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.uint8, device="cuda")
    wide[:, : q.shape[1]] = q.view(torch.uint8)
    return wide.view(q.dtype)[:, : q.shape[1]]


def prepare(case, seed):
    d = _inputs(case, seed)
    op = case["op"]
    e4m3 = torch.float8_e4m3fn
    s = {"op": op, "out": _TYPES[case["out"]], "p": case["p"], "fmt": _TYPES[case["fmt"]], "both": case["both"],
         "key": d["key"], "offset": d["offset"]}
    if op in ("checkpoint", "dropout", "step"):
        s["X"] = d["X"]
    if op == "dropout":
        s["R"], s["dY"] = d["R"], d["dY"]
        s["X"].requires_grad_(True)
    if op == "step":
        s["W"], s["mask"], s["dY"] = d["W"], d["mask"], d["dY"]
        s["X"].requires_grad_(True)
        s["W"].requires_grad_(True)
    if op in ("linear", "backward"):
        # the layer's codes, laid out once, and the activations' as the forward pass left them
        q, scale = _codes(d["W"].float(), e4m3, BLOCK, BLOCK)
        s["w"] = _stored(q), scale
        X = d["X"].float()
        if op == "linear":
            q, scale = _codes(X, e4m3)
            s["x"] = _stored(q), scale
        else:
            q, scale = _codes(d["W"].float().t().contiguous(), e4m3, BLOCK, BLOCK)
            s["wt"] = _stored(q), scale
            if case["p"] != 0.0:
                X = _drop(X, _keep(case["T"], case["n"], d, case["p"]), case["p"])
            q, scale = _codes(X.t().contiguous(), e4m3)
            s["xt"] = _stored(q), scale
            s["mask"], s["dY"] = d["mask"], d["dY"]
    if own:
        # the handles that the package's calls take
        import post_pruning_amd as sg
        s["drop"] = sg.Dropout(case["p"], d["key"], d["offset"]) if case["p"] != 0.0 else None
        for k in ("x", "xt"):
            if k in s:
                s[k] = sg.F8Tensor(*s[k])
        if "w" in s:
            s["layer"] = sg.F8Layer(sg.F8Tensor(*s["w"]), sg.F8Tensor(*s["wt"]) if "wt" in s else None)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    import post_pruning_amd as sg
    op = s["op"]
    if op == "checkpoint":
        if not s["both"]:
            q = sg.sg_quantize_f8(s["X"], dtype=s["fmt"], drop=s["drop"])
            return sg.sg_dequantize_f8(q, dtype=s["out"]), q.scale
        q, qt = sg.sg_quantize_f8(s["X"], dtype=s["fmt"], form="both", drop=s["drop"])
        return sg.sg_dequantize_f8(q, dtype=s["out"]), q.scale, sg.sg_dequantize_f8(qt, dtype=s["out"]), qt.scale
    if op == "linear":
        return sg.sg_linear_f8(s["x"], s["layer"], dtype=s["out"])
    if op == "backward":
        dy, dyt = sg.sg_quantize_f8(s["dY"], dtype=s["fmt"], form="both")
        return (sg.sg_linear_f8_grad_input(dy, s["layer"], dtype=s["out"], drop=s["drop"]),
                sg.sg_linear_f8_grad_weight(dyt, s["xt"], mask=s["mask"], dtype=s["out"]))
    if op == "dropout":
        Y = sg.dropout(s["X"], s["drop"], residual=s["R"])
        return Y.detach(), torch.autograd.grad(Y, s["X"], s["dY"])[0]
    Y = sg.linear_f8(s["X"], s["W"], mask=s["mask"], drop=s["drop"], grad_dtype=s["fmt"])
    dX, dW = torch.autograd.grad(Y, (s["X"], s["W"]), s["dY"])
    return Y.detach(), dX, dW


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "checkpoint":
        return _plain_checkpoint(_dropped(s), s)
    if op == "linear":
        return (_values(*s["x"]) @ _values(*s["w"]).t()).to(s["out"])
    if op == "backward":
        return _plain_backward(_values(*s["w"]), _values(*s["xt"]), s)
    if op == "dropout":
        keep = _keep(*s["X"].shape, s, s["p"])
        Y = _drop(s["X"].detach(), keep, s["p"])
        if s["R"] is not None:
            Y = Y + s["R"].float()
        return Y.to(s["out"]), _drop(s["dY"], keep, s["p"]).to(s["out"])
    X = _dropped(s)
    w_hat = _values(*_codes(s["W"].detach().float(), torch.float8_e4m3fn, BLOCK, BLOCK))
    Y = _values(*_codes(X, torch.float8_e4m3fn)) @ w_hat.t()
    xt_hat = _values(*_codes(X.t().contiguous(), torch.float8_e4m3fn))
    return (Y.to(s["out"]), *_plain_backward(w_hat, xt_hat, s))


def work(case):
    T, n, m, e, i = case["T"], case["n"], case["m"], _SIZE[case["out"]], _SIZE[case["x"]]
    mul = 2.0 * T * n * m
    op = case["op"]
    if op == "checkpoint":
        # each form: codes written and read, the values written, a scale for every block
        form = T * n * (2 + e) + T * n // 64
        return {"bytes": T * n * i + form * (2 if case["both"] else 1), "flops": 0}
    if op == "linear":
        return {"bytes": (T * n + m * n) * 129 // 128 + T * m * e, "flops": mul}
    if op == "backward":
        return {"bytes": 2 * T * m + (T * n + m * n) * 129 // 128 + m * n + (T * n + m * n) * e, "flops": 2 * mul}
    if op == "dropout":
        return {"bytes": T * n * i * (5 if case["residual"] else 4), "flops": 0}
    return {"bytes": 2 * T * n + 3 * m * n + 2 * T * m + (T * m + T * n + m * n) * e, "flops": 3 * mul}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------
def _exact_hat(X, fmt, rows=1):
    """(values, scale bytes) of a float64 X from the formats' definition: blocks of rows x 128."""
    power = torch.tensor([2.0**k for k in range(-300, 301)], dtype=torch.float64).cuda()

    def two(k):  # exactly
        return power[k.long() + 300]

    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)  # fraction bits, least exponent
    top = 448.0 if fmt == "e4m3" else 57344.0
    h, w = X.shape
    wide = torch.zeros((h + rows - 1) // rows * rows, (w + 127) // 128 * 128, dtype=torch.float64, device="cuda")
    wide[:h, :w] = X
    tiles = wide.unfold(0, rows, rows).unfold(1, 128, 128).abs().flatten(2).max(2).values
    # the logarithm finds the exponent up to one; comparing puts it right
    e = torch.ceil(torch.log2(torch.where(tiles > 0, tiles, top) / top))
    e = torch.where(two(e) * top < tiles, e + 1, e)
    e = torch.where((two(e - 1) * top >= tiles) & (tiles > 0), e - 1, e).clamp(min=-127)
    unit = two(e).repeat_interleave(rows, 0)[:h].repeat_interleave(128, 1)[:, :w]
    x = X / unit
    mag = x.abs()
    step = two(torch.floor(torch.log2(torch.where(mag > 0, mag, 1.0))).clamp(min=low) - bits)
    return torch.round(x / step) * step * unit, (e + 127).to(torch.uint8).repeat_interleave(rows, 0)[:h].t().contiguous()


def _exact_keep(T, n, key, offset, p):
    """The kept elements, with 32-bit products taken in 16-bit parts."""
    def product(x, k):
        x0, x1, k0, k1 = x & 0xFFFF, x >> 16, k & 0xFFFF, k >> 16
        mid = x1 * k0 + ((x0 * k0) >> 16)
        rest = x0 * k1 + (mid & 0xFFFF)
        return x1 * k1 + (mid >> 16) + (rest >> 16), ((rest & 0xFFFF) << 16) | ((x0 * k0) & 0xFFFF)

    at = torch.arange(T * ((n + 3) // 4), device="cuda")
    x = [at % ((n + 3) // 4), at // ((n + 3) // 4), torch.zeros_like(at) + offset % 2**32, torch.zeros_like(at) + offset // 2**32]
    for i in range(10):
        hi, lo = product(x[0], 0xD2511F53)
        hi2, lo2 = product(x[2], 0xCD9E8D57)
        x = [hi2 ^ x[1] ^ ((key % 2**32 + i * 0x9E3779B9) % 2**32), lo2,
             hi ^ x[3] ^ ((key // 2**32 + i * 0xBB67AE85) % 2**32), lo]
    words = torch.empty(at.numel(), 4, dtype=torch.int64, device="cuda")
    for i in range(4):
        words[:, i] = x[i]
    return words.view(T, -1)[:, :n] >= int(round(p * 4294967296.0))


def exact(case, seed):
    """The same outputs from the definition, in 64 bits."""
    d = _inputs(case, seed)
    f64 = torch.float64
    T, n, p, op = case["T"], case["n"], case["p"], case["op"]
    grow = float(torch.tensor(1.0 / (1.0 - p), dtype=torch.float32)) if p else 1.0
    keep = _exact_keep(T, n, d["key"], d["offset"], p) if p else None
    X = d["X"].to(f64)
    if op == "dropout":
        Y = torch.where(keep, X * grow, torch.zeros_like(X))
        G = d["dY"].to(f64) * grow
        return (Y if d["R"] is None else Y + d["R"].to(f64)), torch.where(keep, G, torch.zeros_like(G))
    if p:
        # what is quantized is the fp32 value: this rounding is part of the definition
        X = (X * grow).float().to(f64).masked_fill(~keep, 0.0)
    if op == "checkpoint":
        got = _exact_hat(X, case["fmt"])
        return got + _exact_hat(X.T, case["fmt"]) if case["both"] else got
    w = _exact_hat(d["W"].to(f64), "e4m3", 128)[0]
    got = []
    if op != "backward":
        got.append(torch.matmul(_exact_hat(X, "e4m3")[0], w.T))
    if op != "linear":
        grad = d["dY"].to(f64)
        dX = torch.matmul(_exact_hat(grad, case["fmt"])[0], w) * grow
        got.append(dX if keep is None else dX.masked_fill(~keep, 0.0))
        full = torch.matmul(_exact_hat(grad.T, case["fmt"])[0], _exact_hat(X.T, "e4m3")[0].T)
        got.append(full.masked_fill(d["mask"] != 0, 0.0))
    return got[0] if len(got) == 1 else tuple(got)
