"""The linear layer in 8-bit floating point on the GPU, against 64-bit
implementations of its formulas.

Codes are compared exactly.  Products of small whole numbers (codes of -8 .. 8,
scales of 1/2, 1 and 2) have to be equal: eight products of a block differ by
less than 2^13, so that not even the matrix instruction's alignment cuts
anything, and all partial sums are fp32 numbers.

Tolerances of other products: with K products a sum in fp32 is off by at most
K 2^-24 of the sum of their magnitudes (a generous bound for any order), a bf16
result by another 2^-8 of its value, and in bf16 outputs every eight products by
8 * 2^-12 of the largest of them (what lies 2^-13 below it, an exponent of
slack for its significand, is dropped)."""

import numpy as np
import pytest
import torch

import post_pruning_amd as sg
from oracle import float8

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
NAME = {E4: "e4m3", E5: "e5m2"}


def _dev(t):
    return torch.as_tensor(t).cuda()


def _codes(t):
    return t.codes.view(torch.uint8).cpu().numpy()


def _check(q, x, fmt, rows=1):
    """The F8Tensor q against the float64 matrix x."""
    codes, scale = float8.quantize(x, NAME[fmt], rows)
    assert (q.scale.cpu().numpy() == scale).all()
    got, want = _codes(q), codes
    nan = (want & 0x7F) == 0x7F
    assert (got[~nan] == want[~nan]).all()
    assert ((got[nan] & 0x7F) == 0x7F).all()
    wide = q._wide()[0].view(torch.uint8).cpu().numpy()
    assert (wide[:, q.cols:] == 0).all()


def _input(T, n, seed=0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, n, generator=g) * torch.exp(2 * torch.randn(T, n, generator=g))
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 4096), (3, 127), (2, 129), (128, 128), (129, 300), (17, 1001), (300, 136)])
def test_quantize(T, n, fmt, dtype):
    X = _input(T, n, T + n, dtype)
    x = X.double().numpy()
    _check(sg.sg_quantize_f8(X.cuda(), fmt), x, fmt)
    _check(sg.sg_quantize_f8(X.cuda(), fmt, form="columns"), x.T, fmt)
    q, qt = sg.sg_quantize_f8(X.cuda(), fmt, form="both")
    _check(q, x, fmt)
    _check(qt, x.T, fmt)
    for t, want in ((q, x), (qt, x.T)):
        v = float8.values(*float8.quantize(want, NAME[fmt]), NAME[fmt])
        assert (sg.sg_dequantize_f8(t, torch.float32).double().cpu().numpy() == v).all()
        assert (sg.sg_dequantize_f8(t).double().cpu().numpy() == v).all()  # bf16 holds every value


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("offset,pitch", [(0, 304), (1, 301), (8, 320), (3, 300)])
def test_quantize_strides(offset, pitch, fmt):
    store = _input(140, pitch, 5).reshape(-1)
    store = torch.cat([store, store[:16]]).cuda()
    X = torch.as_strided(store, (140, 297), (pitch, 1), offset)
    q, qt = sg.sg_quantize_f8(X, fmt, form="both")
    _check(q, X.double().cpu().numpy(), fmt)
    _check(qt, X.double().cpu().numpy().T, fmt)
    out = torch.full((140, 333), 7.0, device="cuda")
    sg.sg_dequantize_f8(q, torch.float32, X_out=out[:, 5:302])
    assert (out[:, :5] == 7).all() and (out[:, 302:] == 7).all()
    assert (out[:, 5:302] == sg.sg_dequantize_f8(q, torch.float32)).all()


@pytest.mark.parametrize("fmt", [E4, E5])
def test_quantize_extremes(fmt):
    x = torch.zeros(130, 256)
    x[0, :4] = torch.tensor([1e-45, -3e-45, 1e-40, 0.0])          # a block of subnormal numbers
    x[1, :3] = torch.tensor([2.0 ** 127, -(2.0 ** 126), 1.0])      # next to the end of the range
    x[2, 5], x[3, 200], x[4, 7] = float("nan"), float("inf"), -float("inf")
    x[5, :3] = torch.tensor([-0.0, 1.75, -1.75])
    x[6, :2] = torch.tensor([1.7500001, 2.0 ** -20])
    x[7, 3] = 2.0 ** -118
    x[129] = 3.0
    for X in (x, x[:, :200], x[:130, :131]):
        d = X.double().numpy()
        q, qt = sg.sg_quantize_f8(X.contiguous().cuda(), fmt, form="both")
        _check(q, d, fmt)
        _check(qt, d.T, fmt)
        _check(sg.sg_quantize_f8(X.contiguous().cuda(), fmt), d, fmt)


@pytest.mark.parametrize("T,n", [(5, 200), (130, 133), (300, 64)])
@pytest.mark.parametrize("form", ["rows", "columns", "both"])
def test_quantize_after_dropout(T, n, form):
    X = _input(T, n, 3, torch.bfloat16)
    X[1, 2] = float("nan")
    kept = float8.keep(T, n, 0.3, 99, 1 << 40)
    kept[1, 2] = False
    seed = next(s for s in range(99, 400) if not float8.keep(2, 4, 0.3, s, 1 << 40)[1, 2])
    kept = float8.keep(T, n, 0.3, seed, 1 << 40)
    x = float8.drop(X.double().numpy(), kept, 0.3)  # the dropped NaN is a zero
    assert np.isfinite(x).all()
    got = sg.sg_quantize_f8(X.cuda(), form=form, drop=sg.Dropout(0.3, seed, 1 << 40))
    got = got if form == "both" else (got, got)
    if form != "columns":
        _check(got[0], x, E4)
    if form != "rows":
        _check(got[1], x.T, E4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(1, 1), (128, 256), (130, 127), (257, 300), (64, 1001)])
def test_pack(m, n, dtype):
    W = _input(m, n, 8, dtype)
    W[W.abs() < 0.3] = 0
    layer = sg.sg_pack_f8(W.cuda())
    w = W.double().numpy()
    _check(layer.w, w, E4, rows=128)
    _check(layer.wt, w.T, E4, rows=128)
    v = sg.sg_dequantize_f8(layer.w, torch.float32)
    assert (sg.sg_dequantize_f8(layer.wt, torch.float32).t() == v).all()
    assert (v[W.cuda() == 0] == 0).all()
    alone = sg.sg_pack_f8(W.cuda(), transposed=False)
    assert alone.wt is None and (_codes(alone.w) == _codes(layer.w)).all()


def test_rows_behind_the_last_are_left():
    store = torch.full((300, 256), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((2, 304), 0x66, dtype=torch.uint8, device="cuda")
    q = sg.F8Tensor._of(store.view(E4)[:37], scale[:, :48], 37, 256)
    X = _input(37, 256, 2).cuda()
    sg.sg_quantize_f8(X, q=q)
    assert (store[37:] == 0x55).all() and (scale[:, 37:] == 0x66).all()
    _check(q, X.double().cpu().numpy(), E4)
    qt = sg.F8Tensor._of(store.view(E4)[:256, :128], scale[:1], 256, 37)
    store.fill_(0x55), scale.fill_(0x66)
    sg.sg_quantize_f8(X, form="columns", qt=qt)
    assert (store[256:] == 0x55).all() and (store[:, 128:] == 0x55).all() and (scale[:, 256:] == 0x66).all()


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------
def _whole(rows, cols, fmt, seed):
    """An F8Tensor of small whole numbers times 1/2, 1 or 2, and its values in float64."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-8, 9, (rows, cols), generator=g, device="cuda").float()
    e = torch.randint(126, 129, (-(-cols // 128), rows), generator=g, device="cuda", dtype=torch.uint8)
    unit = torch.ldexp(torch.ones(1, device="cuda", dtype=torch.float64), e.t().to(torch.int32) - 127)
    return sg.F8Tensor(v.to(fmt), e), v.double() * unit.repeat_interleave(128, 1)[:, :cols]


def _layer(m, n, seed):
    w, wv = _whole(m, n, E4, seed)
    # the transposed form is an operand of its own to the library
    wt, wtv = _whole(n, m, E4, seed + 1)
    return sg.F8Layer(w, wt), wv, wtv


# small and odd ones, ones of whole tiles, long contractions with few rows
SHAPES = [(1, 1, 1), (1, 128, 64), (1, 4096, 4096), (2, 130, 70), (16, 1000, 520), (17, 257, 100), (33, 4100, 130),
          (64, 512, 300), (65, 640, 257), (100, 128, 1000), (130, 129, 385), (200, 2000, 200), (257, 1100, 511),
          (300, 1000, 1130), (512, 4096, 768), (515, 300, 2050), (1030, 520, 1300), (2048, 1024, 2048), (4100, 200, 140),
          (2500, 384, 4099)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,m", SHAPES)
def test_linear_whole_numbers(T, n, m, out):
    layer, wv, _ = _layer(m, n, T)
    for fmt in (E4, E5):
        q, xv = _whole(T, n, fmt, n)
        Y = sg.sg_linear_f8(q, layer, dtype=out)
        assert torch.equal(Y, (xv @ wv.t()).to(out))
        assert torch.equal(Y, sg.sg_linear_f8(q, layer, dtype=out))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,m", SHAPES)
def test_grad_input_whole_numbers(T, n, m, out):
    layer, _, wtv = _layer(m, n, T)
    dy, dyv = _whole(T, m, E5 if T % 2 else E4, 7)
    want = dyv @ wtv.t()
    assert torch.equal(sg.sg_linear_f8_grad_input(dy, layer, dtype=out), want.to(out))
    # p = 1/2: the factor is 2, so that dropout stays exact
    drop = sg.Dropout(0.5, 1234567890123456789, 1 << 63)
    kept = sg.sg_dropout(torch.ones(T, n, device="cuda"), drop) == 2
    got = sg.sg_linear_f8_grad_input(dy, layer, dtype=out, drop=drop)
    assert torch.equal(got, torch.where(kept, 2 * want, 0.0).to(out))


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,m", SHAPES)
def test_grad_weight_whole_numbers(T, n, m, out):
    xt, xv = _whole(n, T, E4, 3)
    dyt, dyv = _whole(m, T, E5 if T % 2 else E4, 4)
    want = dyv @ xv.t()
    assert torch.equal(sg.sg_linear_f8_grad_weight(dyt, xt, dtype=out), want.to(out))
    mask = (torch.rand(m, n, device="cuda") < 0.5).to(torch.uint8)
    kept = torch.where(mask.bool(), 0.0, want)
    assert torch.equal(sg.sg_linear_f8_grad_weight(dyt, xt, mask, dtype=out), kept.to(out))
    start = torch.randint(-5, 6, (m, n), device="cuda").to(out)
    start[0, 0], mask[0, 0], kept[0, 0] = -0.0, 1, 0.0
    dW = start.clone()
    sg.sg_linear_f8_grad_weight(dyt, xt, mask, dW=dW, accumulate=True)
    assert torch.equal(dW, (start.double() + kept).to(out))
    assert torch.signbit(dW[0, 0])  # what a pruned weight held stays


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,m,shift,pitch", [(20, 300, 260, 1, 263), (300, 256, 130, 3, 135), (300, 256, 132, 4, 140),
                                               (1, 128, 64, 1, 64), (700, 300, 901, 0, 901)])
def test_outputs_of_any_pitch(T, n, m, shift, pitch, out):
    layer, wv, _ = _layer(m, n, 1)
    q, xv = _whole(T, n, E4, 2)
    store = torch.full((T * pitch + shift + 8,), 9.0, dtype=out, device="cuda")
    Y = torch.as_strided(store, (T, m), (pitch, 1), shift)
    sg.sg_linear_f8(q, layer, Y=Y)
    assert torch.equal(Y, (xv @ wv.t()).to(out))
    inside = torch.zeros_like(store, dtype=torch.bool)
    torch.as_strided(inside, (T, m), (pitch, 1), shift).fill_(True)
    assert (store[~inside] == 9).all()
    # a mask whose rows lie unaligned
    mask = (torch.rand(T * m + 1, device="cuda") < 0.5).to(torch.uint8)[1:].view(T, m)
    a, av = _whole(m, n, E4, 5)
    sg.sg_linear_f8_grad_weight(q, a, mask, dW=Y)
    assert torch.equal(Y, torch.where(mask.bool(), 0.0, xv @ av.t()).to(out))
    assert (store[~inside] == 9).all()


def _groups(a, b):
    """The sum over every eight products of their largest magnitude, for all outputs (small sizes)."""
    K = a.shape[1]
    pad = -K % 8
    a = torch.nn.functional.pad(a.abs(), (0, pad)).view(a.shape[0], 1, -1, 8)
    b = torch.nn.functional.pad(b.abs(), (0, pad)).view(1, b.shape[0], -1, 8)
    return (a * b).amax(3).sum(2)


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("T,n,m", [(1, 700, 100), (40, 1000, 72), (150, 640, 136), (300, 260, 90), (90, 4096, 60)])
def test_linear_of_real_numbers(T, n, m, fmt):
    q = sg.sg_quantize_f8(_input(T, n, 1).cuda(), fmt)
    layer = sg.sg_pack_f8((0.02 * _input(m, n, 2)).cuda())
    x = torch.from_numpy(float8.values(_codes(q), q.scale.cpu().numpy(), NAME[fmt]))
    w = torch.from_numpy(float8.values(_codes(layer.w), layer.w.scale.cpu().numpy()))
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    Y = sg.sg_linear_f8(q, layer, dtype=torch.float32).double().cpu()
    assert ((Y - want).abs() <= n * 2.0 ** -24 * size).all()
    Y = sg.sg_linear_f8(q, layer).double().cpu()
    cut = 8 * 2.0 ** -12 * _groups(x, w)
    assert ((Y - want).abs() <= 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * (cut + n * 2.0 ** -24 * size)).all()


def test_scales_far_apart():
    # products whose scales nearly cancel, and ones far below and above
    T, n, m = 40, 384, 48
    for sx, sw in ((0, 247), (10, 240), (247, 0), (60, 60), (127, 1)):
        q, xv = _whole(T, n, E4, 1)
        w, wv = _whole(m, n, E4, 2)
        q.scale.fill_(sx), w.scale.fill_(sw)
        unit = 2.0 ** (sx + sw - 254)
        a, b = q.codes.double(), w.codes.double()
        want = (a @ b.t()) * unit
        for T0 in (T, 1):
            small = sg.F8Tensor(q.codes[:T0], q.scale[:, :T0])
            Y = sg.sg_linear_f8(small, sg.F8Layer(w), dtype=torch.float32).double()
            # (subnormal results are exact multiples of 2^-149 or rounded to one, once a block)
            assert ((Y - want[:T0]).abs() <= 3 * 2.0 ** -150).all()


def test_what_is_not_finite():
    T, n, m = 150, 300, 200
    X = _input(T, n, 1)
    X[7, 150], X[140, 299] = float("nan"), float("inf")
    W = 0.02 * _input(m, n, 2)
    q, qt = sg.sg_quantize_f8(X.cuda(), form="both")
    for out in (torch.bfloat16, torch.float32):
        Y = sg.sg_linear_f8(q, sg.sg_pack_f8(W.cuda()), dtype=out)
        bad = torch.zeros(T, dtype=torch.bool, device="cuda")
        bad[[7, 140]] = True
        assert torch.isnan(Y[bad]).all() and torch.isfinite(Y[~bad]).all()
        dyt = sg.sg_quantize_f8(_input(T, m, 3).cuda(), form="columns")
        dW = sg.sg_linear_f8_grad_weight(dyt, qt, dtype=out)
        cols = torch.zeros(n, dtype=torch.bool, device="cuda")
        cols[[150, 299]] = True
        assert torch.isnan(dW[:, cols]).all() and torch.isfinite(dW[:, ~cols]).all()
        mask = torch.ones(m, n, dtype=torch.uint8, device="cuda")
        assert (sg.sg_linear_f8_grad_weight(dyt, qt, mask, dtype=out) == 0).all()
    W[130, 299] = float("nan")  # its 128 x 128
    Y = sg.sg_linear_f8(sg.sg_quantize_f8(_input(3, n, 4).cuda()), sg.sg_pack_f8(W.cuda()))
    assert torch.isnan(Y[:, 128:]).all() and torch.isfinite(Y[:, :128]).all()


def test_empty_batch():
    X = torch.zeros(0, 200, device="cuda")
    layer = sg.sg_pack_f8(_input(60, 200, 1).cuda())
    q, qt = sg.sg_quantize_f8(X, form="both")
    assert sg.sg_dequantize_f8(q).shape == (0, 200) and sg.sg_dequantize_f8(qt).shape == (200, 0)
    assert sg.sg_linear_f8(q, layer).shape == (0, 60)
    dy, dyt = sg.sg_quantize_f8(torch.zeros(0, 60, device="cuda"), form="both")
    assert sg.sg_linear_f8_grad_input(dy, layer).shape == (0, 200)
    dW = torch.full((60, 200), 3.0, device="cuda")
    sg.sg_linear_f8_grad_weight(dyt, qt, dW=dW, accumulate=True)
    assert (dW == 3).all()
    sg.sg_linear_f8_grad_weight(dyt, qt, dW=dW)
    assert (dW == 0).all()


# ---------------------------------------------------------------------------
# used together
# ---------------------------------------------------------------------------
def _reference_step(X, W, dY, mask, kept, p, fmt, out):
    """Y, dX, dW in float64 from the formulas."""
    x = X.double().numpy() if kept is None else float8.drop(X.double().numpy(), kept, p)

    def hat(v, f="e4m3", rows=1):
        return torch.from_numpy(float8.values(*float8.quantize(v, f, rows), f))

    w, xh, xth = hat(W.double().numpy(), rows=128), hat(x), hat(x.T)
    g, gt = hat(dY.double().numpy(), NAME[fmt]), hat(dY.double().numpy().T, NAME[fmt])
    dX = g @ w
    if kept is not None:
        dX = torch.where(torch.from_numpy(kept), dX * float(np.float32(1 / (1 - p))), 0.0)
    dW = torch.where(mask.bool().cpu(), 0.0, gt @ xth.t())
    return (xh @ w.t(), xh.abs() @ w.abs().t()), (dX, g.abs() @ w.abs() * 2), (dW, gt.abs() @ xth.abs().t())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p,fmt", [(0.0, E4), (0.4, E5)])
@pytest.mark.parametrize("T,n,m", [(3, 200, 150), (40, 300, 129), (150, 128, 256)])
def test_training_step(T, n, m, p, fmt, dtype):
    X, W, dY = _input(T, n, 1, dtype), 0.02 * _input(m, n, 2), 0.01 * _input(T, m, 3, dtype)
    mask = (W.abs() < 0.02).to(torch.uint8)
    W[mask.bool()] = 0
    drop = sg.Dropout(p, 77, 5) if p else None
    kept = float8.keep(T, n, p, 77, 5) if p else None
    want = _reference_step(X, W, dY, mask, kept, p, fmt, dtype)
    x, w = X.cuda().requires_grad_(True), W.cuda().requires_grad_(True)
    Y = sg.linear_f8(x, w, mask=mask.cuda(), drop=drop, grad_dtype=fmt)
    Y.backward(dY.cuda())
    assert Y.dtype == dtype and x.grad.dtype == dtype and w.grad.dtype == torch.float32
    for got, (ref, size), K in ((Y, want[0], n), (x.grad, want[1], m), (w.grad, want[2], T)):
        eps = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
        cut = 8 * 2.0 ** -12 if got.dtype == torch.bfloat16 else 0.0  # (of sums of magnitudes, above those of the largest)
        off = (got.detach().double().cpu() - ref).abs()
        # (two more roundings where the dropout's factor meets the sum)
        assert (off <= eps * ref.abs() + (1 + eps) * (cut + (K + 2) * 2.0 ** -24) * size).all()
    assert (w.grad[mask.cuda().bool()] == 0).all()


def test_gradients_against_differences():
    # inputs that 8 bits hold exactly, moved by steps that 8 bits hold exactly
    T, n, m = 4, 130, 12
    g = torch.Generator().manual_seed(0)
    X = torch.randint(-3, 4, (T, n), generator=g).float().cuda()
    W = torch.randint(-3, 4, (m, n), generator=g).float().cuda()
    X[:, 0], X[:, 129], W[0, 0], W[0, 129] = 4, 4, 4, 4  # (the blocks' scales stay)
    dY = torch.randint(-3, 4, (T, m), generator=g).float().cuda()
    drop = sg.Dropout(0.5, 3)
    x, w = X.clone().requires_grad_(True), W.clone().requires_grad_(True)
    (sg.linear_f8(x, w, drop=drop) * dY).sum().backward()

    def loss(a, b):
        return float((sg.linear_f8(a, b, drop=drop).double() * dY.double()).sum())

    for t, c in ((0, 5), (1, 17), (3, 128), (2, 60), (1, 3), (0, 101)):
        up, down = X.clone(), X.clone()
        up[t, c] += 1
        down[t, c] -= 1
        assert x.grad[t, c].item() == (loss(up, W) - loss(down, W)) / 2
    for r, c in ((1, 5), (11, 128), (3, 77), (7, 1)):
        up, down = W.clone(), W.clone()
        up[r, c] += 1
        down[r, c] -= 1
        assert w.grad[r, c].item() == (loss(X, up) - loss(X, down)) / 2


def test_linear_f8_forms():
    X = _input(24, 256, 1, torch.bfloat16).cuda()
    W = (0.02 * _input(60, 256, 2)).cuda()
    layer = sg.sg_pack_f8(W)
    Y = sg.linear_f8(X, W)
    assert torch.equal(sg.linear_f8(X, None, layer), Y)
    assert torch.equal(sg.linear_f8(X.view(2, 3, 4, 256), W, layer).view(24, 60), Y)
    assert torch.equal(sg.linear_f8(X.t().contiguous().t(), W), Y)
    assert sg.linear_f8(X[0], W).shape == (60,)
    x = X.clone().requires_grad_(True)
    with pytest.raises(ValueError):
        sg.linear_f8(x, None, sg.sg_pack_f8(W, transposed=False))
    # one gradient alone, an expanded one, a broadcast input
    y = sg.linear_f8(x, W)
    y.sum().backward()
    w = W.clone().requires_grad_(True)
    one = X[:1].clone().requires_grad_(True)
    sg.linear_f8(one.expand(24, 256), w).sum().backward()
    assert one.grad.shape == (1, 256) and w.grad.shape == W.shape
    dy, dyt = sg.sg_quantize_f8(torch.ones(24, 60, device="cuda"), form="both")
    assert torch.equal(x.grad, sg.sg_linear_f8_grad_input(dy, layer))
    assert torch.equal(w.grad, sg.sg_linear_f8_grad_weight(dyt, sg.sg_quantize_f8(X[:1].expand(24, 256).contiguous(), form="columns"),
                                                           dtype=torch.float32))


def test_layer_changed_before_the_backward_pass():
    X = _input(8, 128, 1, torch.bfloat16).cuda().requires_grad_(True)
    W = _input(16, 128, 2).cuda()
    layer = sg.sg_pack_f8(W)
    Y = sg.linear_f8(X, None, layer)
    layer.wt.codes.view(torch.uint8).add_(1)
    with pytest.raises(RuntimeError):
        Y.sum().backward()


def test_checkpoint_as_calibration():
    X = _input(500, 200, 4, torch.bfloat16).cuda()
    W = _input(30, 200, 5).cuda()
    q = sg.sg_quantize_f8(X)
    a = sg.solve_layer(W, [q], 0.5)
    b = sg.solve_layer(W, [sg.sg_dequantize_f8(q)], 0.5)
    assert torch.equal(a["H"], b["H"]) and torch.equal(a["mask"], b["mask"])


def test_another_stream():
    X, W = _input(300, 512, 1, torch.bfloat16).cuda(), (0.02 * _input(256, 512, 2)).cuda()
    want = sg.linear_f8(X, W)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = sg.linear_f8(X, W)
    s.synchronize()
    assert torch.equal(got, want)


def test_captured_training_step():
    T, n, m = 260, 384, 300
    X, W = _input(T, n, 1, torch.bfloat16).cuda(), (0.02 * _input(m, n, 2)).cuda()
    dY = (0.01 * _input(T, m, 3, torch.bfloat16)).cuda()
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    bump = torch.tensor([0, 1], device="cuda")

    def step():
        drop = sg.Dropout(0.25, 11, 4, state)
        q, qt = sg.sg_quantize_f8(X, form="both", drop=drop)
        layer = sg.sg_pack_f8(W)
        Y = sg.sg_linear_f8(q, layer)
        dy, dyt = sg.sg_quantize_f8(dY, form="both")
        return (drop, Y, sg.sg_linear_f8_grad_input(dy, layer, drop=drop), sg.sg_linear_f8_grad_weight(dyt, qt, dtype=torch.float32),
                sg.sg_dropout(Y, drop))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        keep = step()
        state.add_(bump)
    for k in range(3):
        state.copy_(torch.tensor([0, 10 * k], device="cuda"))
        X.copy_(_input(T, n, 10 + k, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        assert state.tolist() == [0, 10 * k + 1]
        got = [t.clone() for t in keep[1:]]
        state.copy_(torch.tensor([0, 10 * k], device="cuda"))
        for a, b in zip(got, step()[1:]):
            assert torch.equal(a, b)


def test_captured_autograd_step():
    T, n, m = 130, 256, 140
    X = _input(T, n, 1, torch.bfloat16).cuda().requires_grad_(True)
    W = (0.02 * _input(m, n, 2)).cuda().requires_grad_(True)
    dY = (0.01 * _input(T, m, 3, torch.bfloat16)).cuda()

    def step():
        Y = sg.linear_f8(X, W, drop=sg.Dropout(0.25, 11))
        Z = sg.dropout(Y, sg.Dropout(0.25, 11, 1), residual=dY)
        return (Z.detach(), *torch.autograd.grad(Z, (X, W), dY))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            a.zero_()
