"""The 8-bit linear layer against plain implementations in 64 bits.

Codes, their sums and the packed bytes are whole numbers and have to be equal.
Tolerances of the rest, with u(t) = finfo(t).eps / 2 for one rounding to t:

  product   the integer sum is exact; int -> fp32 and two fp32 products are
            three roundings, then one to the output type:
            |err| <= (4 u(f32) + u(out)) |y|
  gradients the products are exact in fp32; K additions in fp32, each off by
            at most 2 u(f32) of the running sum (the matrix cores may truncate),
            so |err| <= 2 K u(f32) sum |a b|, then one rounding to the output
            type, u(out) |ref|.
"""

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

U32 = torch.finfo(torch.float32).eps / 2
U = {torch.float32: U32, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    import post_pruning_amd as sg
    sg.load_library()
    assert torch.cuda.is_available()
    return sg


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _x(T, n, dtype, seed, pitch=None, shift=0):
    """A [T, n] GPU tensor whose rows lie `pitch` elements apart and start
    `shift` elements into the storage; everything around it is NaN."""
    g = _gen(seed)
    v = torch.randn(T, n, generator=g) * torch.exp(0.5 * torch.randn(n, generator=g))
    pitch = pitch or n
    store = torch.full((shift + T * pitch + 8,), float("nan"), dtype=dtype, device="cuda")
    x = store[shift:shift + T * pitch].view(T, pitch)[:, :n]
    x.copy_(v.to(dtype))
    return x


def _layer(sg, m, n, seed, bits=8, pruned=0.5):
    g = _gen(seed)
    W = 0.02 * torch.randn(m, n, generator=g)
    top = 2 ** bits - 1
    lo, hi = W.amin(1).clamp(max=0.0), W.amax(1).clamp(min=0.0)
    scale = (hi - lo) / top
    zero = torch.round(-lo / scale)
    mask = torch.rand(m, n, generator=g) < pruned
    if m > 2:
        mask[1] = True  # a row with nothing left
    codes = torch.clamp(torch.round(W / scale[:, None]) + zero[:, None], 0, top)
    codes = torch.where(mask, zero[:, None].expand(m, n), codes).to(torch.uint8)
    d = {"codes": codes, "scale": scale, "zero": zero, "mask": mask.to(torch.uint8)}
    d["w"] = (codes.double() - zero.double()[:, None])  # whole numbers
    d["w_hat"] = (d["w"].float() * scale[:, None])       # fp32
    d["packed"] = sg.sg_pack_w8(codes.cuda(), scale.cuda(), zero.cuda())
    return d


def _codes_ref(X):
    """Exact codes: 254 |x| and (2k + 1) a are compared as whole numbers."""
    x = X.double().cpu().numpy()
    a = np.abs(x).max(axis=1)
    d = np.where(a > 0, a, 1.0)
    # the quotient of the exact 127 x by a in 64 bits is off by 2^-53, far
    # less than the distance of a 24-bit quotient from a half it does not hit
    q = np.rint(127.0 * x / d[:, None])
    s = np.where(a > 0, (a / 127.0).astype(np.float32), np.float32(1.0)).astype(np.float32)
    return q.astype(np.int64), s


QSHAPES = [(1, 1), (3, 7), (5, 63), (4, 64), (4, 65), (3, 1000), (9, 1024), (6, 1025), (130, 384), (3, 4096),
           (5, 8192), (2, 8193), (2, 28672), (1, 32769), (2, 65536), (131, 1000), (129, 1032), (200, 8192), (140, 8200)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,n", QSHAPES)
def test_quantize_and_read_back(sg, T, n, dtype):
    for pitch, shift in ((n, 0), (n + 3, 1), (-(-n // 8) * 8 + 8, 0)):
        X = _x(T, n, dtype, 10 * n + T, pitch, shift)
        q, s, total = sg.sg_quantize_tokens(X)
        qr, sr = _codes_ref(X)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), qr)
        assert np.array_equal(s.cpu().numpy(), sr)
        assert np.array_equal(total.cpu().numpy().astype(np.int64), qr.sum(1))
        # the padding of the rows is zero
        wide = torch.as_strided(q, (T, q.stride(0)), (q.stride(0), 1))
        assert not wide[:, n:].any()
        for out in (BF16, F32):
            back = sg.sg_dequantize_tokens(q, s, dtype=out)
            want = (q.float().cpu() * s.cpu()[:, None]).to(out)
            assert torch.equal(back.cpu(), want)
        # no value is further from its code than half a step
        err = (back.double().cpu() - X.double().cpu()).abs().amax(1)
        assert (err <= (0.5 + 1e-5) * s.double().cpu()).all()


def test_quantize_halves_and_borders(sg):
    # a peak of 127 makes the scale 1: values k + 1/2 are exact halves
    k = torch.arange(-126, 126).float() + 0.5
    row = torch.cat([torch.tensor([127.0]), k])
    q, s, _ = sg.sg_quantize_tokens(torch.stack([row, -row]).cuda())
    assert s.tolist() == [1.0, 1.0]
    assert torch.equal(q[0].cpu().float(), torch.round(row))  # halves to even
    assert torch.equal(q[1].cpu().float(), torch.round(-row))
    # fp32 neighbours of every border, for peaks of many significands
    rng = np.random.default_rng(3)
    rows = []
    for a in np.concatenate([rng.uniform(0.5, 2.0, 40), [1.0, 1.5, 126.99999, 1e-30, 3e38]]).astype(np.float32):
        b = ((np.arange(0, 127) + 0.5) * np.float64(a) / 127.0).astype(np.float32)
        near = np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(np.inf))])
        near = np.minimum(near, a)
        sign = rng.choice([-1.0, 1.0], near.size).astype(np.float32)
        rows.append(np.concatenate([[a], near * sign]).astype(np.float32))
    X = torch.from_numpy(np.stack(rows)).cuda()
    q, s, _ = sg.sg_quantize_tokens(X)
    # exact decision in whole numbers
    from fractions import Fraction
    for i, r in enumerate(rows):
        a = Fraction(float(r[0]))
        want = [int(round(Fraction(float(v)) * 127 / a)) for v in r]  # round() of a Fraction: halves to even
        assert q[i].tolist() == want, i


def test_quantize_extreme_rows(sg):
    n = 70
    X = torch.randn(9, n, generator=_gen(4))
    X[0] = 0.0
    X[1] = -0.0
    X[2, 5] = float("nan")
    X[3, 69] = float("inf")
    X[4, 0] = -float("inf")
    X[5] *= 1e-42   # subnormal
    X[6] = 0.0
    X[6, 3] = 1e-45  # the smallest number: its scale rounds to 0
    X[7] *= 5e37
    X[8] *= 1e-37
    q, s, total = sg.sg_quantize_tokens(X.cuda())
    qc, sc = q.cpu(), s.cpu()
    for r in (0, 1):
        assert not qc[r].any() and sc[r] == 1.0 and total[r] == 0
    for r in (2, 3, 4):
        assert not qc[r].any() and torch.isnan(sc[r]) and total[r] == 0
    assert qc[6].tolist() == [0, 0, 0, 127] + [0] * 66 and sc[6] == 0.0
    for r in (5, 7, 8):
        qr, sr = _codes_ref(X[r:r + 1])
        assert np.array_equal(qc[r].numpy(), qr[0]) and sc[r].item() == sr[0]
    back = sg.sg_dequantize_tokens(q, s, dtype=F32).cpu()
    assert torch.isnan(back[2:5]).all() and torch.isfinite(back[[0, 1, 5, 6, 7, 8]]).all()
    ok = [0, 1, 5, 6, 7, 8]
    assert torch.equal(back[ok], (qc.float() * sc[:, None])[ok])
    assert torch.equal(sg.sg_dequantize_tokens(q, s).cpu()[ok], (qc.float() * sc[:, None]).to(BF16)[ok])
    # the product of such a token is NaN, the other tokens' are untouched
    L = _layer(sg, 5, n, 5)
    Y = sg.sg_linear_w8a8(q, s, total, L["packed"], dtype=F32).cpu()
    assert torch.isnan(Y[2:5]).all() and torch.isfinite(Y[[0, 1, 5, 6, 7, 8]]).all()


@pytest.mark.parametrize("m,n", [(1, 1), (3, 5), (7, 64), (5, 1003), (70, 4096)])
def test_pack(sg, m, n):
    g = _gen(m + n)
    codes = torch.randint(0, 256, (m, n), generator=g, dtype=torch.uint8)
    scale, zero = torch.rand(m, generator=g), torch.randint(0, 256, (m,), generator=g).float()
    p = sg.sg_pack_w8(codes.cuda(), scale.cuda(), zero.cuda())
    assert torch.equal(p.codes.cpu().int(), codes.int() - 128)
    assert torch.equal(p.offset.cpu(), 128 - zero.int())
    assert torch.equal(p.scale.cpu(), scale)
    wide = torch.as_strided(p.codes, (m, p.codes.stride(0)), (p.codes.stride(0), 1))
    assert not wide[:, n:].any()


def test_pack_marks_bad_zero_points(sg):
    zero = torch.tensor([0.0, 255.0, -1.0, 256.0, 3.5, float("nan"), float("inf")])
    p = sg.sg_pack_w8(torch.zeros(7, 16, dtype=torch.uint8).cuda(), torch.ones(7).cuda(), zero.cuda())
    assert torch.isnan(p.scale.cpu()).tolist() == [False, False, True, True, True, True, True]


def _linear_ref(q, s, L):
    """The exact integer sums and the product in 64 bits."""
    acc = q.double().cpu() @ L["w"].t()  # whole numbers below 2^53
    return acc * s.double().cpu()[:, None] * L["scale"].double()[None, :]


def _check_linear(sg, T, n, m, out, bits=8, seed=0, pruned=0.5):
    L = _layer(sg, m, n, seed + 1, bits, pruned)
    q, s, total = sg.sg_quantize_tokens(_x(T, n, BF16, seed + 2))
    # outputs in the middle of a larger buffer that has to stay as it is
    store = torch.full((T + 2, m + 5), 7.0, dtype=out, device="cuda")
    Y = store[1:T + 1, 2:m + 2]
    got = sg.sg_linear_w8a8(q, s, total, L["packed"], Y=Y)
    assert got.data_ptr() == Y.data_ptr()
    ref = _linear_ref(q, s, L)
    err = (Y.double().cpu() - ref).abs()
    assert (err <= (4 * U32 + U[out]) * ref.abs()).all(), float((err / ref.abs().clamp(min=1e-30)).max())
    store[1:T + 1, 2:m + 2] = 7.0
    assert (store == 7.0).all()
    again = sg.sg_linear_w8a8(q, s, total, L["packed"], dtype=out)
    first = sg.sg_linear_w8a8(q, s, total, L["packed"], dtype=out)
    assert torch.equal(again, first)
    assert (again.double().cpu() - ref).abs().le((4 * U32 + U[out]) * ref.abs()).all()


LSHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 64, 16), (3, 65, 17), (16, 1000, 130), (17, 1000, 130), (33, 130, 1),
           (64, 4096, 48), (65, 200, 1000), (127, 192, 257), (128, 128, 128), (129, 127, 129), (300, 1000, 1130),
           (257, 4096, 513), (512, 576, 256), (515, 3000, 770), (1, 65536, 33), (40, 28672, 100), (1030, 64, 1300)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,n,m", LSHAPES)
def test_linear(sg, T, n, m, out):
    _check_linear(sg, T, n, m, out, seed=T + n + m)


@pytest.mark.parametrize("bits,pruned", [(2, 0.0), (3, 0.9), (4, 0.5), (8, 1.0)])
def test_linear_bits_and_pruned(sg, bits, pruned):
    _check_linear(sg, 70, 520, 140, F32, bits, 50 + bits, pruned)


def test_linear_largest_sums(sg):
    # every code at its limit: |sum| = 65536 * 127 * 255, just inside 32 bits
    n = 65536
    X = torch.ones(3, n, device="cuda")
    X[1] = -1.0
    q, s, total = sg.sg_quantize_tokens(X)
    assert (q[0] == 127).all() and (q[1] == -127).all()
    codes = torch.full((4, n), 255, dtype=torch.uint8, device="cuda")
    codes[1] = 0
    codes[3] = 0
    zero = torch.tensor([0.0, 255.0, 255.0, 0.0], device="cuda")
    L = sg.sg_pack_w8(codes, torch.ones(4, device="cuda"), zero)
    for T in (3, 2):
        Y = sg.sg_linear_w8a8(q[:T], s[:T], total[:T], L, dtype=F32).double().cpu()
        top = float(n * 127 * 255) * float(s[0])
        want = torch.tensor([[top, -top, 0, 0], [-top, top, 0, 0], [top, -top, 0, 0]], dtype=torch.float64)[:T]
        assert ((Y - want).abs() <= 4 * U32 * want.abs()).all()


def test_codes_beside_the_layer_do_not_count(sg):
    # a column slice of wider codes: what lies behind column n is not read as data
    T, n, m = 5, 100, 20
    wide = torch.randint(-127, 128, (T, 256), generator=_gen(8), dtype=torch.int8).cuda()
    q = wide[:, :n]
    s = torch.rand(T, generator=_gen(9)).cuda()
    L = _layer(sg, m, n, 10)
    Y = sg.sg_linear_w8a8(q, s, q.int().sum(1).int(), L["packed"], dtype=F32)
    ref = _linear_ref(q, s, L)
    assert ((Y.double().cpu() - ref).abs() <= 4 * U32 * ref.abs()).all()


def _dy(T, m, seed, pitch=None, shift=0):
    return _x(T, m, BF16, seed, pitch, shift)


def _close_sum(got, ref, mag, K, out):
    tol = 2 * K * U32 * mag + U[out] * ref.abs() * (1 + 2 * K * U32) + U[out] * 2 * K * U32 * mag
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-300)).max())


GSHAPES = [(1, 1, 1), (1, 4096, 300), (2, 64, 32), (3, 65, 33), (16, 1000, 130), (64, 130, 200), (129, 1000, 2050),
           (130, 384, 96), (200, 72, 264), (256, 256, 256), (515, 1000, 770), (1024, 200, 40), (300, 28672, 24),
           (257, 513, 129)]


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,n,m", GSHAPES)
def test_grad_input(sg, T, n, m, out):
    L = _layer(sg, m, n, T + n + m)
    w = L["w_hat"].to(BF16).double()
    for pitch, shift in ((m, 0), (m + 5, 3)):
        dY = _dy(T, m, 3 * T + m, pitch, shift)
        store = torch.full((T + 2, n + 7), 7.0, dtype=out, device="cuda")
        dX = store[1:T + 1, 3:n + 3]
        sg.sg_linear_w8_grad_input(dY, L["packed"], dX=dX)
        g = dY.double().cpu()
        _close_sum(dX, g @ w, g.abs() @ w.abs(), m, out)
        store[1:T + 1, 3:n + 3] = 7.0
        assert (store == 7.0).all()
    a = sg.sg_linear_w8_grad_input(dY, L["packed"], dtype=out)
    b = sg.sg_linear_w8_grad_input(dY.clone(), L["packed"], dtype=out)
    assert torch.equal(a, b)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,n,m", GSHAPES)
def test_grad_weight(sg, T, n, m, out):
    L = _layer(sg, m, n, T + n + m)
    mask = L["mask"].cuda()
    q, s, _ = sg.sg_quantize_tokens(_x(T, n, BF16, T + 7))
    x = sg.sg_dequantize_tokens(q, s).double().cpu()
    for pitch, shift in ((m, 0), (m + 5, 3)):
        dY = _dy(T, m, 3 * T + m, pitch, shift)
        g = dY.double().cpu()
        full, mag = g.t() @ x, g.abs().t() @ x.abs()
        kept = (L["mask"] == 0).double()
        store = torch.full((m + 2, n + 7), 7.0, dtype=out, device="cuda")
        dW = store[1:m + 1, 3:n + 3]
        sg.sg_linear_w8_grad_weight(dY, q, s, mask, dW=dW)
        _close_sum(dW, full * kept, mag * kept, T, out)
        assert not dW[mask != 0].any()
        store[1:m + 1, 3:n + 3] = 7.0
        assert (store == 7.0).all()
    _close_sum(sg.sg_linear_w8_grad_weight(dY, q, s, dtype=out), full, mag, T, out)  # no mask
    a = sg.sg_linear_w8_grad_weight(dY, q, s, mask, dtype=out)
    b = sg.sg_linear_w8_grad_weight(dY.clone(), q, s, mask, dtype=out)
    assert torch.equal(a, b)
    # adding to what is there: one more rounding of the sum
    base = torch.randn(m, n, generator=_gen(6)).to(out).cuda()
    acc = base.clone()
    sg.sg_linear_w8_grad_weight(dY, q, s, mask, dW=acc, accumulate=True)
    assert torch.equal(acc[mask != 0], base[mask != 0])
    ref = full * kept + base.double().cpu()
    tol = 2 * T * U32 * mag * kept + (U32 + U[out]) * (ref.abs() + 2 * T * U32 * mag)
    assert ((acc.double().cpu() - ref).abs() <= tol).all()


# Outputs whose rows (and the mask's) lie on every alignment, in tiles whose
# contraction is whole and in tiles that are joined.
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("T,m", [(70, 300), (9000, 70)])
@pytest.mark.parametrize("n,extra,shift", [(144, 0, 0), (136, 0, 0), (132, 0, 0), (132, 4, 4), (132, 4, 2), (132, 2, 0),
                                           (130, 0, 0), (129, 0, 1), (128, 0, 4), (128, 0, 2), (130, 6, 0), (131, 1, 0)])
def test_rows_of_every_alignment(sg, T, m, n, extra, shift, out):
    pitch = n + extra
    mask = (torch.rand(m, n, generator=_gen(n + T)) < 0.5).to(torch.uint8)
    q, s, _ = sg.sg_quantize_tokens(_x(T, n, BF16, T + 7))
    x = sg.sg_dequantize_tokens(q, s).double().cpu()
    dY = _dy(T, m, 3 * T + m)
    g = dY.double().cpu()
    kept = (mask == 0).double()
    full, mag = (g.t() @ x) * kept, (g.abs().t() @ x.abs()) * kept
    base = torch.randn(m, n, generator=_gen(6)).to(out)
    for add in (False, True):
        store = torch.full((shift + (m + 1) * pitch,), 7.0, dtype=out, device="cuda")
        dW = store[shift:shift + m * pitch].view(m, pitch)[:, :n]
        dW.copy_(base)
        sg.sg_linear_w8_grad_weight(dY, q, s, mask.cuda(), dW=dW, accumulate=add)
        if add:
            assert torch.equal(dW.cpu()[mask != 0], base[mask != 0])
            ref = full + base.double()
            tol = 2 * T * U32 * mag + (U32 + U[out]) * (ref.abs() + 2 * T * U32 * mag)
            assert ((dW.double().cpu() - ref).abs() <= tol).all()
        else:
            _close_sum(dW, full, mag, T, out)
            assert not dW.cpu()[mask != 0].any()
        dW.fill_(7.0)
        assert (store == 7.0).all()


# Odd shapes that between them reach every tile of the library, with its
# contraction whole and divided over workgroups.
TILES = {
    "product": [(33000, 33, 33), (70, 33, 33000), (70, 33000, 4100), (70, 33, 8200), (33, 8200, 4100), (70, 33, 33),
                (70, 4100, 33), (70, 28672, 300), (300, 130, 9000), (2303, 200, 2001), (3301, 100, 3295), (5, 130, 131077)],
    "input": [(130, 33000, 33), (203, 8200, 20001), (20001, 130, 70), (4100, 203, 8200), (8200, 70, 770),
              (2050, 70, 4100), (33, 33, 770), (33, 33, 2600), (70, 20001, 33), (70, 2050, 4100), (70, 8200, 33),
              (33, 2050, 4100), (33, 33, 33), (33, 33, 2050), (3301, 3295, 100), (20, 130, 131077)],
    "weight": [(33, 130, 33000), (20001, 203, 8200), (70, 130, 20001), (8200, 203, 4100), (770, 70, 8200),
               (4100, 70, 2050), (770, 33, 33), (2600, 33, 33), (33, 70, 20001), (4100, 2050, 70), (33, 70, 8200),
               (2050, 4100, 33), (33, 33, 33), (2050, 33, 33), (100, 3295, 3301), (33, 130, 131077)],
}


@pytest.mark.parametrize("op,T,n,m", [(op, *shape) for op, shapes in TILES.items() for shape in shapes])
def test_every_tile(sg, op, T, n, m):
    g = torch.Generator(device="cuda").manual_seed(T + n + m)
    codes = torch.randint(0, 256, (m, n), generator=g, device="cuda", dtype=torch.uint8)
    scale = 0.001 + 0.001 * torch.rand(m, generator=g, device="cuda")
    zero = torch.randint(100, 156, (m,), generator=g, device="cuda").float()
    layer = sg.sg_pack_w8(codes, scale, zero)
    w = codes.double() - zero.double()[:, None]
    q, s, total = sg.sg_quantize_tokens(torch.randn(T, n, generator=g, device="cuda").to(BF16))
    if op == "product":
        Y = sg.sg_linear_w8a8(q, s, total, layer, dtype=F32)
        ref = (q.double() @ w.t()) * s.double()[:, None] * scale.double()[None, :]
        assert ((Y.double() - ref).abs() <= 4 * U32 * ref.abs()).all()
        assert torch.equal(Y, sg.sg_linear_w8a8(q, s, total, layer, dtype=F32))
        return
    dY = torch.randn(T, m, generator=g, device="cuda").to(BF16)
    d = dY.double()
    if op == "input":
        w_hat = (w.float() * scale[:, None]).to(BF16).double()
        got = sg.sg_linear_w8_grad_input(dY, layer, dtype=F32)
        again = sg.sg_linear_w8_grad_input(dY, layer, dtype=F32)
        ref, mag, K = d @ w_hat, d.abs() @ w_hat.abs(), m
    else:
        mask = (torch.rand(m, n, generator=g, device="cuda") < 0.5).to(torch.uint8)
        x = sg.sg_dequantize_tokens(q, s).double()
        got = sg.sg_linear_w8_grad_weight(dY, q, s, mask, dtype=F32)
        again = sg.sg_linear_w8_grad_weight(dY, q, s, mask, dtype=F32)
        ref, mag, K = (d.t() @ x) * (mask == 0), (d.t().abs() @ x.abs()) * (mask == 0), T
    assert torch.equal(got, again)
    tol = 2 * K * U32 * mag + U32 * ref.abs() * (1 + 2 * K * U32)
    assert ((got.double() - ref).abs() <= tol).all()


def test_masks_that_leave_nothing(sg):
    T, n, m = 70, 130, 40
    q, s, _ = sg.sg_quantize_tokens(_x(T, n, BF16, 1))
    dY = _dy(T, m, 2)
    every = torch.ones(m, n, dtype=torch.uint8, device="cuda")
    assert not sg.sg_linear_w8_grad_weight(dY, q, s, every).any()
    # a pruned entry is 0 whatever its sum is
    dY[3, 7] = float("nan")
    got = sg.sg_linear_w8_grad_weight(dY, q, s, every)
    assert not got.any()
    free = sg.sg_linear_w8_grad_weight(dY, q, s)
    assert torch.isnan(free[7]).all() and torch.isfinite(free[:7]).all() and torch.isfinite(free[8:]).all()


@pytest.mark.parametrize("T,m", [(70, 40), (33, 33), (300, 264)])
def test_a_bad_token_stays_its_own(sg, T, m):
    # an infinity or a NaN in one token's gradient reaches no other token's
    n = 96
    L = _layer(sg, m, n, 12)
    dY = _dy(T, m, 13)
    clean = sg.sg_linear_w8_grad_input(dY, L["packed"], dtype=F32)
    dY[5, 0] = float("inf")
    dY[T - 1, m - 1] = float("nan")
    got = sg.sg_linear_w8_grad_input(dY, L["packed"], dtype=F32)
    rows = [t for t in range(T) if t not in (5, T - 1)]
    assert torch.equal(got[rows], clean[rows])
    assert not torch.isfinite(got[T - 1]).any()


def test_empty_batch(sg):
    L = _layer(sg, 24, 40, 1)
    X = torch.empty(0, 40, dtype=BF16, device="cuda")
    q, s, total = sg.sg_quantize_tokens(X)
    assert q.shape == (0, 40) and s.shape == (0,) and total.shape == (0,)
    assert sg.sg_dequantize_tokens(q, s).shape == (0, 40)
    assert sg.sg_linear_w8a8(q, s, total, L["packed"]).shape == (0, 24)
    dY = torch.empty(0, 24, dtype=BF16, device="cuda")
    assert sg.sg_linear_w8_grad_input(dY, L["packed"]).shape == (0, 40)
    dW = torch.full((24, 40), 3.0, device="cuda")
    sg.sg_linear_w8_grad_weight(dY, q, s, dW=dW, accumulate=True)
    assert (dW == 3.0).all()
    sg.sg_linear_w8_grad_weight(dY, q, s, dW=dW)
    assert (dW == 0.0).all()


def test_gradients_against_differences(sg):
    # the loss sum(dY * Y) is linear in every code: a step of one code is the
    # gradient times the step's size
    T, n, m = 6, 130, 40
    L = _layer(sg, m, n, 21)
    q, s, total = sg.sg_quantize_tokens(_x(T, n, BF16, 22))
    dY = _dy(T, m, 23)
    g = dY.double()

    def loss(q, total, layer):
        return (sg.sg_linear_w8a8(q, s, total, layer, dtype=F32).double() * g).sum().item()

    dX = sg.sg_linear_w8_grad_input(dY, L["packed"], dtype=F32).double().cpu()
    dW = sg.sg_linear_w8_grad_weight(dY, q, s, dtype=F32).double().cpu()
    base = loss(q, total, L["packed"])
    Y = sg.sg_linear_w8a8(q, s, total, L["packed"], dtype=F32).double()
    # the losses: 4 u(f32) of every term, twice; the gradients: u(bf16) and
    # u(f32) of every bf16 operand's term, K additions
    lost = 2 * 4 * U32 * 1.1 * (Y.abs() * g.abs()).sum().item()
    mag_x = (g.cpu().abs() @ L["w_hat"].double().abs())
    x = q.double().cpu() * s.double().cpu()[:, None]
    mag_w = g.cpu().abs().t() @ x.abs()
    slack = U[BF16] + U32 + 2 * m * U32
    for t, c in ((0, 0), (2, 77), (5, 129)):
        q2, total2 = q.clone(), total.clone()
        step = -1 if q[t, c] > 0 else 1
        wide = torch.zeros(T, 192, dtype=torch.int8, device="cuda")
        wide[:, :n] = q2
        wide[t, c] += step
        total2[t] += step
        d = loss(wide[:, :n], total2, L["packed"]) - base
        size = step * float(s[t])
        assert abs(d - size * float(dX[t, c])) <= lost + abs(size) * slack * float(mag_x[t, c])
    for r, c in ((0, 0), (17, 64), (39, 129)):
        codes = L["codes"].clone()
        step = -1 if int(codes[r, c]) > 0 else 1
        codes[r, c] = int(codes[r, c]) + step
        p2 = sg.sg_pack_w8(codes.cuda(), L["scale"].cuda(), L["zero"].cuda())
        d = loss(q, total, p2) - base
        size = step * float(L["scale"][r])
        assert abs(d - size * float(dW[r, c])) <= lost + abs(size) * slack * float(mag_w[r, c])


def _all_calls(sg, X, dY, L, bufs):
    q, s, total = sg.sg_quantize_tokens(X, *bufs["q"])
    sg.sg_dequantize_tokens(q, s, X_out=bufs["X"])
    sg.sg_linear_w8a8(q, s, total, L["packed"], Y=bufs["Y"], workspace=bufs["ws"][0])
    sg.sg_linear_w8_grad_input(dY, L["packed"], dX=bufs["dX"], workspace=bufs["ws"][1])
    sg.sg_linear_w8_grad_weight(dY, q, s, L["mask"].cuda() if not L["mask"].is_cuda else L["mask"], dW=bufs["dW"],
                                workspace=bufs["ws"][2])


def _bufs(sg, T, n, m):
    ops = (sg.SG_OP_LINEAR_W8A8, sg.SG_OP_GRAD_INPUT, sg.SG_OP_GRAD_WEIGHT)
    return {"q": (sg._code_rows(T, n, torch.device("cuda")), torch.empty(T, device="cuda"),
                  torch.empty(T, dtype=torch.int32, device="cuda")),
            "X": torch.empty(T, n, dtype=BF16, device="cuda"), "Y": torch.empty(T, m, dtype=BF16, device="cuda"),
            "dX": torch.empty(T, n, device="cuda"), "dW": torch.empty(m, n, device="cuda"),
            "ws": [torch.empty(max(256, sg.sg_workspace_bytes(op, m, n, T, 0)), dtype=torch.uint8, device="cuda")
                   for op in ops]}


def _outs(b):
    return [b["q"][0], b["q"][1], b["q"][2], b["X"], b["Y"], b["dX"], b["dW"]]


@pytest.mark.parametrize("T,n,m", [(1, 256, 128), (40, 1000, 130), (300, 640, 520)])
def test_captured_and_replayed(sg, T, n, m):
    L = _layer(sg, m, n, 31)
    L["mask"] = L["mask"].cuda()
    X, dY = _x(T, n, BF16, 32), _dy(T, m, 33)
    bufs, eager = _bufs(sg, T, n, m), _bufs(sg, T, n, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _all_calls(sg, X, dY, L, bufs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _all_calls(sg, X, dY, L, bufs)
    for k in range(4):
        X.copy_(_x(T, n, BF16, 40 + k))
        dY.copy_(_dy(T, m, 50 + k))
        for b in _outs(bufs):
            b.zero_()
        graph.replay()
        _all_calls(sg, X, dY, L, eager)
        torch.cuda.synchronize()
        for a, b in zip(_outs(bufs), _outs(eager)):
            assert torch.equal(a, b)


def test_two_streams_at_once(sg):
    shapes = [(300, 640, 520), (70, 1000, 264)]
    work = []
    for i, (T, n, m) in enumerate(shapes):
        L = _layer(sg, m, n, 61 + i)
        L["mask"] = L["mask"].cuda()
        work.append((_x(T, n, BF16, 63 + i), _dy(T, m, 65 + i), L, _bufs(sg, T, n, m), _bufs(sg, T, n, m)))
    for X, dY, L, bufs, _ in work:
        _all_calls(sg, X, dY, L, bufs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in shapes]
    for _ in range(5):
        for st, (X, dY, L, _, other) in zip(streams, work):
            with torch.cuda.stream(st):
                _all_calls(sg, X, dY, L, other)
    torch.cuda.synchronize()
    for _, _, _, bufs, other in work:
        for a, b in zip(_outs(bufs), _outs(other)):
            assert torch.equal(a, b)


def test_from_the_sweep_to_a_training_step(sg):
    # prune + quantize, pack, run, and both gradients through autograd
    m, n, T = 96, 256, 200
    cfg = synth.LayerConfig("step", m, n, 2048, 0.02, "bf16", "linear", 4, 20.0, ("2:4",), 128, config_id=970,
                            chunk_tokens=2048)
    W, Xc = synth.make_weight(cfg, "cuda"), synth.make_x(cfg, "cuda")
    H = torch.zeros(n, n, device="cuda")
    sg.sg_hessian_accumulate(H, Xc)
    Hinv, _ = sg.sg_prepare_hinv(H, cfg.damp)
    W_hat, mask, codes, scale, zero = sg.sg_prune_quantize_layer(W, Hinv, "2:4", 8)
    layer = sg.sg_pack_w8(codes, scale, zero)
    w = (codes.double() - zero.double()[:, None]) * scale.double()[:, None]
    # the sweep's own weights are the packed layer's (one fp32 product apart)
    assert ((W_hat.double() - w).abs() <= U32 * w.abs()).all()
    X = Xc[:T].view(4, 50, n).clone().requires_grad_(True)
    Wp = W_hat.clone().requires_grad_(True)
    Y = sg.linear_w8(X, Wp, layer, mask)
    assert Y.shape == (4, 50, m) and Y.dtype == BF16
    q, s, total = sg.sg_quantize_tokens(Xc[:T])
    assert torch.equal(Y.detach().view(T, m), sg.sg_linear_w8a8(q, s, total, layer))
    dY = _dy(T, m, 5).view(4, 50, m)
    Y.backward(dY)
    assert X.grad.dtype == BF16 and Wp.grad.dtype == F32
    assert torch.equal(X.grad.view(T, n), sg.sg_linear_w8_grad_input(dY.view(T, m), layer))
    assert torch.equal(Wp.grad, sg.sg_linear_w8_grad_weight(dY.view(T, m), q, s, mask, dtype=F32))
    assert not Wp.grad[mask != 0].any()
    # an expanded gradient, a layer without a trained weight, an inference call
    X2 = Xc[:T].clone().requires_grad_(True)
    sg.linear_w8(X2, None, layer).sum().backward()
    one = torch.ones(T, m, dtype=BF16, device="cuda")
    assert torch.equal(X2.grad, sg.sg_linear_w8_grad_input(one, layer))
    Y32 = sg.linear_w8(Xc[:T].float(), None, layer)
    assert Y32.dtype == F32 and not Y32.requires_grad


def test_training_step_shapes_and_strides(sg):
    n, m = 130, 70
    L = _layer(sg, m, n, 75)
    mask = L["mask"].cuda()
    base = _x(24, n, BF16, 76).clone()
    dY = _dy(24, m, 77).clone()
    W = torch.zeros(m, n, dtype=BF16, device="cuda", requires_grad=True)

    def step(X, g):
        X = X.detach().requires_grad_(True)
        Y = sg.linear_w8(X, W, L["packed"], mask)
        return (Y.detach(), *torch.autograd.grad(Y, (X, W), g))

    want = step(base, dY)
    # a transposed input and a transposed gradient hold the same values
    Y, dX, dW = step(base.t().contiguous().t(), dY.t().contiguous().t())
    assert torch.equal(Y, want[0]) and torch.equal(dX, want[1]) and torch.equal(dW, want[2])
    Y, dX, dW = step(base.view(2, 3, 4, n), dY.view(2, 3, 4, m))
    assert Y.shape == (2, 3, 4, m) and dX.shape == (2, 3, 4, n)
    assert torch.equal(Y.view(24, m), want[0]) and torch.equal(dX.view(24, n), want[1]) and torch.equal(dW, want[2])
    # one token without a batch dimension, and none at all
    Y, dX, dW = step(base[0], dY[0])
    assert Y.shape == (m,) and dX.shape == (n,)
    assert torch.equal(Y, want[0][0])
    Y, dX, dW = step(base[:0], dY[:0])
    assert Y.shape == (0, m) and dX.shape == (0, n) and not dW.any()
    # a frozen input, a frozen weight
    X = base.clone()
    Y = sg.linear_w8(X, W, L["packed"], mask)
    assert torch.equal(torch.autograd.grad(Y, W, dY)[0], want[2])
    X = base.clone().requires_grad_(True)
    Y = sg.linear_w8(X, W.detach(), L["packed"], mask)
    assert torch.equal(torch.autograd.grad(Y, X, dY)[0], want[1])
    # no second derivative
    Y = sg.linear_w8(X, W, L["packed"], mask)
    (dX,) = torch.autograd.grad(Y, X, dY, create_graph=True)
    with pytest.raises(RuntimeError):
        dX.sum().backward()


def test_captured_training_step(sg):
    n, m, T = 256, 192, 96
    L = _layer(sg, m, n, 78)
    mask = L["mask"].cuda()
    X = _x(T, n, BF16, 79).clone().requires_grad_(True)
    W = torch.zeros(m, n, device="cuda", requires_grad=True)
    dY = _dy(T, m, 80).clone()

    def step():
        Y = sg.linear_w8(X, W, L["packed"], mask)
        return (Y, *torch.autograd.grad(Y, (X, W), dY))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(3):
        with torch.no_grad():
            X.copy_(_x(T, n, BF16, 83 + k))
            dY.copy_(_dy(T, m, 86 + k))
        for t in got:
            t.detach().zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_the_kept_checkpoint_is_eight_bits(sg):
    T, n, m = 256, 512, 64
    L = _layer(sg, m, n, 71)
    X = _x(T, n, BF16, 72).clone().requires_grad_(True)
    kept = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: kept.append(t) or t, lambda t: t):
        sg.linear_w8(X, torch.zeros(m, n, device="cuda", requires_grad=True), L["packed"], L["mask"].cuda())
    assert any(t.dtype == torch.int8 and t.shape == (T, n) for t in kept)
    assert not any(t.shape == (T, n) and t.element_size() > 1 for t in kept)


def test_solve_layer_from_checkpoints(sg):
    # recorded inputs in 8 bits: the Hessian is that of the tensors they stand for
    m, n = 64, 300
    W = (0.02 * torch.randn(m, n, generator=_gen(81))).cuda()
    chunks = [_x(700, n, BF16, 82 + i) for i in range(2)]
    recorded = [sg.sg_quantize_tokens(c) for c in chunks]
    wide = [torch.zeros(700, 304, dtype=BF16, device="cuda") for _ in chunks]
    for w, (q, s, _) in zip(wide, recorded):
        w[:, :n] = sg.sg_dequantize_tokens(q, s)
    a = sg.solve_layer(W, [w[:, :n] for w in wide], 0.5)
    b = sg.solve_layer(W, recorded, 0.5)
    c = sg.solve_layer(W, [r[:2] for r in recorded], 0.5)
    for k in ("H", "Hinv", "W_hat", "mask"):
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k])


def test_offsets_past_32_bits(sg):
    # codes of more than 2^32 bytes: the last tokens against the same tokens alone
    T, n = 66000, 65536
    X = torch.zeros(T, n, dtype=BF16, device="cuda")
    tail = _x(3, n, BF16, 91)
    X[-3:] = tail
    q, s, total = sg.sg_quantize_tokens(X)
    q3, s3, t3 = sg.sg_quantize_tokens(tail)
    assert torch.equal(q[-3:], q3) and torch.equal(s[-3:], s3) and torch.equal(total[-3:], t3)
    sg.sg_dequantize_tokens(q, s, X_out=X)
    assert torch.equal(X[-3:], sg.sg_dequantize_tokens(q3, s3)) and not X[:4].any()
    del X
    L = _layer(sg, 20, n, 92)
    Y = sg.sg_linear_w8a8(q, s, total, L["packed"])
    assert torch.equal(Y[-3:], sg.sg_linear_w8a8(q3, s3, t3, L["packed"])) and not Y[:100].any()
    dY = torch.zeros(T, 20, dtype=BF16, device="cuda")
    dY[-3:] = _dy(3, 20, 93)
    g = dY[-3:].double().cpu()
    x = sg.sg_dequantize_tokens(q3, s3).double().cpu()
    del Y
    dW = sg.sg_linear_w8_grad_weight(dY, q, s, dtype=F32)
    _close_sum(dW, g.t() @ x, g.abs().t() @ x.abs(), T, F32)


def test_outputs_past_32_bits(sg):
    T, n, m = 70000, 64, 65536
    L = _layer(sg, m, n, 95)
    X = torch.zeros(T, n, dtype=BF16, device="cuda")
    tail = _x(2, n, BF16, 96)
    X[-2:] = tail
    q, s, total = sg.sg_quantize_tokens(X)
    Y = sg.sg_linear_w8a8(q, s, total, L["packed"])
    ref = _linear_ref(q[-2:], s[-2:], L)
    assert ((Y[-2:].double().cpu() - ref).abs() <= (4 * U32 + U[BF16]) * ref.abs()).all()
    assert not Y[:50].any()
    dX = sg.sg_linear_w8_grad_input(Y, L["packed"], dtype=F32)
    w = L["w_hat"].to(BF16).double()
    g = Y[-2:].double().cpu()
    _close_sum(dX[-2:], g @ w, g.abs() @ w.abs(), m, F32)
    assert not dX[:50].any()
