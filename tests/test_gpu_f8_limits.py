"""Dropout and the linear layer in 8-bit floating point at the ends of their
ranges, in unusual use, and their refusals.

Products are of whole numbers where they are compared exactly: codes of -1 and 1
or small ones, scales that are powers of two, and sums that fp32 holds."""

import threading

import numpy as np
import pytest
import torch

import post_pruning_amd as sg
from oracle import float8

pytestmark = pytest.mark.gpu

E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(autouse=True)
def _give_memory_back():
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _signs(rows, cols, fmt, seed):
    """An F8Tensor of 1 and -1, every scale 1 (cols a multiple of 128)."""
    one = 0x38 if fmt is E4 else 0x3C
    c = torch.empty(rows, cols, dtype=torch.uint8, device="cuda").random_(0, 256, generator=_gen(seed))
    c.bitwise_and_(0x80).bitwise_or_(one)
    return sg.F8Tensor(c.view(fmt), torch.full((cols // 128, rows), 127, dtype=torch.uint8, device="cuda"))


def _small(rows, cols, fmt, seed):
    """An F8Tensor of -8 .. 8 times 1/2, 1 or 2, and its values in float64."""
    v = torch.randint(-8, 9, (rows, cols), generator=_gen(seed), device="cuda").float()
    e = torch.randint(126, 129, (-(-cols // 128), rows), generator=_gen(seed + 1), device="cuda", dtype=torch.uint8)
    unit = torch.tensor([0.5, 1.0, 2.0], device="cuda", dtype=torch.float64)[e.t().long() - 126]
    return sg.F8Tensor(v.to(fmt), e), v.double() * unit.repeat_interleave(128, 1)[:, :cols]


# One shape for every tile whose contraction is split (64-row tiles are split at
# many sizes): the sums of the parts are whole numbers below 2^24 units.
@pytest.mark.parametrize("T,n,m,out", [(4588, 8200, 139, BF16), (4588, 58543, 139, BF16), (77, 35851, 4489, BF16),
                                       (69, 5735, 4490, BF16), (65, 2509, 3, BF16), (69, 7457, 8223, F32),
                                       (4712, 4424, 68, F32), (66, 4300, 5, F32)])
@pytest.mark.parametrize("fmt", [E4, E5])
def test_split_products(T, n, m, out, fmt):
    q, xv = _small(T, n, fmt, 1)
    w, wv = _small(m, n, E4, 2)
    Y = sg.sg_linear_f8(q, sg.F8Layer(w), dtype=out)
    want = xv @ wv.t()
    assert torch.equal(Y, want.to(out))
    mask = (torch.rand(T, m, device="cuda") < 0.5).to(torch.uint8)
    start = torch.randint(-5, 6, (T, m), device="cuda").to(out)
    dW = start.clone()
    sg.sg_linear_f8_grad_weight(q, w, mask, dW=dW, accumulate=True)
    assert torch.equal(dW, (start.double() + torch.where(mask.bool(), 0.0, want)).to(out))
    drop = sg.Dropout(0.5, 9, 3)
    kept = sg.sg_dropout(torch.ones(T, m, device="cuda"), drop) == 2
    # (the second operand is a layer's transposed form)
    layer = sg.F8Layer(sg.F8Tensor(w.codes.t(), torch.full((-(-m // 128), n), 127, dtype=torch.uint8, device="cuda")), w)
    got = sg.sg_linear_f8_grad_input(q, layer, dtype=out, drop=drop)
    assert torch.equal(got, torch.where(kept, 2 * want, 0.0).to(out))


# codes of more than 2^32 bytes, outputs of more than 2^31 elements
def test_product_of_many_tokens():
    T, n, m = 34_000_000, 128, 72
    q = _signs(T, n, E4, 1)
    w = _signs(m, n, E4, 2)
    Y = sg.sg_linear_f8(q, sg.F8Layer(w))
    wv = w.codes.float()
    for a in (0, 2 ** 24 - 100, 33_554_400, T - 300):
        want = q.codes[a:a + 300].float() @ wv.t()
        assert torch.equal(Y[a:a + 300], want.to(BF16))
    # every row: its sum of outputs against its product with the sum of the weights
    total = wv.sum(0)
    for a in range(0, T, 4_000_000):
        x = q.codes[a:a + 4_000_000].float()
        assert torch.equal(Y[a:a + 4_000_000].float().sum(1), x @ total)


def test_weight_gradient_of_many_tokens():
    T, n, m = 1 << 23, 640, 264
    xt = _signs(n, T, E4, 1)
    at = torch.randint(0, T, (4000,), generator=_gen(5), device="cuda")
    at[-3:] = torch.arange(T - 3, T, device="cuda")
    at = at.unique()
    codes = torch.zeros(m, T, dtype=torch.uint8, device="cuda")
    some = torch.randint(-3, 4, (m, at.numel()), generator=_gen(6), device="cuda").float()
    codes[:, at] = some.to(E5).view(torch.uint8)
    dyt = sg.F8Tensor(codes.view(E5), torch.full((T // 128, m), 128, dtype=torch.uint8, device="cuda"))
    want = 2 * (some.double() @ xt.codes.view(torch.uint8)[:, at].view(E4).double().t())
    assert torch.equal(sg.sg_linear_f8_grad_weight(dyt, xt, dtype=F32).double(), want)
    with pytest.raises(ValueError):
        sg.sg_linear_f8_grad_weight(dyt, sg.F8Tensor(xt.codes[:, :T - 128], xt.scale[:-1]))


# more rows than a launch has groups of them, and rows past 2^32 bytes
@pytest.mark.parametrize("T,n", [(4_400_003, 130), (17_000_001, 129)])
def test_quantize_many_rows(T, n):
    X = torch.zeros(T, n, dtype=BF16, device="cuda")
    at = torch.randint(0, T, (5000,), generator=_gen(1), device="cuda")
    at[-3:] = torch.arange(T - 3, T, device="cuda")
    at = at.unique()
    X[at] = torch.randn(at.numel(), n, generator=_gen(2), device="cuda").to(BF16)
    drop = sg.Dropout(0.5, 21)
    q = sg.sg_quantize_f8(X, drop=drop)
    kept = np.concatenate([float8.keep(1, n, 0.5, 21, row0=int(r)) for r in at.tolist()[-3:]])
    Z = sg.sg_dropout(X, drop)[at]
    assert torch.equal(Z[-3:], torch.where(torch.from_numpy(kept).cuda(), 2 * X[at[-3:]], 0.0))
    want = sg.sg_quantize_f8(Z)
    assert torch.equal(q.codes.view(torch.uint8)[at], want.codes.view(torch.uint8))
    assert torch.equal(q.scale[:, at], want.scale)
    back = sg.sg_dequantize_f8(q)
    assert torch.equal(back[at], sg.sg_dequantize_f8(want))
    assert int((back != 0).any(1).sum()) == int((Z != 0).any(1).sum())


def test_widest_matrices():
    # 2^20 columns, and a layer of 2^20 outputs and one of 65536 inputs
    X = torch.randn(130, 1 << 20, generator=_gen(1), device="cuda").to(BF16)
    q, qt = sg.sg_quantize_f8(X, form="both")
    for c in (0, 524_288, (1 << 20) - 384):
        part, partt = sg.sg_quantize_f8(X[:, c:c + 384].contiguous(), form="both")
        assert torch.equal(q.codes.view(torch.uint8)[:, c:c + 384], part.codes.view(torch.uint8))
        assert torch.equal(qt.codes.view(torch.uint8)[c:c + 384], partt.codes.view(torch.uint8))
        assert torch.equal(q.scale[c // 128:c // 128 + 3], part.scale) and torch.equal(qt.scale[:, c:c + 384], partt.scale)
    for T, n, m in ((5, 256, 1 << 20), (90, 128, 1 << 20), (3, 65536, 200), (70, 65536, 300)):
        q, w = _signs(T, n, E4, 3), _signs(m, n, E4, 4)
        for out in (F32, BF16):
            assert torch.equal(sg.sg_linear_f8(q, sg.F8Layer(w), dtype=out),
                               (q.codes.double() @ w.codes.double().t()).to(out))


# ---------------------------------------------------------------------------
# unusual use
# ---------------------------------------------------------------------------
def test_scales_far_apart_in_bf16():
    # 100 products of at most 64 a row: the cut of every eight is below 8 * 2^-12 * 64 units
    T, n, m = 40, 384, 48
    for sx, sw in ((0, 247), (10, 240), (247, 0), (60, 160), (127, 1)):
        q, _ = _small(T, n, E4, 1)
        w, _ = _small(m, n, E4, 2)
        q.scale.fill_(sx), w.scale.fill_(sw)
        want = (q.codes.double() @ w.codes.double().t()) * 2.0 ** (sx + sw - 254)
        for T0 in (T, 1):
            Y = sg.sg_linear_f8(sg.F8Tensor(q.codes[:T0], q.scale[:, :T0]), sg.F8Layer(w)).double()
            # (whole numbers are not cut; bf16 rounds, and below 2^-126 to a multiple of 2^-133)
            assert ((Y - want[:T0]).abs() <= 2.0 ** -8 * want[:T0].abs() + 2.0 ** -134 + 3 * 2.0 ** -150).all()


def test_rows_inside_a_wider_matrix():
    # what lies beside the columns, NaN here, is not used
    store = torch.full((300, 520), float("nan"), dtype=BF16, device="cuda")
    X = store[:, 7:407]
    X.copy_(torch.randn(300, 400, generator=_gen(1), device="cuda"))
    W = 0.02 * torch.randn(90, 400, generator=_gen(2), device="cuda")
    assert torch.equal(sg.linear_f8(X, W), sg.linear_f8(X.contiguous(), W))
    Y = torch.full((300, 520), 5.0, dtype=BF16, device="cuda")
    drop = sg.Dropout(0.3, 4)
    sg.sg_dropout(X, drop, residual=X, Y=Y[:, 3:403])
    assert torch.equal(Y[:, 3:403], sg.sg_dropout(X.contiguous(), drop, residual=X.contiguous()))
    assert (Y[:, :3] == 5).all() and (Y[:, 403:] == 5).all()


def test_codes_laid_out_in_other_ways():
    q, xv = _small(50, 300, E4, 1)
    w, wv = _small(70, 300, E4, 2)
    want = (xv @ wv.t()).to(F32)
    other = [q.codes.contiguous(), q.codes.t().contiguous().t()]
    store = torch.zeros(50 * 300 + 5, dtype=torch.uint8, device="cuda")
    store[5:].view(50, 300).copy_(q.codes.view(torch.uint8))
    other.append(store[5:].view(50, 300).view(E4))
    scales = [q.scale.contiguous(), q.scale.t().contiguous().t()]
    odd = torch.zeros(3 * 50 + 1, dtype=torch.uint8, device="cuda")
    odd[1:].view(3, 50).copy_(q.scale)
    scales.append(odd[1:].view(3, 50))
    for c in other:
        for s in scales:
            assert torch.equal(sg.sg_linear_f8(sg.F8Tensor(c, s), sg.F8Layer(w), dtype=F32), want)
    # parts of a matrix: some of its rows, some of its blocks
    part = sg.F8Tensor(q.codes[8:41, 128:256], q.scale[1:2, 8:41])
    wp = sg.F8Layer(sg.F8Tensor(w.codes[:, 128:256], w.scale[1:2]))
    assert torch.equal(sg.sg_linear_f8(part, wp, dtype=F32), (xv[8:41, 128:256] @ wv[:, 128:256].t()).to(F32))


def test_empty_batch_in_autograd():
    W = torch.randn(60, 200, device="cuda", requires_grad=True)
    X = torch.zeros(0, 200, device="cuda", requires_grad=True)
    Y = sg.dropout(sg.linear_f8(X, W, drop=sg.Dropout(0.5, 1)), sg.Dropout(0.5, 2))
    assert Y.shape == (0, 60)
    Y.sum().backward()
    assert X.grad.shape == (0, 200) and (W.grad == 0).all()


def test_layer_packed_again_before_the_backward_pass():
    W = torch.randn(60, 200, generator=_gen(1), device="cuda")
    layer = sg.sg_pack_f8(W)
    X = torch.randn(20, 200, generator=_gen(2), device="cuda", requires_grad=True)
    Y = sg.linear_f8(X, None, layer)
    sg.sg_pack_f8(2 * W, layer=layer)
    with pytest.raises(RuntimeError):
        Y.sum().backward()
    Y = sg.linear_f8(X, None, layer)
    Y.sum().backward()
    assert torch.isfinite(X.grad).all()


def test_state_changed_before_the_backward_pass():
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    X = torch.randn(20, 200, generator=_gen(2), device="cuda", requires_grad=True)
    Y = sg.dropout(X, sg.Dropout(0.5, 1, state=state))
    state.add_(1)
    with pytest.raises(RuntimeError):
        Y.sum().backward()


def test_what_is_kept_may_move():
    X = torch.randn(140, 300, generator=_gen(1), device="cuda")
    W = 0.02 * torch.randn(90, 300, generator=_gen(2), device="cuda")
    mask = (W.abs() < 0.01).to(torch.uint8)

    def run(layer):
        x, w = X.clone().requires_grad_(True), W.clone().requires_grad_(True)
        sg.linear_f8(x, w, layer, mask, sg.Dropout(0.2, 3)).square().sum().backward()
        return x.grad, w.grad

    for layer in (None, sg.sg_pack_f8(W)):
        want = run(layer)
        with torch.autograd.graph.save_on_cpu():
            got = run(layer)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_inference_tensors():
    with torch.inference_mode():
        X = torch.randn(40, 300, generator=_gen(1), device="cuda").to(BF16)
        W = 0.02 * torch.randn(90, 300, generator=_gen(2), device="cuda")
        layer = sg.sg_pack_f8(W)
        Y = sg.linear_f8(X, None, layer, drop=sg.Dropout(0.5, 2))
        assert torch.equal(Y, sg.sg_linear_f8(sg.sg_quantize_f8(X, drop=sg.Dropout(0.5, 2)), layer))
        sg.sg_pack_f8(W, layer=layer)
        q = sg.sg_quantize_f8(X)
        sg.sg_quantize_f8(X, q=q)


def test_two_threads_and_streams():
    W = 0.02 * torch.randn(500, 4096, generator=_gen(2), device="cuda")
    Xs = [torch.randn(70 + i, 4096, generator=_gen(10 + i), device="cuda").to(BF16) for i in range(4)]
    want = [sg.linear_f8(x, W) for x in Xs]
    got = [None] * 4
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got[i] = sg.linear_f8(Xs[i], W)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_with_one_workspace():
    T, n, m = 70, 8192, 500
    q, xv = _small(T, n, E4, 1)
    w, wv = _small(m, n, E4, 3)
    q2, xv2 = _small(T, n, E4, 5)
    layer = sg.F8Layer(w)
    size = sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, m, n, T)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs = [torch.empty(T, m, device="cuda") for _ in range(2)]
    sg.sg_linear_f8(q, layer, Y=outs[0], workspace=ws)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, a, o in zip(graphs, (q, q2), outs):
        with torch.cuda.graph(g):
            sg.sg_linear_f8(a, layer, Y=o, workspace=ws)
    for _ in range(3):
        for o in outs:
            o.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], (xv @ wv.t()).float()) and torch.equal(outs[1], (xv2 @ wv.t()).float())


# ---------------------------------------------------------------------------
# refusals (nothing is launched)
# ---------------------------------------------------------------------------
def test_refusals():
    X = torch.randn(40, 300, device="cuda")
    q, qt = sg.sg_quantize_f8(X, form="both")
    layer = sg.sg_pack_f8(torch.randn(50, 300, device="cuda"))
    dy, dyt = sg.sg_quantize_f8(torch.randn(40, 50, device="cuda"), E5, form="both")
    bad = (ValueError, TypeError, sg.SGError)
    calls = [
        lambda: sg.sg_quantize_f8(X.half()), lambda: sg.sg_quantize_f8(X, torch.uint8), lambda: sg.sg_quantize_f8(X, form="row"),
        lambda: sg.sg_quantize_f8(X[0]), lambda: sg.sg_quantize_f8(X.t()), lambda: sg.sg_quantize_f8(X, q=qt),
        lambda: sg.sg_quantize_f8(X, E5, q=q), lambda: sg.sg_quantize_f8(X[:1].expand(40, 300)),
        lambda: sg.sg_dequantize_f8(q, torch.float16), lambda: sg.sg_dequantize_f8(q, X_out=torch.empty(40, 299, device="cuda")),
        lambda: sg.sg_pack_f8(X.double()), lambda: sg.sg_pack_f8(X, layer=layer), lambda: sg.sg_pack_f8(X[0]),
        lambda: sg.sg_linear_f8(dy, layer), lambda: sg.sg_linear_f8(q, layer, dtype=torch.float16),
        lambda: sg.sg_linear_f8(q, layer, Y=torch.empty(40, 49, device="cuda")),
        lambda: sg.sg_linear_f8(q, layer, Y=torch.empty(50, 40, device="cuda").t()),
        lambda: sg.sg_linear_f8(q, layer, Y=torch.empty(40, 50)),
        lambda: sg.sg_linear_f8_grad_input(q, layer), lambda: sg.sg_linear_f8_grad_input(dy, sg.F8Layer(layer.w)),
        lambda: sg.sg_linear_f8_grad_weight(dy, qt), lambda: sg.sg_linear_f8_grad_weight(qt, dyt),
        lambda: sg.sg_linear_f8_grad_weight(dyt, qt, torch.zeros(50, 299, dtype=torch.uint8, device="cuda")),
        lambda: sg.sg_linear_f8_grad_weight(dyt, qt, torch.zeros(50, 300, device="cuda")),
        lambda: sg.sg_linear_f8_grad_weight(dyt, qt, accumulate=True),
        lambda: sg.F8Layer(dy), lambda: sg.F8Layer(layer.w, layer.w), lambda: sg.F8Tensor(q.codes, q.scale[:, :39]),
        lambda: sg.F8Tensor(q.codes, q.scale.float()), lambda: sg.F8Tensor(q.codes[0], q.scale),
        lambda: sg.F8Tensor(q.codes, q.scale.cpu()),
        lambda: sg.sg_dropout(X, sg.Dropout(0.5, 1), residual=X.bfloat16()),
        lambda: sg.sg_dropout(X, sg.Dropout(0.5, 1), residual=X[:, :299]),
        lambda: sg.sg_dropout(X, sg.Dropout(0.5, 1), Y=torch.empty(40, 300, dtype=BF16, device="cuda")),
        lambda: sg.sg_dropout(X[0], sg.Dropout(0.5, 1)), lambda: sg.sg_dropout(X.long(), sg.Dropout(0.5, 1)),
        lambda: sg.linear_f8(X, torch.randn(50, 299, device="cuda")),
        lambda: sg.linear_f8(X, torch.randn(50, 300, device="cuda"), mask=torch.zeros(50, 300, device="cuda")),
        lambda: sg.linear_f8(X, torch.randn(49, 300, device="cuda"), layer),
        lambda: sg.dropout(X, sg.Dropout(0.5, 1), residual=X[:1]),
        lambda: sg.solve_layer(torch.randn(8, 299, device="cuda"), [q], 0.5),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(bad):
            call()
            pytest.fail(f"call {k} was taken")
    big, few = sg.F8Layer(_signs(4489, 8192, E4, 1)), _signs(70, 8192, E4, 2)
    need = sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, 4489, 8192, 70)
    if need:
        with pytest.raises(bad):
            sg.sg_linear_f8(few, big, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
