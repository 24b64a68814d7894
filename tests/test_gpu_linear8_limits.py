"""The 8-bit linear layer at the ends of its ranges, with whole numbers.

Codes, gradients and powers of two as scales make every product and every
partial sum a whole number (times a power of two) that fp32 holds, in whatever
order it is formed, so results have to be equal, not close: a row left out or
read from another place shows at any length of the contraction.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sg():
    import post_pruning_amd as sg
    sg.load_library()
    assert torch.cuda.is_available()
    return sg


@pytest.fixture(autouse=True)
def _give_memory_back():
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# The bf16 copy of the checkpoint would have rows of 2 T bytes, 256 and 64 of
# which span more than 2^32.  dY is 0 but for 3000 tokens, the last among them:
# |sums| <= 3000 * 3 * 127 < 2^24.
@pytest.mark.parametrize("T,n,m", [(9_000_000, 1024, 264), (34_200_000, 128, 128)])
def test_weight_gradient_of_many_tokens(sg, T, n, m):
    g = _gen(T)
    q = torch.randint(-127, 128, (T, n), generator=g, device="cuda", dtype=torch.int8)
    scale = torch.full((T,), 0.5, device="cuda")
    at = torch.randint(0, T, (3000,), generator=g, device="cuda")
    at[-3:] = torch.arange(T - 3, T, device="cuda")
    at = at.unique()
    dY = torch.zeros(T, m, dtype=BF16, device="cuda")
    some = torch.randint(-3, 4, (at.numel(), m), generator=g, device="cuda")
    dY[at] = some.to(BF16)
    want = 0.5 * (some.double().t() @ q[at].double())
    got = sg.sg_linear_w8_grad_weight(dY, q, scale, dtype=F32)
    assert torch.equal(got.double(), want)


# More rows than one launch has threads for.
@pytest.mark.parametrize("T,n", [((1 << 26) + 5, 1), ((1 << 24) + 3, 1025)])
def test_quantize_many_tokens(sg, T, n):
    g = _gen(T)
    at = torch.randint(0, T, (5000,), generator=g, device="cuda")
    at[-3:] = torch.arange(T - 3, T, device="cuda")
    at = at.unique()
    X = torch.zeros(T, n, dtype=BF16, device="cuda")
    X[at] = torch.randn(at.numel(), n, generator=g, device="cuda").to(BF16)
    pitch = -(-n // 64) * 64
    store = torch.full((T, pitch), 77, dtype=torch.int8, device="cuda")
    scale, total = torch.full((T,), -1.0, device="cuda"), torch.full((T,), 77, dtype=torch.int32, device="cuda")
    q, _, _ = sg.sg_quantize_tokens(X, store[:, :n], scale, total)
    qa, sa, ta = sg.sg_quantize_tokens(X[at])
    assert torch.equal(q[at], qa) and torch.equal(scale[at], sa) and torch.equal(total[at], ta)
    store[at] = 0
    scale[at] = 1.0
    total[at] = 0
    assert not store.view(torch.int64).any() and not total.any() and (scale == 1.0).all()
    q[at] = qa
    scale[at] = sa
    X.fill_(7.0)
    sg.sg_dequantize_tokens(q, scale, X_out=X)
    assert torch.equal(X[at], sg.sg_dequantize_tokens(qa, sa))
    X[at] = 0.0
    assert not X.any()


def test_products_of_many_tokens(sg):
    # rows of tokens in two launches
    T, n, m = (1 << 28) + 70, 1, 1
    g = _gen(5)
    codes = torch.tensor([[201]], dtype=torch.uint8, device="cuda")
    layer = sg.sg_pack_w8(codes, torch.full((1,), 0.25, device="cuda"), torch.full((1,), 77.0, device="cuda"))
    q = torch.zeros(T, 64, dtype=torch.int8, device="cuda")[:, :1]
    q.copy_(torch.randint(-127, 128, (T, 1), generator=g, device="cuda", dtype=torch.int8))
    Y = torch.full((T, 1), 7.0, device="cuda")
    sg.sg_linear_w8a8(q, torch.full((T,), 2.0, device="cuda"), q[:, 0].int(), layer, Y=Y)
    assert torch.equal(Y, q.float() * (0.5 * (201 - 77)))
    del Y
    dY = q.to(BF16)
    dX = torch.full((T, 1), 7.0, device="cuda")
    sg.sg_linear_w8_grad_input(dY, layer, dX=dX)
    assert torch.equal(dX, q.float() * (0.25 * (201 - 77)))


# The last position of every prompt: rows S n apart, more than the library's 2^23 bytes.
@pytest.mark.parametrize("B", [1, 4])
def test_last_position_of_a_prompt(sg, B):
    S, n, m = 2048, 4096, 72
    g = _gen(B)
    codes = torch.randint(0, 256, (m, n), generator=g, device="cuda", dtype=torch.uint8)
    layer = sg.sg_pack_w8(codes, torch.rand(m, generator=g, device="cuda"), torch.full((m,), 128.0, device="cuda"))
    hidden = torch.zeros(B, S, n, dtype=BF16, device="cuda")
    hidden[:, -1] = torch.randn(B, n, generator=g, device="cuda").to(BF16)
    W = torch.zeros(m, n, device="cuda", requires_grad=True)
    last = hidden[:, -1, :]
    assert last.stride(0) * 2 > 1 << 23

    def step(X, dY):
        X = X.detach().requires_grad_(True)
        Y = sg.linear_w8(X, W, layer)
        return (Y.detach(), *torch.autograd.grad(Y, (X, W), dY))

    far = torch.empty(B * (1 << 23), dtype=BF16, device="cuda").as_strided((B, m), (1 << 23, 1))
    far.copy_(torch.randn(B, m, generator=g, device="cuda").to(BF16))
    for a, b in zip(step(last, far), step(last.contiguous(), far.contiguous())):
        assert torch.equal(a, b)
    if B == 1:
        for a, b in zip(sg.sg_quantize_tokens(last), sg.sg_quantize_tokens(last.contiguous())):
            assert torch.equal(a, b)
        assert torch.equal(sg.sg_linear_w8_grad_input(far, layer), sg.sg_linear_w8_grad_input(far.contiguous(), layer))
    else:
        with pytest.raises(sg.SGError):  # nothing is copied behind a direct call's back
            sg.sg_quantize_tokens(last)


# Odd shapes that between them reach every tile of the gradients, whole and
# split: |dY| <= 3, |codes| <= 32 and at most 131077 products keep every partial
# sum below 2^24.  A stage of 64 rows left out of any contraction would show.
GRADS = {
    "input": [(130, 33000, 33), (203, 8200, 20001), (20001, 130, 70), (4100, 203, 8200), (8200, 70, 770),
              (2050, 70, 4100), (33, 33, 770), (33, 33, 2600), (70, 20001, 33), (70, 2050, 4100), (70, 8200, 33),
              (33, 2050, 4100), (33, 33, 33), (33, 33, 2050), (3301, 3295, 100), (20, 130, 131077), (129, 1000, 2050),
              (512, 4096, 4096), (300, 28672, 24)],
    "weight": [(33, 130, 33000), (20001, 203, 8200), (70, 130, 20001), (8200, 203, 4100), (770, 70, 8200),
               (4100, 70, 2050), (770, 33, 33), (2600, 33, 33), (33, 70, 20001), (4100, 2050, 70), (33, 70, 8200),
               (2050, 4100, 33), (33, 33, 33), (2050, 33, 33), (100, 3295, 3301), (33, 130, 131077), (131077, 130, 20),
               (515, 1000, 770), (512, 4096, 4096)],
}


@pytest.mark.parametrize("op,T,n,m", [(op, *shape) for op, shapes in GRADS.items() for shape in shapes])
def test_gradients_are_exact(sg, op, T, n, m):
    g = _gen(T + n + m)
    dY = torch.randint(-3, 4, (T, m), generator=g, device="cuda")
    if op == "input":
        w = torch.randint(-32, 33, (m, n), generator=g, device="cuda")
        zero = torch.randint(40, 200, (m,), generator=g, device="cuda")
        layer = sg.sg_pack_w8((w + zero[:, None]).to(torch.uint8), torch.full((m,), 0.125, device="cuda"), zero.float())
        want = dY.double() @ w.double() * 0.125
        for dtype in (F32, BF16):
            got = sg.sg_linear_w8_grad_input(dY.to(BF16), layer, dtype=dtype)
            assert torch.equal(got, want.to(F32).to(dtype))
        last = dY[:, -min(m, 64):].double() @ w[-min(m, 64):].double()
    else:
        q = sg._code_rows(T, n, torch.device("cuda"))
        q.copy_(torch.randint(-32, 33, (T, n), generator=g, device="cuda"))
        scale = torch.full((T,), 0.125, device="cuda")
        mask = (torch.rand(m, n, generator=g, device="cuda") < 0.5).to(torch.uint8)
        full = dY.double().t() @ q.double() * 0.125
        for dtype in (F32, BF16):
            assert torch.equal(sg.sg_linear_w8_grad_weight(dY.to(BF16), q, scale, dtype=dtype), full.to(F32).to(dtype))
            got = sg.sg_linear_w8_grad_weight(dY.to(BF16), q, scale, mask, dtype=dtype)
            assert torch.equal(got, (full * (mask == 0)).to(F32).to(dtype))
        base = torch.randint(-64, 65, (m, n), generator=g, device="cuda").float()
        both = base.double() + full * (mask == 0)
        sg.sg_linear_w8_grad_weight(dY.to(BF16), q, scale, mask, dW=base, accumulate=True)
        assert torch.equal(base.double(), both)
        last = dY[-min(T, 64):].double().t() @ q[-min(T, 64):].double()
    assert (last != 0).any()  # the last stage counts


def test_layer_of_a_column_slice(sg):
    T, n, m = 9, 200, 17
    g = _gen(3)
    codes = torch.randint(0, 256, (m, n), generator=g, device="cuda", dtype=torch.uint8)
    wide = sg.sg_pack_w8(codes, torch.full((m,), 0.5, device="cuda"), torch.full((m,), 128.0, device="cuda"))
    with pytest.raises(ValueError, match="zeros"):
        sg.W8Layer(wide.codes[:, :100], wide.offset, wide.scale)
    part = sg.W8Layer(wide.codes[:, :128], wide.offset, wide.scale)
    again = sg.W8Layer(wide.codes, wide.offset, wide.scale)
    for layer, cols in ((part, 128), (again, n)):
        q = torch.randint(-127, 128, (T, 256), generator=g, device="cuda", dtype=torch.int8)[:, :cols]
        Y = sg.sg_linear_w8a8(q, torch.ones(T, device="cuda"), q.int().sum(1).int(), layer, dtype=F32)
        assert torch.equal(Y.double(), 0.5 * q.double() @ (codes[:, :cols].double() - 128.0).t())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,n,m", [(70, 144, 40), (70, 129, 40), (9000, 132, 70), (9000, 131, 70), (33, 64, 33)])
def test_accumulating_leaves_pruned_weights_as_they_are(sg, T, n, m, dtype):
    # bit for bit, zeros of either sign and values that are no numbers
    g = _gen(T + n)
    dY = torch.randn(T, m, generator=g, device="cuda").to(BF16)
    q, s, _ = sg.sg_quantize_tokens(torch.randn(T, n, generator=g, device="cuda").to(BF16))
    mask = (torch.rand(m, n, generator=g, device="cuda") < 0.5).to(torch.uint8)
    base = torch.randn(m, n, generator=g, device="cuda").to(dtype)
    for k, v in enumerate((0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-40, -1e-40)):
        base[:, k::11] = v
    bits = torch.int32 if dtype is F32 else torch.int16
    got = sg.sg_linear_w8_grad_weight(dY, q, s, mask, dW=base.clone(), accumulate=True)
    assert torch.equal(got.view(bits)[mask != 0], base.view(bits)[mask != 0])
