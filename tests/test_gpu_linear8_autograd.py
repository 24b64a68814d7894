"""linear_w8 between its forward and its backward pass."""

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


def _work(sg, T, n, m, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (m, n), generator=g, device="cuda", dtype=torch.uint8)
    layer = sg.sg_pack_w8(codes, 0.01 * torch.rand(m, generator=g, device="cuda"), torch.full((m,), 128.0, device="cuda"))
    X = torch.randn(T, n, generator=g, device="cuda").to(BF16).requires_grad_(True)
    W = torch.zeros(m, n, device="cuda", requires_grad=True)
    mask = (torch.rand(m, n, generator=g, device="cuda") < 0.5).to(torch.uint8)
    dY = torch.randn(T, m, generator=g, device="cuda").to(BF16)
    return layer, X, W, mask, dY


@pytest.mark.parametrize("part", ["codes", "offset", "scale"])
def test_a_layer_changed_in_between_is_an_error(sg, part):
    layer, X, W, mask, dY = _work(sg, 40, 130, 70)
    other = _work(sg, 40, 130, 70, 2)[0]
    Y = sg.linear_w8(X, W, layer, mask)
    getattr(layer, part).copy_(getattr(other, part))  # packed again into the same tensors
    with pytest.raises(RuntimeError, match="changed in place"):
        Y.backward(dY)
    # after the backward pass it may change, and the next pass takes the new layer
    Y = sg.linear_w8(X, W, layer, mask)
    Y.backward(dY)
    getattr(layer, part).copy_(getattr(other, part))
    want = torch.autograd.grad(sg.linear_w8(X, W, layer, mask), X, dY)[0]
    assert torch.equal(want, sg.sg_linear_w8_grad_input(dY, layer))


def test_layer_packed_in_inference_mode(sg):
    with torch.inference_mode():
        layer = _work(sg, 40, 130, 70)[0]
    _, X, W, mask, dY = _work(sg, 40, 130, 70)
    sg.linear_w8(X, W, layer, mask).backward(dY)
    assert torch.equal(X.grad, sg.sg_linear_w8_grad_input(dY, layer))


@pytest.mark.parametrize("T,n", [(40, 130), (1, 130), (40, 128), (0, 130)])
def test_saved_tensors_that_are_stored_elsewhere(sg, T, n):
    # a hook that keeps the values on the host, not their strides
    layer, X, W, mask, dY = _work(sg, T, n, 70)
    want = torch.autograd.grad(sg.linear_w8(X, W, layer, mask), (X, W), dY)
    with torch.autograd.graph.save_on_cpu():
        Y = sg.linear_w8(X, W, layer, mask)
    for a, b in zip(torch.autograd.grad(Y, (X, W), dY), want):
        assert torch.equal(a, b)


def test_recomputed_in_the_backward_pass(sg):
    from torch.utils.checkpoint import checkpoint
    layer, X, W, mask, dY = _work(sg, 40, 130, 70)
    want = torch.autograd.grad(sg.linear_w8(X, W, layer, mask), (X, W), dY)
    for reentrant in (False, True):
        Y = checkpoint(sg.linear_w8, X, W, layer, mask, use_reentrant=reentrant)
        X.grad = W.grad = None
        Y.backward(dY)
        assert torch.equal(X.grad, want[0]) and torch.equal(W.grad, want[1])
