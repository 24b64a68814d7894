"""Dropout by numbers from a counter on the GPU, against the oracle's.

x times the factor is rounded to fp32, the sum with the residual to fp32 and the
result to its type: all of them are repeated here, so outputs have to be equal."""

import numpy as np
import pytest
import torch

import post_pruning_amd as sg
from oracle import float8

pytestmark = pytest.mark.gpu


def _input(T, n, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, n, generator=g).to(dtype)


def _want(X, kept, p, R=None):
    y = torch.from_numpy(float8.drop(X.double().numpy(), kept, p)).float()
    return (y if R is None else y + R.float()).to(X.dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,n", [(1, 1), (1, 7), (3, 8), (5, 1001), (40, 64), (257, 20), (2, 4096)])
def test_against_the_oracle(T, n, dtype):
    X, R = _input(T, n, 1, dtype), _input(T, n, 2, dtype)
    for p, seed, offset in ((0.1, 0, 0), (0.5, 2 ** 63 + 17, 2 ** 64 - 1), (0.999, 5, 1 << 32), (0.0, 1, 1)):
        kept = float8.keep(T, n, p, seed, offset)
        d = sg.Dropout(p, seed, offset)
        assert torch.equal(sg.sg_dropout(X.cuda(), d).cpu(), _want(X, kept, p))
        assert torch.equal(sg.sg_dropout(X.cuda(), d, residual=R.cuda()).cpu(), _want(X, kept, p, R))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift,px,pr,py", [(0, 304, 320, 304), (1, 301, 300, 299), (8, 304, 304, 301), (0, 304, 301, 304)])
def test_strides(shift, px, pr, py, dtype):
    T, n = 37, 299
    kept = float8.keep(T, n, 0.3, 9)
    mk = lambda pitch, seed: torch.as_strided(_input(1, T * pitch + 16, seed, dtype)[0].cuda(), (T, n), (pitch, 1), shift)  # noqa: E731
    X, R = mk(px, 1), mk(pr, 2)
    store = torch.full((T * py + 16,), 9.0, dtype=dtype, device="cuda")
    Y = torch.as_strided(store, (T, n), (py, 1), shift)
    sg.sg_dropout(X, sg.Dropout(0.3, 9), residual=R, Y=Y)
    assert torch.equal(Y.cpu(), _want(X.cpu(), kept, 0.3, R.cpu()))
    inside = torch.zeros_like(store, dtype=torch.bool)
    torch.as_strided(inside, (T, n), (py, 1), shift).fill_(True)
    assert (store[~inside] == 9).all()


def test_dropped_elements_leave_nothing_behind():
    X = torch.full((64, 128), float("nan"))
    X[::2] = float("inf")
    R = _input(64, 128, 3, torch.float32)
    kept = float8.keep(64, 128, 0.5, 4)
    Y = sg.sg_dropout(X.cuda(), sg.Dropout(0.5, 4), residual=R.cuda()).cpu()
    assert torch.equal(Y[~torch.from_numpy(kept)], R[~torch.from_numpy(kept)])
    assert not torch.isfinite(Y[torch.from_numpy(kept)]).any()
    Y = sg.sg_dropout(-X.cuda(), sg.Dropout(0.5, 4)).cpu()[~torch.from_numpy(kept)]
    assert (Y == 0).all() and not torch.signbit(Y).any()


def test_in_place_and_empty():
    X, R = _input(33, 100, 1, torch.bfloat16).cuda(), _input(33, 100, 2, torch.bfloat16).cuda()
    d = sg.Dropout(0.2, 6, 2)
    want, with_r = sg.sg_dropout(X, d), sg.sg_dropout(X, d, residual=R)
    a = X.clone()
    assert torch.equal(sg.sg_dropout(a, d, Y=a), want) and torch.equal(a, want)
    r = R.clone()
    sg.sg_dropout(X, d, residual=r, Y=r)
    assert torch.equal(r, with_r)
    assert sg.sg_dropout(X[:0], d).shape == (0, 100)


def test_state_on_the_device():
    X = _input(20, 200, 1, torch.float32)
    state = torch.tensor([3, 2 ** 40], device="cuda")
    Y = sg.sg_dropout(X.cuda(), sg.Dropout(0.4, 2 ** 64 - 1, 5, state)).cpu()
    assert torch.equal(Y, _want(X, float8.keep(20, 200, 0.4, 2, 5 + 2 ** 40), 0.4))


def test_more_rows_than_a_launch_has_blocks():
    T = 70000 * 8
    X = torch.ones(T, 30, dtype=torch.bfloat16, device="cuda")
    Y = sg.sg_dropout(X, sg.Dropout(0.5, 8))
    for t in (0, 65535, 65536, 300000, T - 1):
        kept = float8.keep(1, 30, 0.5, 8, row0=t)
        assert torch.equal(Y[t].cpu() == 2, torch.from_numpy(kept[0]))
    # 16.8 million draws: six standard deviations of one half
    assert abs((Y == 2).float().mean().item() - 0.5) < 6 * 0.5 / (T * 30) ** 0.5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient(dtype):
    X = _input(6, 50, 1, dtype).cuda().requires_grad_(True)
    R = _input(6, 50, 2, dtype).cuda().requires_grad_(True)
    d = sg.Dropout(0.5, 12)
    Y = sg.dropout(X, d, residual=R)
    dY = _input(6, 50, 3, dtype).cuda()
    Y.backward(dY)
    kept = float8.keep(6, 50, 0.5, 12)
    assert torch.equal(X.grad.cpu(), _want(dY.cpu(), kept, 0.5)) and torch.equal(R.grad, dY)
    # against differences: the call is linear in X, with powers of two all is exact
    x = torch.ones(6, 50, device="cuda")
    up, down = (sg.sg_dropout(x + h, d) for h in (1.0, -1.0))
    x.requires_grad_(True)
    sg.dropout(x, d).sum().backward()
    assert torch.equal(x.grad, (up - down) / 2)


def test_any_strides_and_shapes():
    d = sg.Dropout(0.3, 5)
    X = _input(24, 40, 1, torch.float32).cuda()
    want = sg.sg_dropout(X, d)
    assert torch.equal(sg.dropout(X.view(2, 3, 4, 40), d).view(24, 40), want)
    assert torch.equal(sg.dropout(X.t().contiguous().t(), d), want)
    assert torch.equal(sg.dropout(X[0], d), want[0])
    x = X[:1].clone().requires_grad_(True)
    y = sg.dropout(x.expand(24, 40), d)
    y.sum().backward()
    kept = torch.from_numpy(float8.keep(24, 40, 0.3, 5)).cuda()
    # (24 equal fp32 numbers are added up: each of the sums is off by half a step)
    grow = float(np.float32(1 / 0.7))
    assert torch.allclose(x.grad[0].double(), kept.sum(0).double() * grow, rtol=24 * 2.0 ** -24, atol=0)
    big = X[:, :10].expand(24, 10)
    assert torch.equal(sg.dropout(big, d), sg.sg_dropout(X[:, :10].contiguous(), d))


def test_state_changed_before_the_backward_pass():
    state = torch.zeros(2, dtype=torch.int64, device="cuda")
    X = _input(4, 8, 1, torch.float32).cuda().requires_grad_(True)
    Y = sg.dropout(X, sg.Dropout(0.5, 1, 0, state))
    state.add_(1)
    with pytest.raises(RuntimeError):
        Y.sum().backward()


def test_binding_refusals():
    d = sg.Dropout(0.5, 1)
    X = torch.zeros(4, 8, device="cuda")
    for bad in (dict(residual=X[:3]), dict(residual=X.bfloat16()), dict(Y=X.bfloat16()), dict(Y=X[:, :4])):
        with pytest.raises(ValueError):
            sg.sg_dropout(X, d, **bad)
    with pytest.raises(ValueError):
        sg.sg_dropout(X.half(), d)
    with pytest.raises(ValueError):
        sg.sg_dropout(X.t(), d)
    with pytest.raises(ValueError):
        sg.dropout(X, d, residual=X[:1])
    with pytest.raises(TypeError):
        sg.dropout(X.half(), d)
