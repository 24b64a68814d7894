"""What the binding of the 8-bit linear layer tells autograd.  The library's
calls are not made, so no GPU is needed."""

import pytest
import torch

import post_pruning_amd as sg

T, N, M = 40, 192, 128


@pytest.fixture(autouse=True)
def _no_library(monkeypatch):
    monkeypatch.setattr(sg, "_same_gpu", lambda first, *others: 0)
    monkeypatch.setattr(sg, "_call", lambda *args: None)
    monkeypatch.setattr(sg, "load_library", lambda *a: type("Lib", (), {"__getattr__": lambda s, n: None})())
    monkeypatch.setattr(sg, "_ws_bytes", lambda *a: 0)


def _given():
    """(tensors, call that writes into them)."""
    X, Y, W = torch.zeros(T, N), torch.zeros(T, M), torch.zeros(M, N)
    q, scale, total = torch.zeros(T, N, dtype=torch.int8), torch.zeros(T), torch.zeros(T, dtype=torch.int32)
    layer = sg.W8Layer._unwritten(M, N, "cpu")
    dY = torch.zeros(T, M, dtype=torch.bfloat16)
    x, y, w = X.clone(), Y.clone(), W.clone()
    return [((q, scale, total), lambda: sg.sg_quantize_tokens(X, q, scale, total)),
            ((q,), lambda: sg.sg_quantize_tokens(X, q)), ((x,), lambda: sg.sg_dequantize_tokens(q, scale, X_out=x)),
            ((y,), lambda: sg.sg_linear_w8a8(q, scale, total, layer, Y=y)),
            ((x,), lambda: sg.sg_linear_w8_grad_input(dY, layer, dX=x)),
            ((w,), lambda: sg.sg_linear_w8_grad_weight(dY, q, scale, dW=w)),
            ((w,), lambda: sg.sg_linear_w8_grad_weight(dY, q, scale, dW=w, accumulate=True))]


@pytest.mark.parametrize("case", range(7))
def test_autograd_hears_of_what_is_written(case):
    ts, call = _given()[case]
    before = [t._version for t in ts]
    call()
    assert all(t._version > v for t, v in zip(ts, before))
    with torch.inference_mode():
        _given()[case][1]()
