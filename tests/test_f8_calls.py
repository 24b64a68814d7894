"""What the binding of the layer in 8-bit floating point asks of the library.
The calls are noted and not made, so no GPU is needed."""

import pytest
import torch

import post_pruning_amd as sg

T, N, M = 40, 200, 150


class _Notes(list):
    """Stands in for the library: takes every call."""

    def of(self, name):
        return [args for where, args in self if where == name]


@pytest.fixture
def calls(monkeypatch):
    notes = _Notes()
    monkeypatch.setattr(sg, "_same_gpu", lambda first, *others: 0)
    monkeypatch.setattr(sg, "_call", lambda where, index, fn, *args: notes.append((where, args)))
    monkeypatch.setattr(sg, "load_library", lambda *a: type("Lib", (), {"__getattr__": lambda s, n: None})())
    monkeypatch.setattr(sg, "_ws_bytes", lambda *a: 0)
    return notes


def _layer(transposed):
    e4m3, like = torch.float8_e4m3fn, torch.empty(1)
    w = sg.F8Tensor._unwritten(M, N, e4m3, like)
    return sg.F8Layer(w, sg.F8Tensor._unwritten(N, M, e4m3, like) if transposed else None)


def _operands(x_grad, w_grad, dtype=torch.bfloat16):
    return torch.zeros(T, N, dtype=dtype, requires_grad=x_grad), torch.zeros(M, N, requires_grad=w_grad)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("x_grad,w_grad", [(False, True), (True, False), (True, True)])
def test_no_transposed_forms(calls, mode, x_grad, w_grad):
    X, W = _operands(x_grad, w_grad)
    with mode():
        assert sg.linear_f8(X, W).shape == (T, M)
    (quantize,), (pack,) = calls.of("sg_quantize_f8"), calls.of("sg_pack_f8")
    assert quantize[0] is not None and quantize[4:8] == (None, 0, None, 0)
    assert pack[0] is not None and pack[4:8] == (None, 0, None, 0)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_layer_without_its_transposed_form(calls, mode):
    X, W = _operands(True, True)
    with mode():
        sg.linear_f8(X, W, _layer(False))
    assert len(calls.of("sg_linear_f8")) == 1
    with pytest.raises(ValueError):
        sg.linear_f8(X, W, _layer(False))


def test_gradients_still_have_them(calls):
    for x_grad, w_grad in ((False, True), (True, False), (True, True)):
        calls.clear()
        X, W = _operands(x_grad, w_grad)
        assert sg.linear_f8(X, W).requires_grad
        (quantize,), (pack,) = calls.of("sg_quantize_f8"), calls.of("sg_pack_f8")
        assert (quantize[4] is not None) == w_grad and (pack[4] is not None) == x_grad


def test_a_form_that_is_not_written_is_refused(calls):
    X, e4m3 = torch.zeros(T, N), torch.float8_e4m3fn
    q, qt = sg.F8Tensor._unwritten(T, N, e4m3, X), sg.F8Tensor._unwritten(N, T, e4m3, X)
    q._gpu = qt._gpu = 0
    for form, given in (("rows", dict(qt=qt)), ("columns", dict(q=q)), ("rows", dict(q=q, qt=qt))):
        with pytest.raises(ValueError):
            sg.sg_quantize_f8(X, form=form, **given)
    assert not calls
    for form, given in (("rows", dict(q=q)), ("columns", dict(qt=qt)), ("both", dict(q=q, qt=qt))):
        got = sg.sg_quantize_f8(X, form=form, **given)
        assert got is q or got is qt or got == (q, qt)
    assert len(calls) == 3


def _given(calls):
    """(tensor, call that writes into it)."""
    e4m3, X, Y = torch.float8_e4m3fn, torch.zeros(T, N), torch.zeros(T, M)
    q, qt, dy, dyt = (sg.F8Tensor._unwritten(*s, e4m3, X) for s in ((T, N), (N, T), (T, M), (M, T)))
    layer = _layer(True)
    for t in (q, qt, dy, dyt):
        t._gpu = 0
    layer.w._gpu = layer.wt._gpu = 0
    d = sg.Dropout(0.5, 1)
    x, y, dx, dw, r = X.clone(), Y.clone(), X.clone(), torch.zeros(M, N), X.clone()
    return [(x, lambda: sg.sg_dropout(X, d, Y=x)), (r, lambda: sg.sg_dropout(X, d, residual=r, Y=r)),
            (x, lambda: sg.sg_dropout(x, d, Y=x)), (x, lambda: sg.sg_dequantize_f8(q, torch.float32, X_out=x)),
            (y, lambda: sg.sg_linear_f8(q, layer, Y=y)), (dx, lambda: sg.sg_linear_f8_grad_input(dy, layer, dX=dx)),
            (dw, lambda: sg.sg_linear_f8_grad_weight(dyt, qt, dW=dw)),
            (dw, lambda: sg.sg_linear_f8_grad_weight(dyt, qt, dW=dw, accumulate=True)),
            (q._store, lambda: sg.sg_quantize_f8(X, q=q)), (layer.w._store, lambda: sg.sg_pack_f8(dw, layer=layer))]


@pytest.mark.parametrize("case", range(10))
def test_autograd_hears_of_what_is_written(calls, case):
    t, call = _given(calls)[case]
    before = t._version
    call()
    assert t._version > before
    with torch.inference_mode():
        t, call = _given(calls)[case]
        call()
    assert len(calls) == 2
