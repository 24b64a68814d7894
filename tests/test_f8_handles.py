"""Handles of dropout and of the layer in 8-bit floating point: what they say is
what the library takes."""

import copy
import ctypes
import pickle

import pytest
import torch

import post_pruning_amd as sg


def _struct(d):
    return sg._DropStruct.from_address(sg._drop_address(d))


@pytest.mark.parametrize("name,value", [("p", 0.0), ("seed", 3), ("offset", 9), ("state", None)])
def test_a_dropout_does_not_change(name, value):
    d = sg.Dropout(0.25, 7, 5)
    with pytest.raises(AttributeError):
        setattr(d, name, value)
    with pytest.raises(AttributeError):
        delattr(d, name)
    s = _struct(d)
    assert (d.p, d.seed, d.offset, d.state) == (0.25, 7, 5, None) == (s.p, s.seed, s.offset, s.state)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda d: pickle.loads(pickle.dumps(d))])
def test_copies_of_a_dropout(how):
    d = sg.Dropout(0.25, 2 ** 64 - 1, 2 ** 63 + 5)
    e = how(d)
    assert e is not d and type(e) is sg.Dropout
    address = sg._drop_address(e)
    assert address != sg._drop_address(d)
    del d
    s = _struct(e)
    assert (e.p, e.seed, e.offset, e.state) == (0.25, 2 ** 64 - 1, 2 ** 63 + 5, None) == (s.p, s.seed, s.offset, s.state)


def test_a_module_that_holds_one_is_copied():
    m = torch.nn.Linear(4, 4)
    m.drop = sg.Dropout(0.5, 1, 2)
    other = copy.deepcopy(m)
    assert other.drop is not m.drop and other.drop.offset == 2
    assert ctypes.sizeof(sg._DropStruct) == 32


def _matrix(rows, cols):
    return sg.F8Tensor._unwritten(rows, cols, torch.float8_e4m3fn, torch.empty(1))


@pytest.mark.parametrize("name", ["w", "wt", "m", "n"])
def test_the_parts_of_a_layer_stay(name):
    w, wt = _matrix(40, 200), _matrix(200, 40)
    layer = sg.F8Layer(w, wt)
    with pytest.raises(AttributeError):
        setattr(layer, name, _matrix(8, 200) if name in ("w", "wt") else 8)
    assert layer.w is w and layer.wt is wt and (layer.m, layer.n) == (40, 200)


@pytest.mark.parametrize("how", [copy.deepcopy, lambda t: pickle.loads(pickle.dumps(t))])
@pytest.mark.parametrize("cols", [200, 256])
@pytest.mark.parametrize("whole", [True, False])
def test_copies_of_a_matrix_lie_elsewhere(how, cols, whole):
    t = _matrix(40, cols)
    t._store.random_(0, 120)
    if not whole:  # codes and scale in tensors of their own
        t = sg.F8Tensor._of(*(v.clone() for v in t._wide()), 40, cols)
    c = how(t)
    assert (c.rows, c.cols, c.pitch, c.scale_pitch, c.format, c.dtype, c._gpu) == \
        (t.rows, t.cols, t.pitch, t.scale_pitch, t.format, t.dtype, t._gpu)
    assert torch.equal(c.codes.view(torch.uint8), t.codes.view(torch.uint8)) and torch.equal(c.scale, t.scale)
    assert c._args == (c.codes.data_ptr(), c.pitch, c.scale.data_ptr(), c.scale_pitch)
    assert c._args[0] != t._args[0] and c._args[2] != t._args[2]


def test_copies_of_a_layer():
    layer = sg.F8Layer(_matrix(40, 200), _matrix(200, 40))
    deep, shallow = copy.deepcopy(layer), copy.copy(layer)
    assert (deep.m, deep.n) == (40, 200) and shallow.w is layer.w
    for a, b in ((deep.w, layer.w), (deep.wt, layer.wt)):
        assert a._args[0] == a.codes.data_ptr() != b._args[0]
    t = copy.copy(layer.w)
    assert t._args == layer.w._args


def test_the_state_of_a_dropout_is_its_version_and_memory():
    d = sg.Dropout(0.5, 1)
    before = d._version()
    assert d._version() == before
    d._state = torch.zeros(2, dtype=torch.int64)  # (a public one has to live on the GPU)
    seen = {before, d._version()}
    d._state.add_(1)
    seen.add(d._version())
    old = d._state.data
    d._state.data = torch.zeros(2, dtype=torch.int64)
    seen.add(d._version())
    assert len(seen) == 4 and old is not None
