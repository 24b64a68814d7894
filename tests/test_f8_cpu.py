"""Refusals of dropout and of the layer in 8-bit floating point: checked before
anything reaches a GPU, so pointers are made up."""

import ctypes

import pytest
import torch

P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(10)]
ODD = ctypes.c_void_p(0x100008)


@pytest.fixture(scope="module")
def sg():
    import os

    import post_pruning_amd as sg
    if not os.path.exists(sg.LIB_PATH):
        pytest.skip("libsg.so missing")
    sg.load_library()
    return sg


def _drop(sg, p=0.5, state=None):
    return ctypes.addressof(_drop.keep.setdefault((p, state), sg._DropStruct(p, 1, 2, state)))


_drop.keep = {}


def _refused(sg, status, code):
    assert status == code, (status, sg.sg_last_error_message())
    assert sg.sg_last_error_message()


@pytest.mark.parametrize("args,code", [
    (dict(n=0), 1), (dict(n=(1 << 20) + 1), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1),
    (dict(Y=None), 1), (dict(X=None), 1), (dict(drop=None), 1),
    (dict(dt=2), 2), (dict(ldx=99), 1), (dict(ldy=99), 1), (dict(ldr=99), 1),
    (dict(ldx=1 << 23), 2), (dict(Y=ctypes.c_void_p(0x100001)), 1),
    (dict(p=1.0), 1), (dict(p=-0.1), 1), (dict(p=float("nan")), 1), (dict(p=1 - 2.0 ** -34), 1),
    (dict(state=0x100004), 1),
])
def test_dropout_validation(sg, args, code):
    a = dict(Y=P[0], X=P[1], R=P[2], dt=1, T=5, n=100, ldy=100, ldx=100, ldr=100, p=0.5, state=None)
    a.update(args)
    drop = a["drop"] if "drop" in a else _drop(sg, a["p"], a["state"])
    _refused(sg, sg.load_library().sg_dropout(a["Y"], a["ldy"], a["X"], a["dt"], a["ldx"], a["R"], a["ldr"], a["T"], a["n"],
                                     drop, None), code)


@pytest.mark.parametrize("args,code", [
    (dict(n=0), 1), (dict(n=(1 << 20) + 1), 1), (dict(T=1 << 31), 1),
    (dict(X=None), 1), (dict(Q=None, Qt=None), 1), (dict(qs=None), 1), (dict(qts=None), 1),
    (dict(ldq=200), 1), (dict(ldq=128), 1), (dict(ldq=1 << 24), 1), (dict(Q=ODD), 2), (dict(qs=ODD), 2),
    (dict(ldqs=40), 1), (dict(ldqs=32), 1), (dict(ldqt=0), 1), (dict(ldqts=192), 1), (dict(T=(1 << 23) + 1), 1),
    (dict(fmt=2), 2), (dict(dt=5), 2), (dict(ldx=199), 1), (dict(drop=1.0), 1),
])
def test_quantize_validation(sg, args, code):
    a = dict(Q=P[0], ldq=256, qs=P[1], ldqs=48, Qt=P[2], ldqt=128, qts=P[3], ldqts=208, fmt=0, X=P[4], dt=1, T=40,
             n=200, ldx=200, drop=None)
    a.update(args)
    drop = None if a["drop"] is None else _drop(sg, a["drop"])
    _refused(sg, sg.load_library().sg_quantize_f8(a["Q"], a["ldq"], a["qs"], a["ldqs"], a["Qt"], a["ldqt"], a["qts"], a["ldqts"],
                                         a["fmt"], a["X"], a["dt"], a["T"], a["n"], a["ldx"], drop, None), code)


@pytest.mark.parametrize("args,code", [
    (dict(rows=-1), 1), (dict(cols=(1 << 23) + 1), 1), (dict(X=None), 1), (dict(Q=None), 1), (dict(s=None), 1),
    (dict(ldq=128), 1), (dict(lds=32), 1), (dict(fmt=-1), 2), (dict(dt=3), 2), (dict(ldx=199), 1),
    (dict(X=ctypes.c_void_p(0x100001)), 1),
])
def test_dequantize_validation(sg, args, code):
    a = dict(X=P[0], dt=0, ldx=200, Q=P[1], ldq=256, s=P[2], lds=48, fmt=1, rows=40, cols=200)
    a.update(args)
    _refused(sg, sg.load_library().sg_dequantize_f8(a["X"], a["dt"], a["ldx"], a["Q"], a["ldq"], a["s"], a["lds"], a["fmt"],
                                           a["rows"], a["cols"], None), code)


@pytest.mark.parametrize("args,code", [
    (dict(m=0), 1), (dict(n=65537), 1), (dict(Wq=None), 1), (dict(ws=None), 1), (dict(W=None), 1), (dict(wts=None), 1),
    (dict(ldw=128), 1), (dict(ldws=16), 1), (dict(ldwt=0), 1), (dict(ldwts=199), 1), (dict(dt=7), 2), (dict(ld=10), 1),
])
def test_pack_validation(sg, args, code):
    a = dict(Wq=P[0], ldw=256, ws=P[1], ldws=48, Wt=P[2], ldwt=128, wts=P[3], ldwts=208, W=P[4], dt=0, m=40, n=200,
             ld=200)
    a.update(args)
    _refused(sg, sg.load_library().sg_pack_f8(a["Wq"], a["ldw"], a["ws"], a["ldws"], a["Wt"], a["ldwt"], a["wts"], a["ldwts"],
                                     a["W"], a["dt"], a["m"], a["n"], a["ld"], None), code)


_PRODUCT = dict(out=P[0], dt=1, ldo=None, Q=P[1], ldq=None, qs=P[2], ldqs=64, fmt=0, T=40, A=P[3], lda=None, as_=P[4],
                ldas=320, m=300, n=200, ws=ctypes.c_void_p(0x40000000), nb=1 << 40)


@pytest.mark.parametrize("call", ["linear", "grad_input", "grad_weight"])
@pytest.mark.parametrize("args,code", [
    (dict(m=0), 1), (dict(m=(1 << 20) + 1), 1), (dict(n=0), 1), (dict(n=65537), 1), (dict(T=-1), 1), (dict(T=1 << 31), 1),
    (dict(out=None), 1), (dict(Q=None), 1), (dict(qs=None), 1), (dict(A=None), 1), (dict(as_=None), 1),
    (dict(dt=2), 2), (dict(fmt=2), 2), (dict(ldo=7), 1), (dict(ldq=100), 1), (dict(ldq=64), 1), (dict(lda=1 << 24), 1),
    (dict(ldqs=8), 1), (dict(ldas=31), 1), (dict(Q=ODD), 2), (dict(as_=ODD), 2),
])
def test_product_validation(sg, call, args, code):
    lib, a = sg.load_library(), dict(_PRODUCT)
    # codes [T, n] and [m, n]; [T, m] and [n, m]; [m, T] and [n, T]
    k = dict(linear=256, grad_input=384, grad_weight=128)[call]
    a["ldq"] = a["lda"] = k
    a["ldo"] = 300 if call == "linear" else 200
    a["ldqs"] = 304 if call == "grad_weight" else 64
    a.update(args)
    head = (a["out"], a["dt"], a["ldo"])
    q = (a["Q"], a["ldq"], a["qs"], a["ldqs"], a["fmt"])
    w = (a["A"], a["lda"], a["as_"], a["ldas"])
    if call == "linear":
        st = lib.sg_linear_f8(*head, *q, a["T"], *w, a["m"], a["n"], a["ws"], a["nb"], None)
    elif call == "grad_input":
        st = lib.sg_linear_f8_grad_input(*head, *q, a["T"], *w, a["m"], a["n"], None, a["ws"], a["nb"], None)
    else:
        st = lib.sg_linear_f8_grad_weight(*head, 0, *q, *w, a["T"], None, a["m"], a["n"], a["ws"], a["nb"], None)
    _refused(sg, st, code)


def test_grad_input_refuses_a_bad_dropout(sg):
    st = sg.load_library().sg_linear_f8_grad_input(P[0], 1, 200, P[1], 384, P[2], 48, 0, 40, P[3], 384, P[4], 208, 300, 200,
                                          _drop(sg, 1.5), ctypes.c_void_p(0x40000000), 1 << 40, None)
    _refused(sg, st, sg.SG_ERR_INVALID_ARGUMENT)


def test_weight_gradient_token_limit(sg):
    T = (1 << 23) + 1
    st = sg.load_library().sg_linear_f8_grad_weight(P[0], 1, 200, 0, P[1], 1 << 24, P[2], 304, 0, P[3], 1 << 24, P[4], 208, T,
                                           None, 300, 200, None, 0, None)
    _refused(sg, st, sg.SG_ERR_INVALID_ARGUMENT)


def test_workspace_bytes(sg):
    for op in (sg.SG_OP_LINEAR_F8, sg.SG_OP_F8_GRAD_INPUT, sg.SG_OP_F8_GRAD_WEIGHT):
        for bad in ((0, 5, 5), (5, 0, 5), (5, 5, -1), (5, 65537, 5), ((1 << 20) + 1, 5, 5), (5, 5, 1 << 31), (5, 5, 0)):
            assert sg.sg_workspace_bytes(op, *bad) == 0
        for T in (1, 7, 64, 500, 4096, 1 << 20):
            for m, n in ((1, 1), (300, 200), (4096, 4096), (1 << 20, 128), (64, 65536)):
                # the partial sums of at most two tiles of 256 x 256 a compute unit
                assert 0 <= sg.sg_workspace_bytes(op, m, n, T) <= 512 * 256 * 256 * 4


def test_workspace_is_checked(sg):
    lib = sg.load_library()
    m, n, T = 4096, 4096, 100
    need = sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, m, n, T)
    if need:
        for ws, nb, code in ((None, need, 3), (P[5], need - 1, 3), (ctypes.c_void_p(0x40000010), need, 1)):
            _refused(sg, lib.sg_linear_f8(P[0], 1, m, P[1], n, P[2], 112, 0, T, P[3], n, P[4], m, m, n, ws, nb, None), code)


def test_dropout_objects(sg):
    for p in (1.0, -0.5, float("nan"), 1 - 2.0 ** -34):
        with pytest.raises(ValueError):
            sg.Dropout(p, 1)
    with pytest.raises(ValueError):
        sg.Dropout(0.5, 1, state=torch.zeros(2, dtype=torch.int64))  # not on the GPU
    with pytest.raises(ValueError):
        sg.Dropout(0.5, 1, state=torch.zeros(3, dtype=torch.int64))
    d = sg.Dropout(0.25, -1, 2 ** 64 + 5)
    assert (d.seed, d.offset) == (2 ** 64 - 1, 5)


def test_binding_refuses_cpu_tensors(sg):
    X = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        sg.sg_dropout(X, sg.Dropout(0.5, 1))
    with pytest.raises(ValueError):
        sg.sg_quantize_f8(X)
    with pytest.raises(ValueError):
        sg.sg_pack_f8(X)
    with pytest.raises(ValueError):
        sg.F8Tensor(X.to(torch.float8_e4m3fn), torch.zeros(1, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sg.F8Tensor(X, torch.zeros(1, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):
        sg.linear_f8(X, None)
    with pytest.raises(ValueError):
        sg.linear_f8(X, torch.zeros(8, 64))
    with pytest.raises(TypeError):
        sg.linear_f8(X.half(), torch.zeros(8, 128))
    with pytest.raises(ValueError):
        sg.linear_f8(X, torch.zeros(8, 128), grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        sg.dropout(X, sg.Dropout(0.5, 1), residual=X[:2])


def test_a_layer_lives_on_one_gpu(sg):
    def matrix(rows, cols, gpu):  # no memory: only what the check looks at
        t = sg.F8Tensor.__new__(sg.F8Tensor)
        t.rows, t.cols, t.format, t._gpu = rows, cols, sg.SG_E4M3, gpu
        return t

    assert sg.F8Layer(matrix(40, 200, 1), matrix(200, 40, 1)).m == 40
    with pytest.raises(ValueError):
        sg.F8Layer(matrix(40, 200, 0), matrix(200, 40, 1))
    with pytest.raises(ValueError):
        sg.F8Layer(matrix(40, 200, 0), matrix(40, 200, 0))
