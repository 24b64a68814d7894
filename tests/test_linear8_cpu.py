"""Refusals of the 8-bit linear layer's calls, and their workspace sizes.

Nothing here runs a kernel: every C call below fails validation or stops at
the device check, every Python call before it reaches the library.
"""

import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_pruning_amd", "libsg.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libsg.so not built")

P = 0x100000  # a device-looking, aligned address that nothing reads


@pytest.fixture(scope="module")
def sg():
    import post_pruning_amd as sg
    sg.load_library()
    return sg


F32, BF16 = 0, 1
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3

QUANT = dict(Q=P, ldq=128, scale=P, sum=P, X=P, x_dtype=BF16, T=4, n=100, ldx=104, stream=None)
DEQUANT = dict(X=P, x_dtype=BF16, ldx=104, Q=P, ldq=128, scale=P, T=4, n=100, stream=None)
PACK = dict(Wq=P, ldw=128, off=P, w_scale=P, codes=P, scale=P, zero=P, m=8, n=100, stream=None)
BIG = 1 << 40
LINEAR = dict(Y=P, y_dtype=F32, ldy=8, Q=P, ldq=128, xs=P, xsum=P, T=4, Wq=P, ldw=128, off=P, ws=P, m=8, n=100,
              workspace=P, ws_bytes=BIG, stream=None)
GRADX = dict(dX=P, dx_dtype=F32, lddx=100, dY=P, dy_dtype=BF16, lddy=8, T=4, Wq=P, ldw=128, off=P, ws=P, m=8,
             n=100, workspace=P, ws_bytes=BIG, stream=None)
GRADW = dict(dW=P, dw_dtype=F32, lddw=100, accumulate=0, dY=P, dy_dtype=BF16, lddy=8, Q=P, ldq=128, xs=P, T=4,
             mask=P, m=8, n=100, workspace=P, ws_bytes=BIG, stream=None)

BAD = [
    ("sg_quantize_tokens", QUANT, dict(Q=None), INVALID),
    ("sg_quantize_tokens", QUANT, dict(X=None), INVALID),
    ("sg_quantize_tokens", QUANT, dict(scale=None), INVALID),
    ("sg_quantize_tokens", QUANT, dict(sum=None), INVALID),
    ("sg_quantize_tokens", QUANT, dict(n=0), INVALID),
    ("sg_quantize_tokens", QUANT, dict(n=65537, ldx=65537, ldq=1 << 17), INVALID),
    ("sg_quantize_tokens", QUANT, dict(T=-1), INVALID),
    ("sg_quantize_tokens", QUANT, dict(T=1 << 31), INVALID),
    ("sg_quantize_tokens", QUANT, dict(ldq=100), UNSUPPORTED),
    ("sg_quantize_tokens", QUANT, dict(ldq=64), INVALID),
    ("sg_quantize_tokens", QUANT, dict(ldq=(1 << 23) + 64), INVALID),
    ("sg_quantize_tokens", QUANT, dict(Q=P + 8), UNSUPPORTED),
    ("sg_quantize_tokens", QUANT, dict(ldx=99), INVALID),
    ("sg_quantize_tokens", QUANT, dict(ldx=1 << 23), UNSUPPORTED),
    ("sg_quantize_tokens", QUANT, dict(x_dtype=2), UNSUPPORTED),
    ("sg_quantize_tokens", QUANT, dict(X=P + 1), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(X=None), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(Q=None), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(scale=None), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(x_dtype=7), UNSUPPORTED),
    ("sg_dequantize_tokens", DEQUANT, dict(x_dtype=F32, X=P + 2), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(ldx=96), INVALID),
    ("sg_dequantize_tokens", DEQUANT, dict(ldq=96), UNSUPPORTED),
    ("sg_pack_w8", PACK, dict(Wq=None), INVALID),
    ("sg_pack_w8", PACK, dict(zero=None), INVALID),
    ("sg_pack_w8", PACK, dict(m=0), INVALID),
    ("sg_pack_w8", PACK, dict(m=(1 << 20) + 1), INVALID),
    ("sg_pack_w8", PACK, dict(ldw=120), UNSUPPORTED),
    ("sg_linear_w8a8", LINEAR, dict(Y=None), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(xsum=None), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(Wq=None), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(Wq=P + 4), UNSUPPORTED),
    ("sg_linear_w8a8", LINEAR, dict(ldw=64), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(ldq=96), UNSUPPORTED),
    ("sg_linear_w8a8", LINEAR, dict(ldy=7), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(y_dtype=5), UNSUPPORTED),
    ("sg_linear_w8a8", LINEAR, dict(m=(1 << 20) + 1, ldy=(1 << 20) + 1), INVALID),
    ("sg_linear_w8a8", LINEAR, dict(workspace=P + 16), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(dX=None), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(dY=None), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(dy_dtype=F32), UNSUPPORTED),
    ("sg_linear_w8_grad_input", GRADX, dict(lddy=7), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(lddx=99), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(ws=None), INVALID),
    ("sg_linear_w8_grad_input", GRADX, dict(ws_bytes=16), WORKSPACE),
    ("sg_linear_w8_grad_input", GRADX, dict(workspace=None), WORKSPACE),
    ("sg_linear_w8_grad_weight", GRADW, dict(dW=None), INVALID),
    ("sg_linear_w8_grad_weight", GRADW, dict(Q=None), INVALID),
    ("sg_linear_w8_grad_weight", GRADW, dict(xs=None), INVALID),
    ("sg_linear_w8_grad_weight", GRADW, dict(dy_dtype=F32), UNSUPPORTED),
    ("sg_linear_w8_grad_weight", GRADW, dict(dw_dtype=3), UNSUPPORTED),
    ("sg_linear_w8_grad_weight", GRADW, dict(lddw=99), INVALID),
    ("sg_linear_w8_grad_weight", GRADW, dict(Q=P + 32 + 8), UNSUPPORTED),
    ("sg_linear_w8_grad_weight", GRADW, dict(ws_bytes=0), WORKSPACE),
]


@pytest.mark.parametrize("call,good,change,want", BAD,
                         ids=[f"{c[3:]}-{'-'.join(f'{k}' for k in ch)}-{i}" for i, (c, _, ch, _) in enumerate(BAD)])
def test_refusals(sg, call, good, change, want):
    lib = sg.load_library()
    args = dict(good, **change)
    assert set(args) == set(good)
    assert getattr(lib, call)(*args.values()) == want
    assert sg.sg_last_error_message()


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no memory")
@pytest.mark.parametrize("call,good", [("sg_quantize_tokens", QUANT), ("sg_dequantize_tokens", DEQUANT),
                                       ("sg_pack_w8", PACK), ("sg_linear_w8a8", LINEAR),
                                       ("sg_linear_w8_grad_input", GRADX), ("sg_linear_w8_grad_weight", GRADW)])
def test_good_arguments_reach_the_device_check(sg, call, good):
    # without a gfx950 device the same arguments stop there and nowhere before
    assert getattr(sg.load_library(), call)(*good.values()) in (2, 4)
    assert "device" in sg.sg_last_error_message()


def test_workspace_sizes(sg):
    for op in (sg.SG_OP_LINEAR_W8A8, sg.SG_OP_GRAD_INPUT, sg.SG_OP_GRAD_WEIGHT):
        for bad in ((0, 8, 8), (8, 0, 8), (8, 8, -1), ((1 << 20) + 1, 8, 8), (8, 65537, 8), (8, 8, 1 << 31)):
            assert sg.sg_workspace_bytes(op, *bad) == 0
        for good in ((1, 1, 1), (130, 1000, 3000), (11008, 4096, 8192), (65536, 65536, 1 << 20), (1 << 20, 65536, 1 << 20)):
            assert sg.sg_workspace_bytes(op, *good) % 256 == 0


def test_python_refusals(sg):
    X = torch.zeros(4, 100, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        sg.sg_quantize_tokens(X)
    q = torch.zeros(4, 128, dtype=torch.int8)[:, :100]
    with pytest.raises(ValueError, match="GPU"):
        sg.sg_dequantize_tokens(q, torch.ones(4))
    layer = sg.W8Layer(torch.zeros(8, 128, dtype=torch.int8)[:, :100], torch.zeros(8, dtype=torch.int32),
                       torch.ones(8))
    with pytest.raises(ValueError, match="GPU"):
        sg.sg_linear_w8a8(q, torch.ones(4), torch.zeros(4, dtype=torch.int32), layer)
    with pytest.raises(ValueError, match="GPU"):
        sg.sg_linear_w8_grad_input(torch.zeros(4, 8, dtype=torch.bfloat16), layer)
    with pytest.raises(ValueError, match="GPU"):
        sg.sg_linear_w8_grad_weight(torch.zeros(4, 8, dtype=torch.bfloat16), q, torch.ones(4))
    with pytest.raises(ValueError, match="columns"):
        sg.linear_w8(torch.zeros(4, 99), None, layer)
    with pytest.raises(TypeError):
        sg.linear_w8(torch.zeros(4, 100, dtype=torch.float64), None, layer)
    with pytest.raises(TypeError, match="bfloat16"):
        sg.linear_w8(torch.zeros(4, 100, requires_grad=True), None, layer)
    with pytest.raises(ValueError, match="W must"):
        sg.linear_w8(X, torch.zeros(8, 99), layer)
    with pytest.raises(ValueError, match="mask"):
        sg.linear_w8(X, None, layer, mask=torch.zeros(8, 100, dtype=torch.bool))


def test_code_rows_need_their_padding(sg):
    # the padded width of the last row has to lie in the storage
    tight = torch.zeros(4, 100, dtype=torch.int8)
    with pytest.raises(ValueError, match="padded"):
        sg._codes(tight, "q")
    with pytest.raises(ValueError, match="row-major"):
        sg._codes(torch.zeros(128, 4, dtype=torch.int8).t(), "q")
    assert sg._codes(torch.zeros(4, 128, dtype=torch.int8)[:, :100], "q") == (4, 100, 128)
    assert sg._codes(torch.zeros(4, 128, dtype=torch.int8)[1:3, :100], "q") == (2, 100, 128)
    # a column slice that runs out of the last row
    with pytest.raises(ValueError, match="padded"):
        sg._codes(torch.zeros(4, 128, dtype=torch.int8)[:, 64 + 32:], "q")
