"""How the binding of the 8-bit linear layer reads the strides of its operands."""

import pytest
import torch

import post_pruning_amd as sg

BF16 = torch.bfloat16


@pytest.mark.parametrize("n", [1, 7, 64, 4096])
@pytest.mark.parametrize("stride", [1, 5000, 1 << 23, 1 << 33])
def test_a_single_row_has_no_pitch(n, stride):
    # as the last position of a prompt has it: hidden[:, -1, :] of [1, S, n]
    X = torch.empty(n, dtype=BF16).as_strided((1, n), (stride, 1))
    code, pitch = sg._rows(X, "X", 1, n)
    assert code == sg.SG_BF16 and n <= pitch <= n + 7 and pitch * 2 <= sg.SG_MAX_PITCH
    q = torch.empty(4096, dtype=torch.int8).as_strided((1, n), (stride, 1))
    rows, cols, pitch = sg._codes(q, "q")
    assert (rows, cols, pitch) == (1, n, -(-n // 64) * 64)
    assert sg._as_rows(X).data_ptr() == X.data_ptr()  # nothing is copied


def test_rows_too_far_apart_are_copied():
    # hidden[:, -1, :] of [4, 2048, 4096]: rows 2^24 bytes apart
    far = torch.empty_strided((4, 8), (1 << 23, 1), dtype=BF16, device="meta")
    near = torch.empty_strided((4, 8), (1 << 22, 1), dtype=BF16, device="meta")
    assert sg._as_rows(far).stride(0) == 8
    assert sg._as_rows(near).stride(0) == 1 << 22
    assert sg._as_rows(torch.empty_strided((4, 8), (1 << 22, 1), device="meta")).stride(0) == 8  # fp32
    assert sg._as_rows(torch.empty(8, dtype=BF16).expand(4, 8)).stride(0) == 8  # expanded


@pytest.mark.parametrize("m", [1, 5])
def test_a_layer_s_padding_holds_zeros(m):
    # behind a column slice lie other weights, which the product would count
    wide = torch.zeros(m, 256, dtype=torch.int8)
    offset, scale = torch.zeros(m, dtype=torch.int32), torch.ones(m)
    layer = sg.W8Layer(wide[:, :100], offset, scale)
    assert (layer.m, layer.n) == (m, 100)
    wide[:, 128:] = 9  # past the padded width nothing is read
    wide[:, :100] = 5
    sg.W8Layer(wide[:, :100], offset, scale)
    for col in (100, 127):
        wide[m - 1, col] = 1
        with pytest.raises(ValueError, match="zeros"):
            sg.W8Layer(wide[:, :100], offset, scale)
        wide[m - 1, col] = 0
    sg.W8Layer(wide[:, :64], offset, scale)  # whole pieces need none
