"""Few rows over a long contraction in 8-bit floating point: the product is
divided over the chip.  (What a call needs as workspace tells whether it is.)"""

import os

import pytest

import post_pruning_amd as sg

pytestmark = pytest.mark.skipif(not os.path.exists(sg.LIB_PATH), reason="libsg.so missing")


@pytest.mark.parametrize("m,n,T", [(16, 64, 1 << 20), (1, 64, 1 << 23), (16, 2048, 1 << 17), (17, 64, 1 << 17),
                                   (64, 64, 16384), (50, 16, 1 << 17)])
def test_long_contractions_are_split(m, n, T):
    assert sg.sg_workspace_bytes(sg.SG_OP_F8_GRAD_WEIGHT, m, n, T) > 0


def test_input_gradient_of_many_outputs_is_split():
    assert sg.sg_workspace_bytes(sg.SG_OP_F8_GRAD_INPUT, 1 << 20, 64, 16) > 0
    assert sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, 64, 65536, 3) > 0


@pytest.mark.parametrize("m,n,T", [(4096, 4096, 1), (8192, 28672, 16), (64, 4096, 1), (11008, 4096, 1), (4096, 4096, 32)])
def test_weights_are_streamed_for_few_tokens(m, n, T):
    assert sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, m, n, T) == 0


def test_workspaces_of_the_refusals():
    # the sizes whose too small workspaces other tests refuse need one
    assert sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, 4096, 4096, 100) > 0
    assert sg.sg_workspace_bytes(sg.SG_OP_LINEAR_F8, 4489, 8192, 70) > 0
