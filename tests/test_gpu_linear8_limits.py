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
