"""The experts' operators where their numbers or sizes end."""
import pytest
import torch

from tests import experts_reference as ref
from tests.test_gpu_experts import int8_of, make, ok

pytestmark = pytest.mark.gpu

def check(got, want, bound, name):
    """ref.check, and the expected values have to be numbers themselves."""
    assert torch.isfinite(want).all() and torch.isfinite(bound).all(), f"{name}: the reference is not finite"
    ref.check(got, want, bound, name)


# ---- 8 bits: large values ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("top", [2.0**100, 2.0**121, 2.0**123, 2.0**127])
def test_quantize_rows_of_large_values(top):
    """Rows up to the largest bf16, where 127 times a value is beyond the largest float: the rule holds to the end."""
    import mixture_experts_rank_b200 as more
    g = torch.Generator(device="cuda").manual_seed(3)
    V = (torch.rand(64, 2096, generator=g, device="cuda") * 2 - 1).bfloat16() * top  # 2096: more than a lane keeps
    V[0, :4] = torch.tensor([1, 0.5, 0.25, 0], device="cuda").bfloat16() * top  # a half and a quarter of 127: both near a half
    V[0, 3] = 1
    V[1] = top
    V[2, 7] = torch.finfo(torch.bfloat16).max
    V[3, 5] = -torch.finfo(torch.bfloat16).max
    q, scale = more.quantize_rows(V)
    assert ok()
    want, sc, _ = ref.to_8_bits(V.double())
    assert torch.equal(q.double(), want)
    assert ((scale.double() - sc[:, 0]).abs() <= 2.0**-24 * sc[:, 0]).all()


# s = 64 and 80: the middle is rounded in the first product's epilogue, or behind it; 9 and 300 tokens: in the few-token
# kernel, or for the grouped products
EIGHT = [(N, 144, s, 8, 2) for N in (9, 300) for s in (64, 80)]


@pytest.mark.parametrize("size", EIGHT, ids=str)
def test_experts_int8_with_large_tokens(size):
    import mixture_experts_rank_b200 as more
    args, _ = make(*size)
    args["X"] = args["X"] * 2.0**121  # a token's largest is some 2^123; the products are of ordinary size
    args["W_up"] = args["W_up"] * 2.0**-121
    args = int8_of(args)
    out = more.experts_int8(**args)
    assert ok()
    check(out, *ref.forward(**args), "out")


@pytest.mark.parametrize("size", EIGHT, ids=str)
def test_experts_int8_with_a_large_middle(size):
    """a and b are 2^61 times ordinary values, silu(a) b up to some 2^126."""
    import mixture_experts_rank_b200 as more
    args, _ = make(*size)
    args["W_up"] = args["W_up"] * 2.0**61
    args["W_down"] = args["W_down"] * 2.0**-115
    args = int8_of(args)
    out = more.experts_int8(**args)
    assert ok()
    check(out, *ref.forward(**args), "out")
