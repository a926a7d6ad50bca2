"""The experts' operators where their numbers or sizes end."""
import pytest
import torch

from tests import experts_reference as ref
from tests.test_gpu_experts import int8_of, layer_inputs, make, ok, rnd

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


# ---- 8 bits: no numbers ----------------------------------------------------------------------------------------------
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("width", [32, 2096])
def test_quantize_rows_keeps_what_is_no_number_in_the_scale(width):
    import mixture_experts_rank_b200 as more
    g = torch.Generator(device="cuda").manual_seed(4)
    V = rnd(g, 40, width)
    want, wscale = more.quantize_rows(V)
    odd = {3: [(5, INF)], 9: [(0, -INF), (width - 1, INF)], 11: [(width - 2, NAN)], 20: [(1, INF), (width - 3, NAN)],
           39: [(7, -NAN)]}
    for row, entries in odd.items():
        for at, v in entries:
            V[row, at] = v
    q, scale = more.quantize_rows(V)
    assert ok()
    plain = torch.ones(40, dtype=torch.bool, device="cuda")
    plain[list(odd)] = False
    assert torch.equal(q[plain], want[plain]) and torch.equal(scale[plain], wscale[plain])
    for row, entries in odd.items():
        if any(v != v for _, v in entries):  # a NaN: no value of the row is known
            assert scale[row].isnan() and (q[row] == 0).all()
        else:  # an infinity: the finite values are nothing next to it
            of = torch.zeros(width, dtype=torch.int8, device="cuda")
            for at, v in entries:
                of[at] = 127 if v > 0 else -127
            assert scale[row] == INF and torch.equal(q[row], of)


@pytest.mark.parametrize("size", EIGHT, ids=str)
def test_not_a_number_stays_with_its_token_in_8_bits(size):
    import mixture_experts_rank_b200 as more
    args = int8_of(make(*size)[0])
    clean = more.experts_int8(**args)
    X = args["X"].clone()
    X[1, 3], X[4, 5], X[8, 0] = NAN, INF, -INF
    out = more.experts_int8(**dict(args, X=X))
    assert ok()
    keep = torch.ones(size[0], dtype=torch.bool, device="cuda")
    keep[[1, 4, 8]] = False
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[~keep]).any() and out[1].isnan().all()


@pytest.mark.parametrize("N", [3, 200])
@pytest.mark.parametrize("s", [16, 80])
def test_an_infinite_middle_in_8_bits_gives_infinity(N, s):
    """The middle overflows to infinity in one column (a, b = 6.4e21 there) and is an ordinary number in the others."""
    import mixture_experts_rank_b200 as more
    args, _ = make(N, 64, s, 1, 1)
    args["X"].fill_(1.0)
    args["W_up"].fill_(2.0**-6)
    args["W_up"][:, [5, s + 5]] = 1e20
    args["W_down"].fill_(0.5)
    args["W_down"][:, 32:] = -0.5
    out = more.experts_int8(**int8_of(args))
    assert ok()
    assert (out[:, :32] == INF).all() and (out[:, 32:] == -INF).all()


def test_layer_in_8_bits_of_a_token_that_is_no_number():
    import mixture_experts_rank_b200 as more
    a = int8_of(layer_inputs(9, 128, 16, 32, 16))
    clean = more.moe_layer_int8(**a, k=3)
    X = a["X"].clone()
    X[4, 7] = NAN  # no logit of it is a number: it selects nothing
    out = more.moe_layer_int8(**dict(a, X=X), k=3)
    torch.cuda.synchronize()
    assert more.device_status() != 0
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(out[keep], clean[keep]) and (out[4] == 0).all()
