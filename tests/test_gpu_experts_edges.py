"""The experts' operators where their numbers or sizes end."""
import math

import pytest
import torch

from tests import experts_reference as ref
from tests.parity import FINE_TOL
from tests.test_gpu_experts import guarded, int8_of, layer_inputs, layer_reference, make, masked, ok, rnd

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


# ---- few tokens of any h ---------------------------------------------------------------------------------------------
# N, h, r, s, M, k.  Sums of all selections of 64 tokens take one CTA's shared memory at k h of some 40000; the sizes lie
# on both sides, up to several times it.  The bounds are those of a call that carries the rows in fp32 throughout.
WIDE = [(64, 4096, 32, 16, 64, 8), (36, 7168, 32, 16, 64, 8), (37, 7168, 32, 16, 64, 8), (64, 7168, 32, 80, 64, 8),
        (18, 7168, 16, 16, 64, 16), (64, 6000, 16, 16, 40, 16), (64, 20016, 16, 16, 24, 16), (2, 131072, 16, 16, 8, 2),
        (64, 40000, 16, 16, 16, 2), (64, 2064, 16, 48, 16, 16)]


def layer_check(out, args, k, **scales):
    """The layer against the experts in 64 bits with more.route's gates.  The few-token kernel has a router of its own, and
    each router's logits may be off by t = FINE_TOL of the token's rms (tests/parity.py; mostly z as a bf16 pair).  Logits
    that differ by 2 t change a gate e^l_j / sum e^l_i by a factor of at most e^(4 t), so the result by as much of the
    sum of its terms' magnitudes."""
    import mixture_experts_rank_b200 as more
    want, bound = layer_reference(args, k, True, **scales)
    idx, gate, _, _ = more.route(args["X"], args["R1"], args["R2"], k)
    offsets, slots = more.dispatch(idx, args["W_down"].shape[0])
    terms = sum(ref.forward(args["X"], args["W_up"], args["W_down"], gate * one, offsets, slots, fp32_rows=True, **scales)[0].abs()
                for one in torch.eye(k, device="cuda"))
    rms = (args["X"].double() @ args["R1"].double() @ args["R2"].double()).square().mean(1, keepdim=True).sqrt()
    check(out, want, bound + torch.expm1(4 * FINE_TOL * rms) * terms, "out")


@pytest.mark.parametrize("size", WIDE, ids=str)
def test_layer_of_wide_tokens(size):
    import mixture_experts_rank_b200 as more
    N, h, r, s, M, k = size
    args = layer_inputs(N, h, r, s, M)
    out, untouched = guarded((N, h), torch.bfloat16)
    more.moe_layer(**args, k=k, out=out)
    assert ok() and untouched()
    layer_check(out, args, k)


@pytest.mark.parametrize("size", WIDE, ids=str)
def test_layer_of_wide_tokens_in_8_bits(size):
    import mixture_experts_rank_b200 as more
    N, h, r, s, M, k = size
    args = int8_of(layer_inputs(N, h, r, s, M))
    out, untouched = guarded((N, h), torch.bfloat16)
    more.moe_layer_int8(**args, k=k, out=out)
    assert ok() and untouched()
    layer_check(out, args, k, **{n: args[n] for n in ("up_scale", "down_scale")})


# N, h, s, M, k; up to 16 tokens of any h, and others with N k <= M up to N k h = 2^21: the third lies on it, the last
# behind it, where each slot's row is rounded to bf16
FEW = [(16, 30000, 16, 16, 16), (16, 7168, 48, 4, 4), (64, 4096, 16, 512, 8), (18, 7280, 32, 300, 16),
       (64, 4112, 16, 512, 8)]


@pytest.mark.parametrize("size", FEW, ids=str)
def test_experts_of_few_wide_tokens(size):
    import mixture_experts_rank_b200 as more
    args, _ = make(*size)
    fp32_rows = size != FEW[-1]
    out, untouched = guarded(size[:2], torch.bfloat16)
    more.experts(**args, out=out)
    assert ok() and untouched()
    check(out, *ref.forward(**args, fp32_rows=fp32_rows), "out")
    args = int8_of(args)
    more.experts_int8(**args, out=out)
    assert ok() and untouched()
    check(out, *ref.forward(**args, fp32_rows=fp32_rows), "out in 8 bits")


def test_layer_in_8_bits_of_more_tokens_is_the_three_calls():
    import mixture_experts_rank_b200 as more
    a = int8_of(layer_inputs(130, 256, 32, 80, 32))
    idx, gate, _, _ = more.route(a["X"], a["R1"], a["R2"], 4)
    offsets, slots = more.dispatch(idx, 32)
    want = more.experts_int8(a["X"], a["W_up"], a["up_scale"], a["W_down"], a["down_scale"], gate, offsets, slots)
    assert torch.equal(more.moe_layer_int8(**a, k=4), want) and ok()


# ---- what counts for nothing -------------------------------------------------------------------------------------------
@pytest.mark.parametrize("size", [(9, 72, 24, 16, 3), (300, 72, 24, 16, 3), (600, 320, 712, 3, 2)], ids=str)
def test_backward_with_gates_of_selections_that_nobody_lists(size):
    import mixture_experts_rank_b200 as more
    N, k = size[0], size[4]
    args, d = make(*size)
    drop = list(range(k)) + [2 * k + 1]  # token 0 keeps nothing, token 2 loses one
    args = masked(args, drop)
    gate = args["gate"].clone()
    gate.view(-1)[drop] = 0.0  # what such a gate comes to
    args["gate"].view(-1)[drop] = torch.tensor([NAN, INF, -INF, NAN], device="cuda")[-len(drop):]
    got = more.experts_backward(**args, out_bar=d)
    assert ok()
    want, bound = ref.backward(**dict(args, gate=gate), out_bar=d)
    for name, t in zip(want, got):
        if name == "logits_bar":  # a selection that is not listed has its own gate as a factor
            listed = torch.ones(N * k, dtype=torch.bool, device="cuda")
            listed[drop] = False
            t, want[name], bound[name] = (v.reshape(-1)[listed] for v in (t, want[name], bound[name]))
        check(t, want[name], bound[name], name)


@pytest.mark.parametrize("size", [(50, 64, 16, 8, 2), (400, 136, 200, 8, 2), (600, 320, 712, 3, 2)], ids=str)
def test_a_slot_out_of_range_brings_in_no_token(size):
    """A slot outside [0, N k) is skipped: an expert that lists one takes nothing of any token by it, whatever that token
    holds."""
    import mixture_experts_rank_b200 as more
    N, h, s, M, k = size
    args, d = make(*size)
    X, d = args["X"].clone(), d.clone()
    X[0], d[0] = NAN, NAN
    slots, ends = args["slots"].clone(), args["offsets"].tolist()
    mine = {e for e in range(M) if (slots[ends[e]:ends[e + 1]] // k == 0).any()}  # experts of token 0
    others = [e for e in range(M) if e not in mine and ends[e + 1] - ends[e] > 2]
    lost = []
    for e, value in zip(others[:2], (N * k, -3)):
        for at in (ends[e], ends[e + 1] - 1):  # the first, and the one that padding follows
            lost.append(int(slots[at]))
            slots[at] = value
    assert lost
    got = more.experts_backward(**dict(args, X=X, slots=slots), out_bar=d)
    torch.cuda.synchronize()
    assert more.device_status() != 0
    gate = args["gate"].clone()
    gate.view(-1)[lost] = 0
    clean = dict(args, gate=gate)
    clean["X"], dd = X.clone(), d.clone()
    clean["X"][0], dd[0] = 0, 0
    want, bound = ref.backward(**clean, out_bar=dd)
    for i, name in ((1, "W_up_bar"), (2, "W_down_bar")):
        check(got[i][others], want[name][others], bound[name][others], name)
    check(got[0][1:], want["X_bar"][1:], bound["X_bar"][1:], "X_bar")


@pytest.mark.parametrize("size", [(50, 64, 16, 8, 2), (400, 136, 200, 8, 2), (600, 320, 712, 3, 2)], ids=str)
def test_an_infinite_gradient_stays_infinite(size):
    """Rows are laid out in sixteens: what fills an expert's last one up has to add nothing, not zero times infinity."""
    import mixture_experts_rank_b200 as more
    N, h, s, M, k = size
    args, d = make(*size)
    d = d.clone()
    e = int(torch.nonzero(args["offsets"].diff() % 16)[0])  # an expert whose rows do not fill their last sixteen
    d[int(args["slots"][args["offsets"][e + 1] - 1]) // k, 3] = INF  # its last row
    W_down_bar = more.experts_backward(**args, out_bar=d)[2]
    assert ok()
    assert (W_down_bar[e, 3].abs() == INF).all()


# ---- magnitudes and bits ------------------------------------------------------------------------------------------------
ROWS = [(200, 136, 72, 8, 4), (300, 520, 64, 16, 8), (600, 320, 712, 3, 2), (1500, 264, 1032, 4, 2)]


@pytest.mark.parametrize("size", ROWS, ids=str)
@pytest.mark.parametrize("power", [-100, 100])
def test_rows_of_any_magnitude(size, power):
    """A power of two times the weights, or the gradient, is that power times the result."""
    import mixture_experts_rank_b200 as more
    args, d = make(*size)
    want, wbar = more.experts(**args), more.experts_backward(**args, out_bar=d)[0]
    out = more.experts(**dict(args, W_down=args["W_down"] * 2.0**power))
    X_bar = more.experts_backward(**args, out_bar=d * 2.0**power)[0]
    assert ok() and torch.equal(out, want * 2.0**power) and torch.equal(X_bar, wbar * 2.0**power)


@pytest.mark.parametrize("size", ROWS, ids=str)
@pytest.mark.parametrize("value", [2.0**-60, 2.0**60, 2.0**125, float("inf"), float("nan")])
def test_columns_next_to_ones_of_another_magnitude(size, value):
    """One output channel of a size of its own, or of no size at all, does not change its neighbours by more than the bf16
    rounding of a row."""
    import mixture_experts_rank_b200 as more
    args, _ = make(*size)
    h = size[1]
    odd = [0, 70, h - 1]
    W_down = args["W_down"].clone()
    W_down[:, odd] = value
    out = more.experts(**dict(args, W_down=W_down))
    assert ok()
    keep = torch.ones(h, dtype=torch.bool, device="cuda")
    keep[odd] = False
    want, bound = ref.forward(**args)
    check(out[:, keep], want[:, keep], bound[:, keep], "out")
    if abs(value) < 2.0**100:
        want, bound = ref.forward(**dict(args, W_down=W_down))
        check(out[:, odd], want[:, odd], bound[:, odd], "out of the odd channels")


BITS = [(2000, 512, 64, 16, 4), (1000, 2048, 64, 16, 4), (500, 4096, 200, 8, 2), (1000, 1024, 40, 8, 8), (1000, 2048, 136, 8, 4),
        (600, 320, 712, 3, 2)]


@pytest.mark.parametrize("size", BITS, ids=str)
def test_gate_gradients_of_long_products(size):
    """The gates' gradient, an fp32 output, in the 2-norm.  The tensor cores cut a sum off at fp32's last place with every 16
    products: on average half a place, 2^-24 of the sum so far, which is 2/3 of the whole sum's magnitude in the mean over
    a sum of random signs.  Products of more than 2048, or of experts of up to 64 columns, are taken in runs of at most 1024.
    Three such factors."""
    import mixture_experts_rank_b200 as more
    N, h, s, M, k = size
    args, d = make(*size)
    gate_bar = more.experts_backward(**args, out_bar=d)[3]
    assert ok()
    want = ref.backward(**args, out_bar=d)[0]["gate_bar"]
    cuts = (min(h, 1024) if s <= 64 or h > 2048 else h) / 16
    assert (gate_bar.double() - want).norm() <= 3 * cuts * 2.0**-24 * 2 / 3 * want.norm()


@pytest.mark.parametrize("size", BITS, ids=str)
def test_results_have_as_many_roundings_as_documented(size):
    """In the 2-norm.  A rounding to bf16 is off by a uniform part of 2^-8 / m of a value with mantissa m; over mantissas of
    even logarithm that is 2^-8 (1 / 3 * 3 / 8 / ln 2)^(1/2) = 0.00166 in the root mean square.  Three roundings: the middle
    (or the gradients of a and b), a slot's row, the result; two for the weights' gradients, and in 8 bits; 5 percent for
    the mantissas' distribution, where one rounding more would be 15 or 22."""
    import mixture_experts_rank_b200 as more
    args, d = make(*size)
    once = 2.0**-8 * (1 / 3 * 3 / 8 / math.log(2)) ** 0.5

    def holds(got, want, roundings):
        return (got.double() - want).norm() <= 1.05 * once * roundings**0.5 * want.norm()

    assert holds(more.experts(**args), ref.forward(**args)[0], 3)
    got, want = more.experts_backward(**args, out_bar=d), ref.backward(**args, out_bar=d)[0]
    assert holds(got[0], want["X_bar"], 3) and holds(got[1], want["W_up_bar"], 2) and holds(got[2], want["W_down_bar"], 2)
    if size[1] % 16 == 0 and size[2] % 16 == 0:
        args = int8_of(args)
        assert holds(more.experts_int8(**args), ref.forward(**args)[0], 2)
    assert ok()


@pytest.mark.parametrize("eight", [False, True])
def test_wide_layers_on_two_streams_and_in_graphs(eight):
    """Calls that take their channels in runs, with the shared memory of a whole SM and the whole GPU each: two at once, and
    captured ones that share nothing but the device."""
    import mixture_experts_rank_b200 as more
    layer = more.moe_layer_int8 if eight else more.moe_layer
    inputs = [layer_inputs(64, 7168, 16, 16, 32, seed) for seed in (0, 1)]
    if eight:
        inputs = [int8_of(a) for a in inputs]
    want = [layer(**a, k=8) for a in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(layer(**inputs[i], k=8))
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i]) for i in (0, 1) for t in got[i])
    graphs, held = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, a in zip(graphs, inputs):
        with torch.cuda.graph(g):
            held.append(layer(**a, k=8))
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert ok() and all(torch.equal(t, w) for t, w in zip(held, want))
