"""The experts' products behind the router (more_experts, more_experts_int8, more_experts_backward) against a plain
implementation in 64 bits, within derived bounds (tests/experts_reference.py): sizes from one token on, odd and ragged
ones, experts without a token, slots that nobody lists, other streams, captured graphs."""
import pytest
import torch

from tests import experts_reference as ref

pytestmark = pytest.mark.gpu

SIZES = [  # N, h, s, M, k
    (1, 8, 8, 8, 1), (1, 64, 16, 8, 8), (2, 2048, 64, 64, 8), (37, 72, 24, 16, 3), (300, 136, 200, 8, 2),
    (130, 520, 64, 40, 5), (1000, 256, 72, 24, 4), (129, 64, 264, 1, 1), (513, 320, 136, 3, 2), (700, 1096, 392, 8, 3),
    (64, 128, 64, 1000, 16),
    (40, 128, 64, 1000, 16), (17, 128, 72, 16, 4), (16, 128, 72, 4, 4),  # few selections an expert, or few tokens
    (260, 1024, 160, 1, 1), (1500, 264, 1032, 4, 2), (3000, 200, 136, 16, 3),  # wide experts with many rows: CTA pairs
    (193, 1096, 712, 1, 1), (900, 72, 704, 4, 2), (600, 520, 520, 3, 2), (420, 2120, 712, 1, 1),
    (70, 4104, 56, 4, 2), (500, 2112, 136, 2, 1),  # h long enough for sums in runs
]
SIZES_8 = [  # the same with h and s in whole 16s
    (1, 16, 16, 8, 1), (1, 64, 16, 8, 8), (2, 2048, 64, 64, 8), (37, 80, 48, 16, 3), (300, 144, 208, 8, 2),
    (130, 528, 64, 40, 5), (129, 64, 272, 1, 1), (513, 320, 144, 3, 2), (700, 1104, 400, 8, 3), (64, 128, 64, 1000, 16),
    (40, 128, 64, 1000, 16), (17, 128, 80, 16, 4), (16, 128, 80, 4, 4),
    (260, 1024, 160, 1, 1), (1500, 272, 1040, 4, 2), (3000, 208, 144, 16, 3),
    (193, 1104, 720, 1, 1), (900, 80, 704, 4, 2), (420, 2128, 720, 1, 1),
]


def rnd(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def routing(g, N, M, k, how):
    """idx int32 [N, k]: 'spread' over all experts, or everything on the 'first' k experts."""
    if how == "first":
        return torch.arange(k, device="cuda", dtype=torch.int32).repeat(N, 1)
    return torch.rand(N, M, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)


def make(N, h, s, M, k, seed=0, how="spread"):
    import mixture_experts_rank_b200 as more
    g = torch.Generator(device="cuda").manual_seed(seed)
    X, W_up, W_down = rnd(g, N, h), rnd(g, M, 2 * s, h, scale=h**-0.5), rnd(g, M, h, s, scale=s**-0.5)
    gate = torch.softmax(torch.randn(N, k, generator=g, device="cuda"), 1)
    offsets, slots = more.dispatch(routing(g, N, M, k, how).contiguous(), M)
    return dict(X=X, W_up=W_up, W_down=W_down, gate=gate, offsets=offsets, slots=slots), rnd(g, N, h)


def guarded(shape, dtype):
    """A tensor of this shape inside a larger buffer of a known pattern, and a check that the rest is untouched."""
    n = 1
    for d in shape:
        n *= d
    buf = torch.full((n + 512,), 77, dtype=dtype, device="cuda")

    def untouched():
        return bool((buf[:256] == 77).all() and (buf[256 + n:] == 77).all())

    return buf[256:256 + n].view(shape), untouched


def ok():
    import mixture_experts_rank_b200 as more
    torch.cuda.synchronize()
    return more.device_status() == 0


def int8_of(args):
    import mixture_experts_rank_b200 as more
    qu, su = more.quantize_rows(args["W_up"])
    qd, sd = more.quantize_rows(args["W_down"])
    return dict(args, W_up=qu, up_scale=su, W_down=qd, down_scale=sd)


@pytest.mark.parametrize("how", ["spread", "first"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_experts(size, how):
    import mixture_experts_rank_b200 as more
    args, _ = make(*size, how=how)
    out, untouched = guarded((size[0], size[1]), torch.bfloat16)
    assert more.experts(**args, out=out) is out
    assert ok() and untouched()
    ref.check(out, *ref.forward(**args), "out")


@pytest.mark.parametrize("size", [(66001, 16, 8, 8, 5), (66000, 16, 8, 16, 1), (33001, 264, 8, 8, 2)], ids=str)
def test_many_tokens_of_short_rows(size):
    """Enough tokens that a thread sums several of them, a last block that is not full, tokens that keep nothing."""
    import mixture_experts_rank_b200 as more
    args, out_bar = make(*size)
    args = masked(args, [0, size[0] * size[4] // 2, size[0] * size[4] - 1])
    out, untouched = guarded((size[0], size[1]), torch.bfloat16)
    more.experts(**args, out=out)
    x_bar = more.experts_backward(**args, out_bar=out_bar)[0]
    assert ok() and untouched()
    ref.check(out, *ref.forward(**args), "out")
    want, bound = ref.backward(**args, out_bar=out_bar)
    ref.check(x_bar, want["X_bar"], bound["X_bar"], "X_bar")


@pytest.mark.parametrize("rows,width", [(1, 16), (3, 48), (130, 2048), (7, 4112)])
def test_quantize_rows_is_exact(rows, width):
    import mixture_experts_rank_b200 as more
    g = torch.Generator(device="cuda").manual_seed(rows)
    V = rnd(g, rows, width)
    V[rows // 2] = 0
    V[-1, 3] = V[-1].abs().max() * 2
    V[-1, 5] = -V[-1, 3] / 2  # 127 v / max is a half exactly
    q, scale = more.quantize_rows(V)
    assert ok()
    want, sc, _ = ref.to_8_bits(V.double())
    assert torch.equal(q.double(), want)
    assert ((scale.double() - sc[:, 0]).abs() <= 2.0**-24 * sc[:, 0]).all()


@pytest.mark.parametrize("top", [2.0**-100, 2.0**-122, 2.0**-124, 2.0**-126, 2.0**-130, 2.0**-133])
def test_quantize_rows_of_tiny_values(top):
    """Rows whose 127 / max overflows, down to the smallest bf16: 2^-133 is one step of its subnormals."""
    import mixture_experts_rank_b200 as more
    steps = torch.arange(-8, 8, device="cuda", dtype=torch.float64)
    V = (steps / 8 * top).to(torch.bfloat16)[None].repeat(3, 3)
    V[1] = top
    V[2, 1:] = 0
    q, scale = more.quantize_rows(V)
    assert ok()
    want, sc, _ = ref.to_8_bits(V.double())
    assert torch.equal(q.double(), want)
    # a rounding to fp32: half a step relative to the value, or half the subnormals' step
    assert ((scale.double() - sc[:, 0]).abs() <= 2.0**-24 * sc[:, 0] + 2.0**-150).all()


@pytest.mark.parametrize("N", [9, 300])
def test_tiny_tokens_among_ordinary_ones_in_8_bits(N):
    import mixture_experts_rank_b200 as more
    args = int8_of(make(N, 144, 80, 8, 2)[0])
    want = more.experts_int8(**args)
    X = args["X"].clone()
    X[::3] = (X[::3].double() * 2.0**-126).bfloat16()
    out = more.experts_int8(**dict(args, X=X))
    assert ok()
    assert torch.equal(out[1::3], want[1::3]) and torch.equal(out[2::3], want[2::3])
    assert (out[::3].abs() < 2.0**-100).all()


@pytest.mark.parametrize("how", ["spread", "first"])
@pytest.mark.parametrize("size", SIZES_8, ids=str)
def test_experts_int8(size, how):
    import mixture_experts_rank_b200 as more
    args = int8_of(make(*size, how=how)[0])
    out, untouched = guarded((size[0], size[1]), torch.bfloat16)
    more.experts_int8(**args, out=out)
    assert ok() and untouched()
    ref.check(out, *ref.forward(**args), "out")


@pytest.mark.parametrize("how", ["spread", "first"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_experts_backward(size, how):
    import mixture_experts_rank_b200 as more
    N, h, s, M, k = size
    args, out_bar = make(*size, how=how)
    shapes = dict(out_Xbar=(N, h), out_W_up_bar=(M, 2 * s, h), out_W_down_bar=(M, h, s), out_gate_bar=(N, k),
                  out_logits_bar=(N, k))
    outs = {n: guarded(sh, torch.float32 if n in ("out_gate_bar", "out_logits_bar") else torch.bfloat16)
            for n, sh in shapes.items()}
    got = more.experts_backward(**args, out_bar=out_bar, **{n: t for n, (t, _) in outs.items()})
    assert ok() and all(f() for _, f in outs.values())
    want, bound = ref.backward(**args, out_bar=out_bar)
    for name, t in zip(("X_bar", "W_up_bar", "W_down_bar", "gate_bar", "logits_bar"), got):
        ref.check(t, want[name], bound[name], name)


LAYERS = [  # N, h, r, s, M, k: few tokens on one kernel, then more than it takes
    (1, 16, 16, 16, 8, 1), (1, 2048, 32, 64, 256, 8), (2, 64, 16, 16, 8, 8), (13, 1040, 64, 352, 64, 6),
    (64, 128, 32, 48, 16, 16), (33, 4112, 128, 32, 24, 2), (64, 256, 32, 1040, 8, 2), (5, 320, 16, 2064, 16, 3),
    (65, 128, 32, 48, 16, 4), (300, 256, 32, 80, 64, 8),
]


def layer_inputs(N, h, r, s, M, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dict(X=rnd(g, N, h), R1=rnd(g, h, r, scale=h**-0.5), R2=rnd(g, r, M, scale=r**-0.5),
                W_up=rnd(g, M, 2 * s, h, scale=h**-0.5), W_down=rnd(g, M, h, s, scale=s**-0.5))


def layer_reference(args, k, fp32_rows, **scales):
    """The experts in 64 bits for the router's own selections and gates."""
    import mixture_experts_rank_b200 as more
    idx, gate, _, _ = more.route(args["X"], args["R1"], args["R2"], k)
    offsets, slots = more.dispatch(idx, args["W_down"].shape[0])
    return ref.forward(args["X"], args["W_up"], args["W_down"], gate, offsets, slots, fp32_rows=fp32_rows, **scales)


@pytest.mark.parametrize("size", LAYERS, ids=str)
def test_moe_layer(size):
    import mixture_experts_rank_b200 as more
    N, h, r, s, M, k = size
    args = layer_inputs(N, h, r, s, M)
    out, untouched = guarded((N, h), torch.bfloat16)
    more.moe_layer(**args, k=k, out=out)
    assert ok() and untouched()
    ref.check(out, *layer_reference(args, k, N <= 64), "out")


@pytest.mark.parametrize("size", LAYERS, ids=str)
def test_moe_layer_int8(size):
    import mixture_experts_rank_b200 as more
    N, h, r, s, M, k = size
    args = int8_of(layer_inputs(N, h, r, s, M))
    out, untouched = guarded((N, h), torch.bfloat16)
    more.moe_layer_int8(**args, k=k, out=out)
    assert ok() and untouched()
    scales = {n: args[n] for n in ("up_scale", "down_scale")}
    ref.check(out, *layer_reference(args, k, N <= 64, **scales), "out")


def masked(args, drop):
    """The same routing with some selections dropped, as dispatch does with an index outside [0, M)."""
    import mixture_experts_rank_b200 as more
    N, k = args["gate"].shape
    M = args["offsets"].numel() - 1
    idx = torch.empty(N * k, dtype=torch.int32, device="cuda")
    idx[args["slots"].long()] = torch.repeat_interleave(torch.arange(M, dtype=torch.int32, device="cuda"),
                                                        args["offsets"].diff().long())
    idx[drop] = M + 5
    offsets, slots = more.dispatch(idx.view(N, k), M)
    torch.cuda.synchronize()
    assert more.device_status() != 0  # dispatch reports the index
    return dict(args, offsets=offsets, slots=slots)


@pytest.mark.parametrize("size", [(37, 72, 24, 16, 3), (700, 320, 136, 3, 2)], ids=str)
def test_selections_that_nobody_lists(size):
    import mixture_experts_rank_b200 as more
    args, d = make(*size)
    N, k = size[0], size[4]
    args = masked(args, list(range(0, 2 * k)) + [5 * k + 1])  # tokens 0 and 1 keep nothing
    out = more.experts(**args)
    got = more.experts_backward(**args, out_bar=d)
    assert ok()
    ref.check(out, *ref.forward(**args), "out")
    assert (out[:2] == 0).all() and (got[0][:2] == 0).all() and (got[3][:2] == 0).all()
    want, bound = ref.backward(**args, out_bar=d)
    for name, t in zip(want, got):
        ref.check(t, want[name], bound[name], name)
    eight = int8_of(make(N, 80, 32, size[3], k)[0])
    eight = masked(eight, list(range(0, 2 * k)))
    out = more.experts_int8(**eight)
    assert ok() and (out[:2] == 0).all()
    ref.check(out, *ref.forward(**eight), "out")


def test_broken_offsets_and_slots_are_reported():
    import mixture_experts_rank_b200 as more
    args, d = make(50, 64, 16, 8, 2)
    for bad in ([0, 120] + [100] * 7, [-1] + [100] * 8, [0, 60, 30, 60, 70, 80, 90, 95, 100]):
        out, untouched = guarded((50, 64), torch.bfloat16)
        more.experts(**dict(args, offsets=torch.tensor(bad, dtype=torch.int32, device="cuda")), out=out)
        torch.cuda.synchronize()
        assert more.device_status() != 0 and untouched() and (out == 0).all()
    slots = args["slots"].clone()
    slots[3], slots[40] = 100, -7
    lost = args["slots"][[3, 40]].long()
    gate = args["gate"].clone()
    gate.view(-1)[lost] = 0  # what a skipped selection comes to
    out = more.experts(**dict(args, slots=slots))
    got = more.experts_backward(**dict(args, slots=slots), out_bar=d)
    torch.cuda.synchronize()
    assert more.device_status() != 0
    ref.check(out, *ref.forward(**dict(args, gate=gate)), "out")
    want, bound = ref.backward(**dict(args, gate=gate), out_bar=d)
    for i, name in enumerate(("X_bar", "W_up_bar", "W_down_bar")):
        ref.check(got[i], want[name], bound[name], name)
    assert (got[3].view(-1)[lost] == 0).all()


def test_not_a_number_stays_with_its_token():
    import mixture_experts_rank_b200 as more
    args, _ = make(200, 128, 40, 8, 2)
    clean = more.experts(**args)
    X = args["X"].clone()
    X[17, 3], X[90, 5] = float("nan"), float("inf")
    out = more.experts(**dict(args, X=X))
    assert ok()
    keep = torch.ones(200, dtype=torch.bool, device="cuda")
    keep[[17, 90]] = False
    assert torch.equal(out[keep], clean[keep]) and not torch.isfinite(out[~keep]).all(1).any()
    a = layer_inputs(9, 128, 16, 32, 16)
    clean = more.moe_layer(**a, k=3)
    X = a["X"].clone()
    X[4, 7] = float("nan")  # no logit of it is a number: it selects nothing
    out = more.moe_layer(**dict(a, X=X), k=3)
    torch.cuda.synchronize()
    assert more.device_status() != 0
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(out[keep], clean[keep]) and (out[4] == 0).all()


@pytest.mark.parametrize("M,k", [(4096, 8), (600, 16), (16, 16)])
def test_layer_with_equal_logits_takes_the_lowest_experts(M, k):
    import mixture_experts_rank_b200 as more
    a = layer_inputs(3, 64, 16, 16, M)
    a["R2"] = a["R2"][:, :1].repeat(1, M).contiguous()
    out = more.moe_layer(**a, k=k)
    assert ok()
    idx = torch.arange(k, device="cuda", dtype=torch.int32).repeat(3, 1)
    offsets, slots = more.dispatch(idx, M)
    gate = torch.full((3, k), 1 / k, device="cuda")
    ref.check(out, *ref.forward(a["X"], a["W_up"], a["W_down"], gate, offsets, slots, fp32_rows=True), "out")
    a["R2"][:, M // 2:] *= 2  # two values: for every token one half is ahead of the other
    out = more.moe_layer(**a, k=k)
    assert ok()
    ref.check(out, *layer_reference(a, k, True), "out")


@pytest.mark.parametrize("N", [9, 300])
def test_gates_of_selections_that_nobody_lists_do_not_count(N):
    import mixture_experts_rank_b200 as more
    args, _ = make(N, 72, 24, 16, 3)
    args = masked(args, [0, 1, 2, 7])  # token 0 keeps nothing, token 2 loses one
    args["gate"].view(-1)[[0, 7]] = float("nan")
    args["gate"].view(-1)[1] = float("inf")
    out = more.experts(**args)
    assert ok() and (out[0] == 0).all()
    ref.check(out, *ref.forward(**args), "out")


@pytest.mark.parametrize("N", [3, 200])
def test_an_infinite_middle_gives_infinity(N):
    import mixture_experts_rank_b200 as more
    args, _ = make(N, 64, 16, 1, 1)
    args["X"].fill_(1.0)
    args["W_up"].fill_(1e20)
    args["W_down"].fill_(0.5)
    out = more.experts(**args)
    assert ok() and (out == float("inf")).all()


def every_call(seed=0):
    """(name, call with given outputs) of each entry point, on inputs of its own."""
    import mixture_experts_rank_b200 as more
    args, d = make(300, 136, 72, 8, 2, seed)
    wide, dw = make(600, 320, 712, 3, 2, seed)
    eight = int8_of(make(300, 144, 80, 8, 2, seed)[0])
    few = layer_inputs(7, 144, 16, 48, 24, seed)
    many = layer_inputs(90, 144, 16, 48, 24, seed)
    return {"experts": lambda: more.experts(**args), "pairs": lambda: more.experts(**wide),
            "int8": lambda: more.experts_int8(**eight), "backward": lambda: more.experts_backward(**args, out_bar=d),
            "backward pairs": lambda: more.experts_backward(**wide, out_bar=dw),
            "layer": lambda: more.moe_layer(**few, k=3), "layer many": lambda: more.moe_layer(**many, k=3),
            "layer int8": lambda: more.moe_layer_int8(**int8_of(few), k=3), "rows": lambda: more.quantize_rows(args["X"][:, :128].contiguous())}


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", list(["experts", "pairs", "int8", "backward", "backward pairs", "layer", "layer many",
                                       "layer int8", "rows"]))
def test_repeated_streamed_and_captured_calls_agree(name):
    f, other = every_call()[name], every_call(1)[name]
    first = f()
    torch.cuda.synchronize()
    assert same(first, f())
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    want = other()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        a = [f() for _ in range(4)]
    with torch.cuda.stream(s2):
        b = [other() for _ in range(4)]
    torch.cuda.synchronize()
    assert all(same(x, first) for x in a) and all(same(x, want) for x in b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got, again = f(), f()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert same(got, first) and same(again, first) and ok()


def test_stream_argument_and_given_scratch():
    import mixture_experts_rank_b200 as more
    args, d = make(64, 72, 24, 8, 2)
    want = more.experts(**args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    scratch = torch.full((more.experts_scratch_bytes(64, 72, 24, 8, 2),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    out = more.experts(**args, scratch=scratch, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    with pytest.raises(more.MoreError):
        more.experts(**args, scratch=scratch[:-256])
    with pytest.raises(ValueError):
        more.experts(**dict(args, X=args["X"].t().contiguous().t()))
    with pytest.raises(ValueError):
        more.experts(**args, out=torch.empty(64, 80, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        more.experts(**args, out=torch.empty(64, 72, device="cuda"))


def test_no_tokens():
    import mixture_experts_rank_b200 as more
    args, d = make(0, 64, 16, 8, 2)
    assert more.experts(**args).shape == (0, 64)
    got = more.experts_backward(**args, out_bar=d)
    assert ok() and got[0].shape == (0, 64) and (got[1] == 0).all() and (got[2] == 0).all()
    a = layer_inputs(0, 64, 16, 16, 8)
    assert more.moe_layer(**a, k=2).shape == (0, 64)


def test_a_training_step_through_the_router_and_the_experts():
    """route_train, dispatch, experts, then the backward of both: the chain that a training step makes of them, each
    gradient against the formulas in 64 bits for the step's own selections."""
    import mixture_experts_rank_b200 as more
    N, h, r, s, M, k = 200, 128, 32, 48, 64, 4
    a = layer_inputs(N, h, r, s, M, seed=5)
    g = torch.Generator(device="cuda").manual_seed(9)
    d, pbar = rnd(g, N, h), torch.randn(M, generator=g, device="cuda") * 0.01
    idx, gate, count, logits, m, Z, psum = more.route_train(a["X"], a["R1"], a["R2"], k)
    offsets, slots = more.dispatch(idx, M)
    out = more.experts(a["X"], a["W_up"], a["W_down"], gate, offsets, slots)
    Xe, dU, dD, dg, dl = more.experts_backward(a["X"], a["W_up"], a["W_down"], gate, offsets, slots, d)
    Xr, dR1, dR2, _ = more.route_backward(a["X"], a["R1"], a["R2"], k, top_idx=idx, top_vals_bar=dl, pbar=pbar, m=m, Z=Z)
    assert ok() and torch.equal(count, offsets.diff())
    ref.check(out, *ref.forward(a["X"], a["W_up"], a["W_down"], gate, offsets, slots), "out")
    want, bound = ref.backward(a["X"], a["W_up"], a["W_down"], gate, offsets, slots, d)
    for name, t in zip(want, (Xe, dU, dD, dg, dl)):
        ref.check(t, want[name], bound[name], name)
    # the router's part: autograd in 64 bits from the same gradient on the selected logits; 2e-3 of the terms' magnitudes
    # is that kernel's own tolerance (its softmax and z are fp32)
    X, R1, R2 = (a[n].double().requires_grad_() for n in ("X", "R1", "R2"))
    l = X @ R1 @ R2
    (l.gather(1, idx.long()) * dl.double()).sum().add((torch.softmax(l, 1).sum(0) * pbar.double()).sum()).backward()
    y = torch.zeros_like(l).scatter_(1, idx.long(), dl.double().abs()) + torch.softmax(l, 1).detach() * 2 * pbar.abs().max()
    z = y @ R2.detach().abs().T
    mags = (z @ R1.detach().abs().T, X.detach().abs().T @ z, (X.detach().abs() @ R1.detach().abs()).T @ y)
    for got, leaf, mag, name in zip((Xr, dR1, dR2), (X, R1, R2), mags, ("X", "R1", "R2")):
        assert ((got.double() - leaf.grad).abs() <= 2e-3 * mag).all(), name


def test_layer_of_more_tokens_is_the_three_calls():
    import mixture_experts_rank_b200 as more
    a = layer_inputs(130, 256, 32, 64, 32)
    idx, gate, _, _ = more.route(a["X"], a["R1"], a["R2"], 4)
    offsets, slots = more.dispatch(idx, 32)
    assert torch.equal(more.moe_layer(**a, k=4), more.experts(a["X"], a["W_up"], a["W_down"], gate, offsets, slots))
