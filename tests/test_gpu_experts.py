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
    (260, 1024, 160, 1, 1), (1500, 264, 1032, 4, 2), (3000, 200, 136, 16, 3),  # wide experts with many rows: CTA pairs
    (70, 4104, 56, 4, 2), (500, 2112, 136, 2, 1),  # h long enough for sums in runs
]
SIZES_8 = [  # the same with h and s in whole 16s
    (1, 16, 16, 8, 1), (1, 64, 16, 8, 8), (2, 2048, 64, 64, 8), (37, 80, 48, 16, 3), (300, 144, 208, 8, 2),
    (130, 528, 64, 40, 5), (129, 64, 272, 1, 1), (513, 320, 144, 3, 2), (700, 1104, 400, 8, 3), (64, 128, 64, 1000, 16),
    (260, 1024, 160, 1, 1), (1500, 272, 1040, 4, 2), (3000, 208, 144, 16, 3),
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
