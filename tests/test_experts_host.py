"""The experts' entry points on the CPU: refusals before any launch, scratch sizes, and the 64-bit reference's gradients
against differences."""
import ctypes

import pytest
import torch

from tests import experts_reference as ref

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    import mixture_experts_rank_b200 as m
    return m._lib


def opt(v):
    return P(v) if v else None


BASE = dict(N=16, h=64, s=32, M=64, k=4, r=32, X=16, R1=16, R2=16, W_up=16, W_down=16, us=16, ds=16, gate=16, offsets=16,
            slots=16, out=16, out_bar=16, dX=16, dU=16, dD=16, dg=16, dl=16, scratch=16, short=0)


def size(lib, name, a):
    return getattr(lib, name + "_scratch_bytes")(max(a["N"], 0), max(a["h"], 1), max(a["s"], 1), max(a["M"], 1), max(a["k"], 1))


def call(lib, name, **kw):
    a = dict(BASE, **kw)
    n = lambda *names: [opt(a[x]) for x in names]  # noqa: E731
    tail = [opt(a["scratch"]), max(size(lib, name, a) - a["short"], 0), None]
    shape = [a["N"], a["h"], a["s"], a["M"], a["k"]]
    if name == "more_experts":
        return lib.more_experts(*n("X", "W_up", "W_down"), *shape, *n("gate", "offsets", "slots", "out"), *tail)
    if name == "more_experts_int8":
        return lib.more_experts_int8(*n("X", "W_up", "us", "W_down", "ds"), *shape, *n("gate", "offsets", "slots", "out"), *tail)
    if name == "more_experts_backward":
        return lib.more_experts_backward(*n("X", "W_up", "W_down"), *shape,
                                         *n("gate", "offsets", "slots", "out_bar", "dX", "dU", "dD", "dg", "dl"), *tail)
    shape = [a["N"], a["h"], a["r"], a["s"], a["M"], a["k"]]
    if name == "more_moe_layer":
        return lib.more_moe_layer(*n("X", "R1", "R2", "W_up", "W_down"), *shape, *n("out"), *tail)
    return lib.more_moe_layer_int8(*n("X", "R1", "R2", "W_up", "us", "W_down", "ds"), *shape, *n("out"), *tail)


ALL = ["more_experts", "more_experts_int8", "more_experts_backward", "more_moe_layer", "more_moe_layer_int8"]
COMMON = [(dict(k=0), 1), (dict(k=65), 1), (dict(N=-1), 1), (dict(h=0), 1), (dict(h=68), 1), (dict(s=0), 1), (dict(s=20), 1),
          (dict(X=0), 1), (dict(W_up=0), 1), (dict(W_down=0), 1), (dict(scratch=0), 1), (dict(scratch=8), 1), (dict(X=24), 1),
          (dict(W_up=4), 1), (dict(short=1), 1), (dict(k=17), 2), (dict(M=262152), 2), (dict(h=131088), 2), (dict(s=131088), 2)]


@pytest.mark.parametrize("name", ALL)
@pytest.mark.parametrize("kwargs,expected", COMMON, ids=str)
def test_refusals_of_every_entry(lib, name, kwargs, expected):
    assert call(lib, name, **kwargs) == expected


@pytest.mark.parametrize("name,kwargs,expected", [
    ("more_experts", dict(gate=0), 1), ("more_experts", dict(offsets=0), 1), ("more_experts", dict(slots=0), 1),
    ("more_experts", dict(out=0), 1), ("more_experts", dict(out=8), 1), ("more_experts", dict(M=0), 1),
    ("more_experts_int8", dict(us=0), 1), ("more_experts_int8", dict(ds=0), 1), ("more_experts_int8", dict(h=72), 1),
    ("more_experts_int8", dict(s=40), 1), ("more_experts_int8", dict(ds=20), 1),
    ("more_experts_backward", dict(out_bar=0), 1), ("more_experts_backward", dict(dX=0), 1),
    ("more_experts_backward", dict(dU=0), 1), ("more_experts_backward", dict(dD=0), 1),
    ("more_experts_backward", dict(dg=0), 1), ("more_experts_backward", dict(dl=0), 1),
    ("more_experts_backward", dict(dU=8), 1), ("more_experts_backward", dict(N=0, dU=0), 1),
    ("more_moe_layer", dict(R1=0), 1), ("more_moe_layer", dict(R2=0), 1), ("more_moe_layer", dict(out=0), 1),
    ("more_moe_layer", dict(M=60), 1), ("more_moe_layer", dict(r=24), 2), ("more_moe_layer", dict(r=144), 2),
    ("more_moe_layer_int8", dict(us=0), 1), ("more_moe_layer_int8", dict(s=24), 1),
    ("more_moe_layer_int8", dict(h=72), 1), ("more_moe_layer_int8", dict(R2=8), 1),
])
def test_refusals_of_one_entry(lib, name, kwargs, expected):
    assert call(lib, name, **kwargs) == expected


@pytest.mark.parametrize("name", ["more_experts", "more_experts_int8", "more_moe_layer", "more_moe_layer_int8"])
def test_no_tokens_need_no_gpu(lib, name):
    assert call(lib, name, N=0, X=0, gate=0, slots=0, out=0, scratch=0) == 0


@pytest.mark.parametrize("args,expected", [((0, 1, 16, 16, 16), 1), ((16, -1, 16, 16, 16), 1), ((16, 1, 24, 16, 16), 1),
                                           ((16, 1, 0, 16, 16), 1), ((16, 1, 16, 0, 16), 1), ((16, 1, 16, 16, 0), 1),
                                           ((24, 1, 16, 16, 16), 1), ((16, 1 << 31, 16, 16, 16), 2), ((0, 0, 16, 0, 0), 0)])
def test_quantize_rows_refusals(lib, args, expected):
    v, rows, width, q, scale = args
    assert lib.more_quantize_rows(opt(v), rows, width, opt(q), opt(scale), None) == expected


@pytest.mark.parametrize("name", ["experts", "experts_int8", "experts_backward", "moe_layer", "moe_layer_int8"])
def test_scratch_sizes(name):
    import mixture_experts_rank_b200 as m
    f = getattr(m, name + "_scratch_bytes")
    sizes = [f(N, 512, 64, 64, 4) for N in (0, 1, 64, 65, 1000, 100000)]
    assert all(b > 0 for b in sizes[1:]) and sizes[-1] >= sizes[-2] >= sizes[-3]
    assert f(-1, 512, 64, 64, 4) == 0 and f(10, 512, 64, 64, 17) == 0 and f(10, 512, 64, 262152, 4) == 0
    assert f(1 << 30, 512, 64, 64, 4) == 0    # more slots than 32 bits count
    assert f(1 << 26, 131072, 64, 64, 8) == 0  # more tiles than 32 bits count


def cpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("name", ["experts", "experts_int8", "experts_backward", "moe_layer", "moe_layer_int8"])
def test_binding_refuses_host_tensors_and_wrong_types(name):
    import mixture_experts_rank_b200 as m
    f = getattr(m, name)
    w = torch.int8 if name.endswith("int8") else torch.bfloat16
    X, U, D = cpu(4, 64), cpu(8, 32, 64, dtype=w), cpu(8, 64, 16, dtype=w)
    su, sd = cpu(8, 32, dtype=torch.float32), cpu(8, 64, dtype=torch.float32)
    route = (cpu(4, 2, dtype=torch.float32), cpu(9, dtype=torch.int32), cpu(8, dtype=torch.int32))
    weights = (U, su, D, sd) if w == torch.int8 else (U, D)
    if name.startswith("moe"):
        args = (X, cpu(64, 16), cpu(16, 8), *weights, 2)
    else:
        args = (X, *weights, *route) + ((X,) if name.endswith("backward") else ())
    with pytest.raises(ValueError):
        f(*args)
    with pytest.raises(TypeError):
        f(X.float(), *args[1:])
    with pytest.raises(ValueError):
        f(X, *args[1:2], *[a.reshape(-1) if isinstance(a, torch.Tensor) else a for a in args[2:]])


def loss(X, U, D, gate, offsets, slots, d):
    return (ref.forward(X, U, D, gate, offsets, slots)[0] * d).sum()


def test_reference_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    N, h, s, M, k = 5, 6, 4, 3, 2
    rnd = lambda *sh: torch.randn(*sh, generator=g, dtype=torch.float64)  # noqa: E731
    t = dict(X=rnd(N, h), W_up=rnd(M, 2 * s, h), W_down=rnd(M, h, s), gate=torch.softmax(rnd(N, k), 1))
    idx = torch.stack([torch.randperm(M, generator=g)[:k] for _ in range(N)]).reshape(-1)
    slots = torch.sort(idx, stable=True).indices
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(idx, minlength=M).cumsum(0)])
    d = rnd(N, h)
    v, _ = ref.backward(**t, offsets=offsets, slots=slots, out_bar=d)
    eps = 1e-5
    for name, grad in (("X", "X_bar"), ("W_up", "W_up_bar"), ("W_down", "W_down_bar"), ("gate", "gate_bar")):
        flat = t[name].reshape(-1)
        num = torch.zeros_like(flat)
        for i in range(flat.numel()):
            old = flat[i].item()
            flat[i] = old + eps
            up = loss(t["X"], t["W_up"], t["W_down"], t["gate"], offsets, slots, d)
            flat[i] = old - eps
            num[i] = (up - loss(t["X"], t["W_up"], t["W_down"], t["gate"], offsets, slots, d)) / (2 * eps)
            flat[i] = old
        # central differences: eps^2 of the third derivative, and the loss's own rounding over eps
        assert torch.allclose(num.view_as(v[grad]), v[grad], rtol=1e-7, atol=1e-7), name
    # the gates as a softmax of logits
    logits = torch.log(t["gate"])
    num = torch.zeros_like(logits)
    for n in range(N):
        for j in range(k):
            e = torch.zeros_like(logits)
            e[n, j] = eps
            a, b = (loss(t["X"], t["W_up"], t["W_down"], torch.softmax(logits + q * e, 1), offsets, slots, d) for q in (1, -1))
            num[n, j] = (a - b) / (2 * eps)
    assert torch.allclose(num, v["logits_bar"], rtol=1e-7, atol=1e-7)
