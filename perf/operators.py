"""What is measured of the experts' operators: the cases, their inputs, and each operator in its plain form.

Five operators stand behind the router.  With e(n, j) and g(n, j) the expert and the gate of token n's j-th selection,
W_up[e] = [A_e; B_e] (2 s x h) and W_down[e] (h x s):

  experts             y_n = sum_j g(n, j) W_down[e] (silu(A_e x_n) * (B_e x_n)) over slots sorted by expert
  experts_backward    the gradients of a sum over y * y_bar: X, W_up, W_down, the gates and the selected logits
  experts_int8        experts with weights in 8 bits (a scale per output channel) and activations rounded to 8 bits
                      (a scale per token) before each of the two products
  moe_layer           the router and the experts together, for a few tokens
  moe_layer_int8      the same with the weights and activations of experts_int8

Outputs are bf16 but for the gates' and logits' gradients (fp32).
"""
import math

import torch

own = False

# ---- cases ---------------------------------------------------------------------------------------------------


def listed():
    return [
        # serving, one sequence: what one decoding step of a layer costs (latency)
        dict(name="layer_1token", op="layer", N=1, h=2048, M=4096, r=32, k=8, s=64),
        # serving, a full decoding batch on many narrow experts: some 480 experts are read once
        dict(name="layer_64tokens", op="layer", N=64, h=2048, M=4096, r=32, k=8, s=64),
        # serving, a small batch on few wide experts, several tokens an expert
        dict(name="layer_16tokens_wide", op="layer", N=16, h=2048, M=64, r=32, k=4, s=1024),
        # the first again with weights in 8 bits
        dict(name="layer_int8_1token", op="layer_int8", N=1, h=2048, M=4096, r=32, k=8, s=64),
        # sizes that fill no tile, an odd batch
        dict(name="layer_int8_13tokens_odd", op="layer_int8", N=13, h=1040, M=256, r=64, k=6, s=352),
        # prefill on the router's own shape: 32 tokens an expert, the weights' reading counts
        dict(name="experts_prefill_h2048", op="experts", N=16384, h=2048, M=4096, r=32, k=8, s=64),
        # prefill of 256 sequences of 1,024 tokens on narrow experts: 256 tokens an expert
        dict(name="experts_prefill_h512", op="experts", N=262144, h=512, M=4096, r=32, k=4, s=64),
        # wide experts of sizes that fill no tile, an odd number of tokens
        dict(name="experts_wide_odd", op="experts", N=5003, h=1096, M=64, r=32, k=6, s=712),
        # training, narrow experts
        dict(name="backward_narrow", op="backward", N=32768, h=512, M=1024, r=32, k=4, s=64),
        # training, wide experts
        dict(name="backward_wide", op="backward", N=8192, h=2048, M=64, r=32, k=4, s=1024),
        # prefill with weights in 8 bits: the router's own shape, and wide experts
        dict(name="experts_int8_prefill", op="experts_int8", N=16384, h=2048, M=4096, r=32, k=8, s=64),
        dict(name="experts_int8_wide", op="experts_int8", N=8192, h=2048, M=64, r=32, k=4, s=1024),
    ]


def draw(rng):
    op = rng.choice(["layer", "layer_int8", "experts", "backward", "experts_int8"])
    layer = op.startswith("layer")
    step = 16 if op.endswith("int8") else 8  # 16-byte rows

    def log(lo, hi, by=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / by)) * by)

    while True:
        c = dict(op=op, N=log(1, 64) if layer else log(1, 262144), h=log(128, 4096, step), M=log(8, 4096, 8),
                 r=rng.choice([16, 32, 64, 128]), k=rng.randint(1, 8), s=log(16, 1408, step))
        slots, weights = c["N"] * c["k"], 3 * c["M"] * c["h"] * c["s"]
        flops = work(c)["flops"]
        if layer:
            fits = weights <= 1.7e9 and slots * 3 * c["h"] * c["s"] <= 1.2e9
        elif op == "backward":
            fits = weights <= 4.1e8 and flops <= 1.2e12 and slots * (c["h"] + 3 * c["s"]) <= 1.7e8
        else:
            fits = weights <= 1.7e9 and flops <= 4.2e11 and slots * (c["h"] + 3 * c["s"]) <= 7.5e8
        if fits:
            return c


def work(case):
    N, h, M, r, k, s = (case[v] for v in ("N", "h", "M", "r", "k", "s"))
    active = M * (1 - (1 - k / M) ** N)  # experts that N k selections are expected to name
    w, slots = 3 * h * s, N * k
    if case["op"].startswith("layer"):
        each = 1 if case["op"] == "layer_int8" else 2
        scales = 4 * (2 * s + h) if case["op"] == "layer_int8" else 0
        return {"bytes": 4 * N * h + 2 * r * (h + M) + active * (each * w + scales), "flops": 2 * N * r * (h + M) + 2 * slots * w}
    lists = 4 * (M + 1) + 8 * slots  # offsets, slots, gates
    if case["op"] == "experts":
        return {"bytes": 4 * N * h + lists + active * 2 * w, "flops": 2 * slots * w}
    if case["op"] == "experts_int8":
        return {"bytes": 4 * N * h + lists + active * (w + 4 * (2 * s + h)), "flops": 2 * slots * w}
    # X, y_bar and the weights read, every gradient written (experts without a token: zeros); products of h s: two
    # again for silu's argument and its factor, one to the middle, two back to X, three for the weights
    return {"bytes": 6 * N * h + lists + 8 * slots + active * 2 * w + 2 * M * w, "flops": 2 * slots * 8 * h * s}


# ---- inputs --------------------------------------------------------------------------------------------------


def _normal(g, *shape, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(scale)


def _to_8_bits(w):
    """Rows of w as (int8, scale): 127 stands for the row's largest magnitude."""
    top = w.abs().amax(-1, keepdim=True).float()
    q = torch.round(w.float() * 127 / torch.where(top > 0, top, 1)).to(torch.int8)
    return q, (top / 127).squeeze(-1)


def prepare(case, seed):
    N, h, M, r, k, s = (case[v] for v in ("N", "h", "M", "r", "k", "s"))
    g = torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)
    st = dict(case=dict(case), k=k)
    st["X"] = _normal(g, N, h)
    st["R1"] = _normal(g, h, r, scale=h**-0.5)
    st["R2"] = _normal(g, r, M, scale=r**-0.5)
    st["W_up"] = _normal(g, M, 2 * s, h, scale=h**-0.5)
    st["W_down"] = _normal(g, M, h, s, scale=s**-0.5)
    if case["op"].endswith("int8"):
        for w in ("W_up", "W_down"):
            st[w], st[w + "_scale"] = _to_8_bits(st[w])
    if case["op"].startswith("layer"):
        return st
    # what the router and the dispatch before this operator leave behind
    logits = st["X"].float() @ st.pop("R1").float() @ st.pop("R2").float()
    top, idx = torch.topk(logits, k, dim=1)
    del logits
    st["gate"] = torch.softmax(top, dim=1)
    flat = idx.reshape(-1)
    st["slots"] = torch.sort(flat, stable=True).indices.to(torch.int32)
    count = torch.bincount(flat, minlength=M)
    st["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).to(torch.int32)
    st["capacity"] = int(count.max())  # the largest group, for the plain form's padded batches
    if case["op"] == "backward":
        st["out_bar"] = _normal(g, N, h)
    return st


# ---- plain forms ---------------------------------------------------------------------------------------------


def _silu(a):
    return a / (1 + torch.exp(-a))


def _plain_quantize(v):
    top = v.abs().amax(-1, keepdim=True)
    q = torch.round(v * 127 / torch.where(top > 0, top, 1))
    return q, top / 127


def _plain_layer(st):
    """Every selection's own weights gathered, one product each; logits in 64 bits (selections next to a border)."""
    X, k = st["X"].float(), st["k"]
    logits = X.double() @ st["R1"].double() @ st["R2"].double()
    top, idx = torch.sort(logits, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    gate = torch.softmax(top, dim=1).float()
    N, h = X.shape
    s = st["W_down"].shape[2]
    e = idx.reshape(-1)
    x = X.repeat_interleave(k, 0)
    eight = "W_up_scale" in st
    if eight:
        x, sx = _plain_quantize(x)
    pre = torch.bmm(st["W_up"][e].float(), x[:, :, None])[:, :, 0]
    if eight:
        pre = pre * sx * st["W_up_scale"][e]
    mid = _silu(pre[:, :s]) * pre[:, s:]
    if eight:
        mid, sm = _plain_quantize(mid)
    y = torch.bmm(st["W_down"][e].float(), mid[:, :, None])[:, :, 0]
    if eight:
        y = y * sm * st["W_down_scale"][e]
    return (y.view(N, k, h) * gate[:, :, None]).sum(1).to(torch.bfloat16)


def _places(st):
    """For each slot in sorted order: its token, its gate, and its row in batches of `capacity` rows an expert."""
    offsets, slots = st["offsets"].long(), st["slots"].long()
    M = offsets.numel() - 1
    e = torch.repeat_interleave(torch.arange(M, device=slots.device), offsets.diff(), output_size=slots.numel())
    row = e * st["capacity"] + torch.arange(slots.numel(), device=slots.device) - offsets[e]
    return slots, slots // st["k"], st["gate"].reshape(-1)[slots], row, M


def _batch(rows, row, M, capacity):
    """Rows of the slots laid out as [M, capacity, .], zero where an expert has fewer."""
    b = rows.new_zeros(M * capacity, rows.shape[1])
    b[row] = rows
    return b.view(M, capacity, -1)


def _by_token(rows, slots, N, k):
    """The sum of each token's k rows, given in the slots' sorted order."""
    y = torch.empty_like(rows)
    y[slots] = rows
    return y.view(N, k, -1).sum(1)


def _plain_experts(st):
    slots, token, gate, row, M = _places(st)
    X, cap, k = st["X"], st["capacity"], st["k"]
    N, h = X.shape
    s = st["W_down"].shape[2]
    eight = "W_up_scale" in st
    x = X.float()
    if eight:
        x, sx = _plain_quantize(x)
    pre = torch.bmm(_batch(x[token], row, M, cap), st["W_up"].float().transpose(1, 2))
    if eight:
        pre = pre * _batch(sx[token], row, M, cap) * st["W_up_scale"][:, None, :]
    mid = _silu(pre[:, :, :s]) * pre[:, :, s:]
    del pre
    if eight:
        mid, sm = _plain_quantize(mid)
    y = torch.bmm(mid, st["W_down"].float().transpose(1, 2))
    if eight:
        y = y * sm * st["W_down_scale"][:, None, :]
    y = y.view(M * cap, h)[row] * gate[:, None]
    return _by_token(y, slots, N, k).to(torch.bfloat16)


def _plain_backward(st):
    slots, token, gate, row, M = _places(st)
    X, cap, k = st["X"], st["capacity"], st["k"]
    N, h = X.shape
    s = st["W_down"].shape[2]
    Wu, Wd = st["W_up"].float(), st["W_down"].float()
    x = _batch(X.float()[token], row, M, cap)
    d = _batch(st["out_bar"].float()[token], row, M, cap)
    gr = _batch(gate[:, None], row, M, cap)
    pre = torch.bmm(x, Wu.transpose(1, 2))
    a, b = pre[:, :, :s], pre[:, :, s:]
    sig = 1 / (1 + torch.exp(-a))
    mid = a * sig * b
    back = torch.bmm(d, Wd)  # the gradient on mid, without the gate
    gate_bar = (back * mid).sum(-1).view(M * cap)[row]
    Wd_bar = torch.bmm(d.transpose(1, 2), mid * gr).to(torch.bfloat16)
    back = back * gr
    pre_bar = torch.cat([back * b * sig * (1 + a * (1 - sig)), back * a * sig], 2)
    Wu_bar = torch.bmm(pre_bar.transpose(1, 2), x).to(torch.bfloat16)
    X_bar = _by_token(torch.bmm(pre_bar, Wu).view(M * cap, h)[row], slots, N, k).to(torch.bfloat16)
    by_slot = torch.empty_like(gate_bar)
    by_slot[slots] = gate_bar
    gate_bar = by_slot.view(N, k)
    g = st["gate"]
    logits_bar = g * (gate_bar - (g * gate_bar).sum(1, keepdim=True))
    return {"X_bar": X_bar, "W_up_bar": Wu_bar, "W_down_bar": Wd_bar, "gate_bar": gate_bar, "logits_bar": logits_bar}


def run(state):
    op, st = state["case"]["op"], state
    if own:
        import mixture_experts_rank_b200 as more

        if op == "layer":
            return more.moe_layer(st["X"], st["R1"], st["R2"], st["W_up"], st["W_down"], st["k"])
        if op == "layer_int8":
            return more.moe_layer_int8(st["X"], st["R1"], st["R2"], st["W_up"], st["W_up_scale"], st["W_down"],
                                       st["W_down_scale"], st["k"])
        if op == "experts":
            return more.experts(st["X"], st["W_up"], st["W_down"], st["gate"], st["offsets"], st["slots"])
        if op == "experts_int8":
            return more.experts_int8(st["X"], st["W_up"], st["W_up_scale"], st["W_down"], st["W_down_scale"],
                                     st["gate"], st["offsets"], st["slots"])
        X_bar, W_up_bar, W_down_bar, gate_bar, logits_bar = more.experts_backward(
            st["X"], st["W_up"], st["W_down"], st["gate"], st["offsets"], st["slots"], st["out_bar"])
        return {"X_bar": X_bar, "W_up_bar": W_up_bar, "W_down_bar": W_down_bar, "gate_bar": gate_bar,
                "logits_bar": logits_bar}
    if op.startswith("layer"):
        return _plain_layer(st)
    return _plain_backward(st) if op == "backward" else _plain_experts(st)


# ---- the definition in 64 bits, one expert at a time -----------------------------------------------------------


def _exact_8_bits(v):
    """(whole numbers, scale) of each row; the division of 127 v by the largest magnitude rounds half to even."""
    top = v.abs().max(dim=-1, keepdim=True).values
    return torch.where(top > 0, (127 * v / top.clamp_min(1e-300)).round(), torch.zeros_like(v)), top / 127


def _exact_expert(st, e, x):
    """(gate part, up part, their product, output) of expert e for the rows x, and the weights."""
    U, D = st["W_up"][e].double(), st["W_down"][e].double()
    s = D.shape[1]
    if "W_up_scale" in st:
        U, D = U * st["W_up_scale"][e].double()[:, None], D * st["W_down_scale"][e].double()[:, None]
        q, sc = _exact_8_bits(x)
        x = q * sc
    p = x @ U.T
    a, b = p[:, :s], p[:, s:]
    m = a * torch.sigmoid(a) * b
    if "W_up_scale" in st:
        q, sc = _exact_8_bits(m)
        return a, b, m, (q * sc) @ D.T, U, D
    return a, b, m, m @ D.T, U, D


def exact(case, seed):
    st = prepare(case, seed)
    X, k = st["X"].double(), st["k"]
    N, h = X.shape
    if case["op"].startswith("layer"):
        logits = torch.einsum("nr,rm->nm", torch.einsum("nh,hr->nr", X, st["R1"].double()), st["R2"].double())
        order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k]
        chosen = torch.gather(logits, 1, order)
        weight = torch.exp(chosen - chosen[:, :1])
        weight = (weight / weight.sum(1, keepdim=True)).reshape(-1)
        expert = order.reshape(-1)
        groups = [(e, (expert == e).nonzero()[:, 0]) for e in sorted(set(expert.tolist()))]
    else:
        weight = st["gate"].double().reshape(-1)
        ends = st["offsets"].tolist()
        groups = [(e, st["slots"][ends[e]:ends[e + 1]].long()) for e in range(len(ends) - 1) if ends[e + 1] > ends[e]]
    if case["op"] != "backward":
        y = torch.zeros(N, h, dtype=torch.float64, device=X.device)
        for e, of in groups:
            y.index_add_(0, of // k, weight[of, None] * _exact_expert(st, e, X[of // k])[3])
        return y
    d = st["out_bar"].double()
    X_bar = torch.zeros_like(X)
    gate_bar = torch.zeros(N * k, dtype=torch.float64, device=X.device)
    Wu_bar = torch.zeros(st["W_up"].shape, dtype=torch.float64, device=X.device)
    Wd_bar = torch.zeros(st["W_down"].shape, dtype=torch.float64, device=X.device)
    for e, of in groups:
        x, dy, w = X[of // k], d[of // k], weight[of, None]
        a, b, m, y, U, D = _exact_expert(st, e, x)
        gate_bar[of] = (dy * y).sum(1)
        Wd_bar[e] = (w * dy).T @ m
        dm = w * dy @ D
        sig = torch.sigmoid(a)
        dp = torch.cat([dm * b * (sig + a * sig * (1 - sig)), dm * a * sig], 1)
        Wu_bar[e] = dp.T @ x
        X_bar.index_add_(0, of // k, dp @ U)
    gate_bar = gate_bar.view(N, k)
    p = weight.view(N, k)
    logits_bar = p * gate_bar - p * (p * gate_bar).sum(1, keepdim=True)
    return {"X_bar": X_bar, "W_up_bar": Wu_bar, "W_down_bar": Wd_bar, "gate_bar": gate_bar, "logits_bar": logits_bar}
