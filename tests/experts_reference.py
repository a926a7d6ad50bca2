"""The experts' operators in 64 bits, one expert at a time, with bounds on what a kernel may be off.

Bounds are derived, not fitted.  u = 2^-8 is the largest relative error of one rounding to bf16 and w = 2^-24 that of one to
fp32.  A sum of K products in fp32 is off by at most K w times the sum of the products' magnitudes (to first order); 4 w
covers the silu's own arithmetic (exp, sum, division, product).  A value rounded to bf16 before a product adds u times the
product's sum of magnitudes.  Every bound below is those terms carried through the formulas in magnitudes; SLACK covers
the second-order terms.
"""
import torch

U, W, SLACK = 2.0**-8, 2.0**-24, 1.05


def groups_of(offsets, slots):
    ends = offsets.tolist()
    return [(e, slots[ends[e]:ends[e + 1]].long()) for e in range(len(ends) - 1) if ends[e + 1] > ends[e]]


def to_8_bits(v):
    """(whole numbers, scale, the two steps between which rounding is undecided at 2^-18): rows of v."""
    top = v.abs().amax(-1, keepdim=True)
    x = torch.where(top > 0, 127 * v / torch.where(top > 0, top, 1), 0)
    near = ((x - x.floor()) - 0.5).abs() < x.abs() * 2.0**-18
    return x.round(), top / 127, near


def _halves(p, s):
    return p[:, :s], p[:, s:]


def _middle(x, U_e, s, K):
    """a, b, silu(a) b and the bounds of their fp32 values."""
    a, b = _halves(x @ U_e.T, s)
    ea, eb = _halves(K * W * (x.abs() @ U_e.abs().T), s)
    sg = torch.sigmoid(a)
    m = a * sg * b
    # |silu'| <= 1.1
    em = 1.1 * ea * b.abs() + (a * sg).abs() * eb + 4 * W * m.abs()
    return a, b, sg, m, ea, eb, em


def forward(X, W_up, W_down, gate, offsets, slots, fp32_rows=False, up_scale=None, down_scale=None):
    """(out, bound).  fp32_rows: the middle is carried as a bf16 pair and the slots' rows in fp32."""
    X, gate = X.double(), gate.double()
    N, h = X.shape
    s, k = W_down.shape[2], gate.shape[1]
    out, bound = torch.zeros_like(X), torch.zeros_like(X)
    eight = up_scale is not None
    for e, of in groups_of(offsets, slots):
        x, g = X[of // k], gate.reshape(-1)[of, None]
        A, D = W_up[e].double(), W_down[e].double()
        if eight:
            q, sc, _ = to_8_bits(x)
            p = (q @ A.T) * sc * up_scale[e].double()
            a, b = _halves(p, s)
            m = a * torch.sigmoid(a) * b
            qm, sm, near = to_8_bits(m)
            y = (qm @ D.T) * sm * down_scale[e].double()
            # exact integer sums; the scales' products cost a few fp32 roundings, a middle next to a half may go either way
            off = (near.double() @ D.abs().T) * sm * down_scale[e].double() + 16 * W * \
                (qm.abs() @ D.abs().T) * sm * down_scale[e].double()
            mag = y.abs()
        else:
            a, b, sg, m, ea, eb, em = _middle(x, A, s, h)
            y = m @ D.T
            mag = m.abs() @ D.abs().T
            # fp32_rows: the middle as a bf16 pair; the second rounding is off by U of a remainder of at most U
            off = em @ D.abs().T + s * W * mag + (U * U if fp32_rows else U) * mag
        off = off + (0 if fp32_rows else U * y.abs()) + 2 * W * y.abs()
        out.index_add_(0, of // k, g * y)
        bound.index_add_(0, of // k, g.abs() * (off + k * W * mag))
    return out, SLACK * (bound + U * (out.abs() + bound))


def backward(X, W_up, W_down, gate, offsets, slots, out_bar):
    """({name: gradient}, {name: bound})."""
    X, G, d = X.double(), gate.double(), out_bar.double()
    N, h = X.shape
    M, s, k = W_down.shape[0], W_down.shape[2], gate.shape[1]
    z = lambda *sh: torch.zeros(*sh, dtype=torch.float64, device=X.device)  # noqa: E731
    v = dict(X_bar=z(N, h), W_up_bar=z(M, 2 * s, h), W_down_bar=z(M, h, s), gate_bar=z(N * k))
    t = {n: torch.zeros_like(x) for n, x in v.items()}
    for e, of in groups_of(offsets, slots):
        x, dy, g = X[of // k], d[of // k], G.reshape(-1)[of, None]
        A, D = W_up[e].double(), W_down[e].double()
        a, b, sg, m, ea, eb, em = _middle(x, A, s, h)
        r = dy @ D
        er = h * W * (dy.abs() @ D.abs())
        v["gate_bar"][of] = (r * m).sum(1)
        t["gate_bar"][of] = (er * m.abs() + r.abs() * em + (s + 2) * W * (r * m).abs()).sum(1)
        ds = sg * (1 + a * (1 - sg))  # silu', |silu''| <= 0.5
        p = torch.cat([g * r * b * ds, g * r * a * sg], 1)
        ep = torch.cat([er * b.abs() * ds.abs() + r.abs() * eb * ds.abs() + (r * b).abs() * (0.5 * ea + 6 * W),
                        er * (a * sg).abs() + r.abs() * 1.1 * ea + 6 * W * (r * a * sg).abs()], 1) * g.abs()
        ep = ep + U * (p.abs() + ep)  # rounded to bf16
        gm, egm = g * m, g.abs() * em
        egm = egm + U * (gm.abs() + egm)
        T = x.shape[0]
        v["W_down_bar"][e] = dy.T @ gm
        t["W_down_bar"][e] = dy.abs().T @ (egm + T * W * gm.abs())
        v["W_up_bar"][e] = p.T @ x
        t["W_up_bar"][e] = (ep + T * W * p.abs()).T @ x.abs()
        row = p @ A
        erow = (ep + 2 * s * W * p.abs()) @ A.abs()
        v["X_bar"].index_add_(0, of // k, row)
        t["X_bar"].index_add_(0, of // k, erow + (U + k * W) * (row.abs() + erow))
    for n in ("X_bar", "W_up_bar", "W_down_bar"):  # written as bf16
        t[n] = t[n] + U * (v[n].abs() + t[n])
    gb, tb = v["gate_bar"].view(N, k), t["gate_bar"].view(N, k)
    v["gate_bar"], t["gate_bar"] = gb, tb
    dot = (G * gb).sum(1, keepdim=True)
    v["logits_bar"] = G * (gb - dot)
    mag = (G * gb).abs().sum(1, keepdim=True)
    t["logits_bar"] = G.abs() * (tb + (G.abs() * tb).sum(1, keepdim=True) + (k + 4) * W * (gb.abs() + mag))
    return v, {n: SLACK * x for n, x in t.items()}


def check(got, want, bound, name):
    got = got.double()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - want).abs() - bound
    worst = over.max().item() if over.numel() else 0.0
    if worst > 1e-30:
        at = tuple(int(i) for i in torch.unravel_index(over.argmax(), over.shape))
        raise AssertionError(f"{name}: off by {(got - want).abs()[at].item():.3g} at {at}, bound {bound[at].item():.3g}, "
                             f"value {want[at].item():.3g}; {(over > 0).sum().item()} of {over.numel()} over")
