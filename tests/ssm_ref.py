"""The selective state space scan and the group norm on the CPU in 64 bits, the
scan a token at a time with a running bound of what fp32 arithmetic may be off.

Bound.  u = 2^-24.  M carries the state's magnitudes, M <- e M + |d x B|, and E
its error.  Per token
    E <- e E + u (c_e e M + c_w |d x B| + c_s M')
where, with k_d roundings in the step size d (10 of its softplus: 2 each of an
exponential and a reciprocal of one ulp, 1 each of dt + bias, the exponent's
product, the denominator, the quotient, the series and the sum; and 2 |dt +
bias|, by which the sum's and the product's rounding move the exponent), the
decay e^(d A) is off by c_e = 4 + |d A| (3 + k_d) (the product with A, with
log2(e), and d itself reach the exponent; exp2 and what scales it 4 more), a
written term by c_w = 4 + k_d, and each sum rounds by c_s = 4: chunks sum a
token's terms 4 times into partial sums at most, and a token at a time once.
Chunks of 64 tokens add 64 u M once: 48 partial sums of products with operands
of 22 bits or more.
An output adds, over n, |C| (E + u (N + 16) M) for its sum, 2^-16 |C| M for
operands of 16 bits or more in products that only feed outputs, u |D x| twice,
and half a bf16 step, 2^-8 relative to the result.
"""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24


def sizes(x, A, B, lead):
    """(heads, groups, head_dim, state_dim)."""
    if A.dim() == 1:
        return A.shape[0], B.shape[-2], x.shape[-1], B.shape[-1]
    g = B.shape[-2] if B.dim() == lead + 2 else 1
    return g, g, A.shape[0] // g, A.shape[1]


def steps(d):
    """Step sizes in 64 bits and their roundings k_d, shaped like dt."""
    v = d["dt"].to(F64)
    if d["dt_bias"] is not None:
        v = v + d["dt_bias"].to(F64)
    k = 10 + 2 * v.abs().clamp(max=100)
    if d["dt_softplus"]:
        v = torch.logaddexp(v, torch.zeros_like(v))
    if d["dt_limit"] is not None:
        v = v.clamp(*d["dt_limit"])
    return v, k


class Row:
    """The states of one entry with their running bounds: (heads, head_dim, state_dim)."""

    def __init__(self, S):
        self.S = S.to(F64).clone()
        self.M = self.S.abs()
        self.E = torch.zeros_like(self.S)

    def step(self, x, dt, k, A, B, C, D, z):
        """x, z (H, P); dt, k (H, P or 1); A (H, P or 1, N or 1); B, C (H, N); D (H, P or 1)."""
        g = (dt[..., None] * A).clamp(max=0)
        e = torch.exp(g)
        w = (dt * x)[..., None] * B[:, None]
        ce = 4 + g.abs().clamp(max=1e4) * (3 + k[..., None])
        before = e * self.M
        self.S = e * self.S + w
        self.M = before + w.abs()
        self.E = e * self.E + U * (ce * before + (4 + k[..., None]) * w.abs() + 4 * self.M)
        c = C[:, None]
        y = (self.S * c).sum(-1)
        mag = (self.M * c.abs()).sum(-1)
        tol = (self.E * c.abs()).sum(-1) + (U * (S_TERMS + 80) + 2.0 ** -16) * mag
        if D is not None:
            y = y + D * x
            tol = tol + 2 * U * (D * x).abs() + U * y.abs() + 2.0 ** -16 * (D * x).abs()
        if z is not None:
            gate = z * torch.sigmoid(z)
            tol = tol * gate.abs() + 8 * U * (y * gate).abs()
            y = y * gate
        return y, tol * (1 + 2.0 ** -7) + 2.0 ** -8 * y.abs() + 1e-37


S_TERMS = 256 + 16          # (states, and a tree's additions)


def fwd(d, state, qsl, cache_indices, has_init, pad=-1):
    """(out, tolerance, state, tolerance, rows that are written); d: the inputs by name."""
    x = d["x"]
    H, G, P, N = sizes(x, d["A"], d["B"], 1)
    out, otol = torch.zeros(x.shape[0], H, P, dtype=F64), torch.zeros(x.shape[0], H, P, dtype=F64)
    live = torch.zeros(x.shape[0], dtype=torch.bool)
    st = None if state is None else state.to(F64).reshape(-1, H, P, N).clone()
    stol = None if state is None else torch.zeros_like(st)
    args = _prepared(d, 1)
    for i in range(len(qsl) - 1):
        a, b = int(qsl[i]), int(qsl[i + 1])
        line = i if cache_indices is None else int(cache_indices[i])
        if (cache_indices is not None and line == pad) or a == b or (st is not None and not 0 <= line < st.shape[0]):
            continue
        S = torch.zeros(H, P, N, dtype=F64)
        if st is not None and has_init is not None and bool(has_init[i]):
            S = state.reshape(-1, H, P, N)[line]
        r = Row(S)
        for t in range(a, b):
            out[t], otol[t] = r.step(*(f(t) for f in args))
            live[t] = True
        if st is not None:
            st[line], stol[line] = r.S, r.E + 64 * U * r.M
    shape = x.shape
    return (out.view(shape), otol.view(shape), st if st is None else st.view(state.shape),
            stol if st is None else stol.view(state.shape), live)


def _prepared(d, lead):
    """Functions of the token's index that give Row.step's arguments."""
    x, A, B, C, D, z = (d[n] for n in ("x", "A", "B", "C", "D", "z"))
    H, G, P, N = sizes(x, A, B, lead)
    v, k = steps(d)
    head = A.dim() == 1
    A = A.to(F64).view(H, 1, 1) if head else A.to(F64).view(H, P, N)
    if D is not None:
        D = D.to(F64).view(H, -1)
    cut = (lambda t: t[..., None]) if head else (lambda t: t.unflatten(-1, (H, P)))
    v, k = cut(v), cut(k)
    xs = x.to(F64).reshape(*x.shape[:lead], H, P)
    zs = None if z is None else z.to(F64).reshape(*x.shape[:lead], H, P)
    of = torch.arange(H) // (H // G)
    bs, cs = (t.to(F64).reshape(*t.shape[:lead], G, N)[..., of, :] for t in (B, C))
    return (lambda t: xs[t], lambda t: v[t], lambda t: k[t], lambda t: A, lambda t: bs[t], lambda t: cs[t], lambda t: D,
            lambda t: None if zs is None else zs[t])


def update(d, state, cache_indices, accepted, osi, pad=-1):
    """Decode: x .. (batch, seqlen, ..).  As fwd."""
    x = d["x"]
    n, seqlen = x.shape[:2]
    H, G, P, N = sizes(x, d["A"], d["B"], 2)
    out, otol = (torch.zeros(n, seqlen, H, P, dtype=F64) for _ in range(2))
    live = torch.zeros(n, dtype=torch.bool)
    st = state.to(F64).reshape(-1, H, P, N).clone()
    stol = torch.zeros_like(st)
    args = _prepared(d, 2)
    read = state.reshape(-1, H, P, N)
    for b in range(n):
        line = b
        if cache_indices is not None:
            ci, s = cache_indices[b], 0
            if accepted is not None:
                s = int(accepted[b]) - 1
                if not 0 <= s < ci.numel():
                    continue
            line = int(ci.reshape(-1)[s])
            if line == pad:
                continue
        if not 0 <= line < st.shape[0]:
            continue
        r = Row(read[line])
        live[b] = True
        for t in range(seqlen):
            out[b, t], otol[b, t] = r.step(*(f((b, t)) for f in args))
            if osi is not None and 0 <= int(osi[b, t]) < st.shape[0]:
                st[int(osi[b, t])], stol[int(osi[b, t])] = r.S, r.E
        if osi is None:
            st[line], stol[line] = r.S, r.E
    return out.view(x.shape), otol.view(x.shape), st.view(state.shape), stol.view(state.shape), live


def draw(lead, form, heads, head_dim, groups, state_dim, seed, raw=True, skip=True, gate=False, dt_limit=None, slow=1.0,
         bias=True):
    """Inputs by name; `lead`: leading dimensions; `slow`: factor on the decays."""
    g = torch.Generator().manual_seed(seed)
    head = form == "head"
    dim = heads * head_dim
    x = torch.randn(*lead, dim + 2 * groups * state_dim, generator=g)
    x = (x * torch.sigmoid(x)).bfloat16()
    B = x[..., dim:dim + groups * state_dim].unflatten(-1, (groups, state_dim))
    C = x[..., dim + groups * state_dim:].unflatten(-1, (groups, state_dim))
    of = (heads,) if head else (dim,)
    step = torch.exp(torch.rand(of, generator=g) * 4.6 - 6.9)
    b = step + torch.log(-torch.expm1(-step))
    dt = torch.randn(*lead, *of, generator=g).bfloat16()
    if head:
        A = -(torch.rand(heads, generator=g) * 15 + 1) * slow
    else:
        A = -torch.arange(1, state_dim + 1).float() * (1 + 0.1 * torch.rand(dim, state_dim, generator=g)) * slow
    if not raw:
        dt = torch.nn.functional.softplus(dt.float() + b)
    return dict(x=x[..., :dim].unflatten(-1, (heads, head_dim)) if head else x[..., :dim], dt=dt, A=A, B=B, C=C,
                D=1 + 0.1 * torch.randn(of, generator=g) if skip else None,
                z=torch.randn(*lead, *((heads, head_dim) if head else (dim,)), generator=g).bfloat16() if gate else None,
                dt_bias=b if raw and bias else None, dt_softplus=raw, dt_limit=dt_limit)


def on(d, dev):
    return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def check(got, want, tol, what):
    d = (got.detach().cpu().to(F64) - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / tol.clamp(min=1e-300))[bad].max()):.3g} "
                           f"tolerances, first at {[int(i) for i in bad.nonzero()[0]]}")


def check_state(got, want, tol):
    """Lines that no entry writes (tolerance 0) are as they were, bit for bit."""
    check(got, want, tol, "state")


# ------------------------------------------------------------------- norm --

def norm(x, size, weight, bias, z, eps, kind, activation, gate_first):
    """(out, tolerance) in 64 bits.  The sums of a group of n are off by (n / 8 + 16) u of their terms' magnitudes at most, an
    activation by 8 u, every other operation by u: a few n u in all beside half a bf16 step, taken as (n / 4 + 64) u of the
    magnitudes, where a mean that is taken out counts with its terms."""
    rows = x.shape[0]
    v = x.to(F64).reshape(rows, -1, size)
    act = {None: lambda t: t, "silu": lambda t: t * torch.sigmoid(t), "sigmoid": torch.sigmoid}[activation]
    zz = None if z is None else z.to(F64).reshape(rows, -1, size)

    def wide(w):
        return None if w is None else (w.to(F64) if w.numel() == size else w.to(F64).view(-1, size))
    if gate_first:
        v = v * act(zz)
    k = (size / 4 + 64) * U
    mag = v.abs()
    if kind == "layer":
        mag = mag + v.abs().mean(-1, keepdim=True)
        v = v - v.mean(-1, keepdim=True)
    r = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)
    # r is off by its own roundings and by what v's error moves it: d r / r <= r^2 mean(|v| dv)
    dr = k + r * r * (v.abs() * k * mag).mean(-1, keepdim=True)
    tol = r * (k * mag + v.abs() * dr)
    v = v * r
    w, b = wide(weight), wide(bias)
    if w is not None:
        v, tol = v * w, tol * w.abs() + U * (v * w).abs()
    if b is not None:
        v, tol = v + b, tol + U * (v + b).abs()
    if zz is None:
        # an activation moves by at most 1.1 times its argument's error
        y, tol = act(v), 1.1 * tol + 8 * U * (act(v).abs() + v.abs())
    elif not gate_first:
        y, tol = v * act(zz), tol * act(zz).abs() + 8 * U * (v * act(zz)).abs()
    else:
        y = v
    tol = tol * (1 + 2.0 ** -7) + 2.0 ** -8 * y.abs() + 1e-37
    return y.view(x.shape), tol.view(x.shape)
