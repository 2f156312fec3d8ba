"""The gated delta rule and draft verification on the CPU in 64 bits, a token /
a request at a time, with a running bound of what fp32 arithmetic may be off.

Bound.  Per value row, with e = e^g <= 1, |k| <= 1 and beta <= 1, an error of
the state row is multiplied by e (I - beta k k^T), of norm <= e, and each token
adds the roundings of its own sums: at most C 2^-24 (|v| + 2 |S row|), where C
counts the roundings of a token (a sum over the key channels in blocks, the
update, the gate).  E carries that.  An output adds |q| (E + F (|S row| + W)),
F the relative rounding of the operands of its products and W the decayed sum
of |u| |k|, and half a bf16 step, 2^-8 relative to the result.
"""
from __future__ import annotations

import numpy as np
import torch

F64 = torch.float64
# Chunks: a column's values of one 64-token chunk share power-of-two scales.
# X, z and S lie below 2^15, their bounds above 2^14, and the bounds are at most
# 128 times the chunk's largest (|v| + |u| |k| + 64 |S row|); an fp16 part is
# rounded at 2^-25 at the least, so nothing is off by more than
# 128 * 2^-25 / 2^14 = 2^-32 of that largest value, per token: E takes it in at
# every token, an output 64 times.
# one token at a time in fp32: 16..32 terms a lane and 3 exchanges in a sum,
# twice in u, 3 for the update, the gate's e^g (|g| + 4 steps, |g| counted for
# what is left of the state after it) and the norms' roots and quotients
C_REC, F_REC = 80.0, 64 * 2.0 ** -24
# chunks: products of operands held to 2^-20 relative (16 steps of 2^-24 each,
# in K S, in T X twice, in K^T U), sums of up to 256 terms; o from operands of
# 11 bits: S, P and U cut to 2^-10 / 2^-11 each
C_CHUNK, F_CHUNK = 240.0, 2.0 ** -9


def gates(g, beta, A_log, dt_bias):
    if A_log is None:
        return g.to(F64).clamp(max=0), beta.to(F64)
    x = g.to(F64) + dt_bias.to(F64)
    return -torch.exp(A_log.to(F64)) * torch.logaddexp(x, torch.zeros_like(x)), torch.sigmoid(beta.to(F64))


def norm_qk(q, k, scale, l2norm, hv):
    q, k = q.to(F64), k.to(F64)
    if l2norm:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    rep = hv // q.shape[-2]
    return (q * scale).repeat_interleave(rep, -2), k.repeat_interleave(rep, -2)


class Row:
    """State of one entry with its running bounds."""

    def __init__(self, S, c, f):
        self.S, self.c, self.f = S.clone(), c, f
        self.E = torch.zeros(S.shape[:2], dtype=F64)
        self.W = torch.zeros(S.shape[:2], dtype=F64)

    def step(self, q, k, v, g, beta, floor=None):
        e = torch.exp(g)[:, None]
        before = self.S.norm(dim=-1)
        S = self.S * e[..., None]
        u = beta[:, None] * (v - (S * k[:, None]).sum(-1))
        self.S = S + u[..., None] * k[:, None]
        kn = k.norm(dim=-1)[:, None]
        self.E = e * self.E + self.c * 2.0 ** -24 * (v.abs() + 2 * e * before + 2 * u.abs() * kn)
        if floor is not None:
            self.E = self.E + floor
        self.W = e * self.W + u.abs() * kn
        self.M = v.abs() + u.abs() * kn + 64 * before
        o = (self.S * q[:, None]).sum(-1)
        qn = q.norm(dim=-1)[:, None]
        tol = 2.0 ** -8 * o.abs() + qn * (self.E + self.f * (before + self.W)) * (1 + 2.0 ** -7) + 1e-38
        if floor is not None:
            tol = tol + 64 * qn * floor
        return o, tol


def fwd(q, k, v, g, beta, state, qsl, cache_indices, has_init, A_log, dt_bias, scale, l2norm, c, f,
        pad=-1):
    """(out, tolerance, state, tolerance, rows that are written)."""
    hv, dv, dk = v.shape[1], v.shape[2], q.shape[2]
    qq, kk = norm_qk(q, k, scale, l2norm, hv)
    gg, bb = gates(g, beta, A_log, dt_bias)
    vv = v.to(F64)
    out = torch.zeros(v.shape, dtype=F64)
    otol = torch.zeros(v.shape, dtype=F64)
    live = torch.zeros(v.shape[0], dtype=torch.bool)
    st = state.to(F64).clone() if state is not None else None
    stol = torch.zeros(st.shape[:3], dtype=F64) if st is not None else None
    for i in range(len(qsl) - 1):
        a, b = int(qsl[i]), int(qsl[i + 1])
        line = i if cache_indices is None else int(cache_indices[i])
        if line == pad and cache_indices is not None or a == b:
            continue
        if st is not None and not 0 <= line < st.shape[0]:
            continue
        S = torch.zeros(hv, dv, dk, dtype=F64)
        if st is not None and has_init is not None and bool(has_init[i]):
            S = state[line].to(F64)
        r, look = Row(S, c, f), Row(S, c, f)
        for t in range(a, b):
            if (t - a) % 64 == 0 and c == C_CHUNK:     # the chunk's largest values, for the floor of its scales
                floor = torch.zeros(r.E.shape, dtype=F64)
                for x in range(t, min(t + 64, b)):
                    look.step(qq[x], kk[x], vv[x], gg[x], bb[x])
                    floor = torch.maximum(floor, look.M)
                floor = floor * 2.0 ** -32
            out[t], otol[t] = r.step(qq[t], kk[t], vv[t], gg[t], bb[t], floor if c == C_CHUNK else None)
            live[t] = True
        if st is not None:
            st[line], stol[line] = r.S, r.E
    return out, otol, st, stol, live


def update(q, k, v, g, beta, state, cache_indices, accepted, osi, A_log, dt_bias, scale, l2norm,
           c=C_REC, f=F_REC, pad=-1):
    """q .. (batch, seqlen, heads, dim)."""
    n, steps, hv, dv = v.shape
    qq, kk = norm_qk(q, k, scale, l2norm, hv)
    gg, bb = gates(g, beta, A_log, dt_bias)
    vv = v.to(F64)
    out, otol = torch.zeros(v.shape, dtype=F64), torch.zeros(v.shape, dtype=F64)
    st = state.to(F64).clone()
    stol = torch.zeros(st.shape[:3], dtype=F64)
    live = torch.zeros(n, dtype=torch.bool)
    for b in range(n):
        step = 0
        if accepted is not None:
            step = int(accepted[b]) - 1
            if not 0 <= step < cache_indices.shape[1]:
                continue
        line = b
        if cache_indices is not None:
            line = int(cache_indices[b, step]) if cache_indices.dim() == 2 else int(cache_indices[b])
            if line == pad:
                continue
        if not 0 <= line < st.shape[0]:
            continue
        live[b] = True
        r = Row(state[line].to(F64), c, f)
        for t in range(steps):
            out[b, t], otol[b, t] = r.step(qq[b, t], kk[b, t], vv[b, t], gg[b, t], bb[b, t])
            if osi is not None and 0 <= int(osi[b, t]) < st.shape[0]:
                st[int(osi[b, t])], stol[int(osi[b, t])] = r.S, r.E
        if osi is None:
            st[line], stol[line] = r.S, r.E
    return out, otol, st, stol, live


def check(got, ref, tol, what):
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs()
    bad = ~(off <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"{got[i].item()!r}, {ref[i].item()!r} +- {tol.expand(ref.shape)[i].item():.3g}")


def check_state(got, ref, tol, what="state"):
    """Rows are held to E in the 2-norm; what no entry wrote is unchanged."""
    got = got.detach().cpu().to(F64)
    off = (got - ref).norm(dim=-1)
    limit = tol + 2.0 ** -24 * ref.norm(dim=-1) * (tol > 0)
    bad = ~(off <= limit)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} rows outside; first at {i}: off {off[i].item():.3g}, "
                             f"allowed {limit[i].item():.3g}, row of norm {ref[i].norm().item():.3g}")


def draw_inputs(lead, hk, hv, dk, dv, seed, raw=True, normed=False, decay=1.0):
    """q, k, v as views of one (rows, channels) buffer, and the gates.  lead: leading sizes."""
    gen = torch.Generator().manual_seed(seed)
    rows = int(np.prod(lead))
    x = torch.randn(rows, 2 * hk * dk + hv * dv, generator=gen)
    x = x * torch.sigmoid(x)
    if normed:                         # keys and queries of norm 1, in bf16 at most 1 + 2^-8 of it
        qk = x[:, :2 * hk * dk].view(rows, 2 * hk, dk)
        x[:, :2 * hk * dk] = (qk / qk.norm(dim=-1, keepdim=True).clamp(min=1e-6) * (1 - 2.0 ** -7)).view(rows, -1)
    x = x.bfloat16()
    q = x[:, :hk * dk].view(*lead, hk, dk)
    k = x[:, hk * dk:2 * hk * dk].view(*lead, hk, dk)
    v = x[:, 2 * hk * dk:].view(*lead, hv, dv)
    a = torch.randn(*lead, hv, generator=gen).bfloat16()
    b = torch.randn(*lead, hv, generator=gen).bfloat16()
    A_log = torch.log(torch.rand(hv, generator=gen) * 15 + 1) * decay
    dt_bias = torch.rand(hv, generator=gen) * 4 - 6
    d = dict(q=q, k=k, v=v, g=a, beta=b, A_log=A_log, dt_bias=dt_bias)
    if not raw:
        gg, bb = gates(a, b, A_log, dt_bias)
        d.update(g=(gg * decay).float(), beta=bb.float(), A_log=None, dt_bias=None)
    return d


def on(d, device):
    """A copy on the device; the views of one buffer stay views of one buffer."""
    rows = d["q"].shape[:-2]
    n = int(np.prod(rows))
    base = torch.cat([d[x].reshape(n, -1) for x in "qkv"], 1).to(device)
    out, at = {}, 0
    for x in "qkv":
        w = d[x].shape[-1] * d[x].shape[-2]
        out[x] = base[:, at:at + w].view(*d[x].shape) if n else d[x].to(device)
        at += w
    for x in ("g", "beta", "A_log", "dt_bias"):
        out[x] = None if d[x] is None else d[x].to(device)
    return out


def verify(tokens, start, p, q, ua, us, max_drafts):
    """The definition, sums in 64 bits in index order."""
    batch = len(start) - 1
    out = torch.full((batch, max_drafts + 1), -1, dtype=torch.int32)
    acc = torch.zeros(batch, dtype=torch.int32)
    pn = p.numpy().astype(np.float64)
    qn = None if q is None else q.numpy().astype(np.float64)
    V = p.shape[1]
    for i in range(batch):
        a, n = int(start[i]), min(int(start[i + 1] - start[i]), max_drafts)
        c = 0
        while c < n:
            x = int(tokens[a + c])
            if not 0 <= x < V:
                break
            qx = 1.0 if qn is None else qn[a + c, x]
            if not float(ua[a + c]) * qx < pn[a + c + i, x]:
                break
            out[i, c] = x
            c += 1
        r = np.where(pn[a + i + c] > 0, pn[a + i + c], 0.0)
        if c < n:
            x = int(tokens[a + c])
            left = r.copy()
            if qn is None:
                if 0 <= x < V:
                    left[x] = 0
            else:
                left = np.maximum(r - np.where(qn[a + c] > 0, qn[a + c], 0.0), 0)
            if left.sum() > 0:
                r = left
        run = np.cumsum(r)
        hit = np.flatnonzero((run > float(us[i]) * run[-1]) & (r > 0))
        some = np.flatnonzero(r > 0)
        out[i, c] = int(hit[0]) if len(hit) else (int(some[-1]) if len(some) else 0)
        acc[i] = c + 1
    return out, acc
