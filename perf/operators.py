"""Measured cases of the gated delta rule (prefill and decode) and of draft verification.

Each case runs one operator: "prefill" (gdr_fwd_varlen), "decode" (gdr_update) or "verify" (sconv_verify_drafts), either as
the framework's call (own = True) or in its plain form in torch (own = False)."""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
CHUNK = 64          # tokens a step of the plain prefill


# ------------------------------------------------------------------ cases --

def _prefill(name, **kw):
    return dict(dict(name=name, op="prefill", hk=16, hv=32, dk=128, dv=128, nseq=1, max_len=1, lens_seed=1, n_pad=0,
                     lines=1, raw=True, l2norm=True), **kw)


def _decode(name, **kw):
    return dict(dict(name=name, op="decode", hk=16, hv=32, dk=128, dv=128, batch=1, seqlen=1, spec=False, n_pad=0, lines=4,
                     raw=True, l2norm=True), **kw)


def _verify(name, **kw):
    return dict(dict(name=name, op="verify", batch=1, drafts=3, ragged=False, lens_seed=1, vocab=32000, draft_probs=True),
                **kw)


def listed():
    return [
        # a short prompt behind the benchmark's 4096-channel convolution (8 * 128 * 2 + 16 * 128 channels)
        _prefill("prefill 128, 4096 channels", hk=8, hv=16, max_len=128),
        # the benchmark's long prefills at 8192 channels (16 * 128 * 2 + 32 * 128)
        _prefill("prefill 4195", max_len=4195),
        _prefill("prefill 14807", max_len=14807),
        # the varlen workload: 64 sequences of U[1, 2048] tokens, 256 cache lines, 4 padded entries
        _prefill("prefill 64 sequences", nseq=64, max_len=2048, lens_seed=7, n_pad=4, lines=256),
        # small ragged batch, odd head sizes, gates and norms computed by the caller
        _prefill("prefill ragged, heads 96/80", hk=4, hv=12, dk=96, dv=80, nseq=17, max_len=301, lens_seed=3, n_pad=1, lines=20,
                 raw=False, l2norm=False),
        # one decoding request: latency
        _decode("decode 1, 4096 channels", hk=8, hv=16),
        # the decode batch of the benchmark
        _decode("decode 64", batch=64, lines=80, n_pad=2),
        # a large serving batch
        _decode("decode 256", batch=256, lines=256),
        # the speculative workload: 64 requests of 4 tokens, every token's state saved
        _decode("decode 64 x 4, states saved", batch=64, seqlen=4, spec=True, lines=256),
        # one request's drafts: latency
        _verify("verify 1 x 3", vocab=32000),
        # the speculative batch against a large vocabulary
        _verify("verify 64 x 3", batch=64, vocab=131072),
        # a serving batch with ragged, deterministic drafts and an odd vocabulary
        _verify("verify 256 ragged", batch=256, drafts=7, ragged=True, lens_seed=5, vocab=100003, draft_probs=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("prefill", "prefill", "decode", "decode", "verify"))
    if kind == "verify":
        batch, drafts = _log_int(rng, 1, 256), rng.randint(1, 8)
        most = min(160000, (300 << 20) // (4 * batch * (drafts + 1)))
        c = _verify("", batch=batch, drafts=drafts, ragged=rng.random() < 0.5, lens_seed=rng.randint(1, 1 << 20),
                    vocab=_log_int(rng, 100, most), draft_probs=rng.random() < 0.6)
        del c["name"]
        return c
    hk = rng.choice((1, 2, 4, 8, 16))
    group = rng.choice((1, 2, 2, 3, 4))
    hv = min(hk * group, 32 // hk * hk)
    dk, dv = rng.choice((64, 128, 128, 96, 100, 72)), rng.choice((64, 128, 128, 80, 100, 40))
    raw = rng.random() < 0.6
    if kind == "prefill":
        nseq = 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
        max_len = _log_int(rng, 1, 14000 if nseq == 1 else min(4000, 100000 // nseq))
        n_pad = rng.randint(0, 2) if nseq > 4 else 0
        c = _prefill("", hk=hk, hv=hv, dk=dk, dv=dv, nseq=nseq, max_len=max_len, lens_seed=rng.randint(1, 1 << 20),
                     n_pad=n_pad, lines=nseq + rng.randint(0, 8), raw=raw, l2norm=raw or rng.random() < 0.5)
    else:
        batch = _log_int(rng, 1, 256)
        seqlen = rng.choice((1, 1, 2, 3, 4, 5))
        spec = seqlen > 1 and batch <= 64 and rng.random() < 0.7
        c = _decode("", hk=hk, hv=hv, dk=dk, dv=dv, batch=batch, seqlen=seqlen, spec=spec,
                    n_pad=rng.randint(0, 2) if batch > 4 else 0,
                    lines=batch * (seqlen if spec else 1) + rng.randint(0, 8), raw=raw, l2norm=raw or rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """Sequence lengths of a prefill case: one of max_len, or U[1, max_len]."""
    if case["nseq"] == 1:
        return [case["max_len"]]
    r = random.Random(case["lens_seed"])
    return [r.randint(1, case["max_len"]) for _ in range(case["nseq"])]


def _draft_counts(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(0, case["drafts"]) if case["ragged"] else case["drafts"] for _ in range(case["batch"])]


def _padded(case, n):
    """Batch positions that are padded."""
    return random.Random(1000 + n).sample(range(n), case["n_pad"])


# ---------------------------------------------------------------- prepare --

def _gates(shape, case, g):
    """Decay and write strength: raw projections with the layer's parameters, or computed ones in fp32."""
    hv = case["hv"]
    a_log = torch.log(torch.rand(hv, device=DEV, generator=g) * 15 + 1)
    dt = torch.exp(torch.rand(hv, device=DEV, generator=g) * math.log(100) + math.log(0.001))
    dt_bias = dt + torch.log(-torch.expm1(-dt))
    a = torch.randn(*shape, device=DEV, generator=g).bfloat16()
    b = torch.randn(*shape, device=DEV, generator=g).bfloat16()
    if case["raw"]:
        return dict(g=a, beta=b, A_log=a_log, dt_bias=dt_bias)
    return dict(g=-torch.exp(a_log) * torch.nn.functional.softplus(a.float() + dt_bias), beta=torch.sigmoid(b.float()),
                A_log=None, dt_bias=None)


def _qkv(rows, case, g):
    """q, k, v as views of one (rows, channels) buffer: the convolution's output after its SiLU."""
    hk, hv, dk, dv = (case[n] for n in ("hk", "hv", "dk", "dv"))
    x = torch.randn(rows, 2 * hk * dk + hv * dv, device=DEV, generator=g)
    x = (x * torch.sigmoid(x)).bfloat16()
    if not case["l2norm"]:           # the caller normalised them
        n = x[:, :2 * hk * dk].float().view(rows, 2 * hk, dk)
        x[:, :2 * hk * dk] = (n * torch.rsqrt((n * n).sum(-1, keepdim=True) + 1e-6)).view(rows, -1).bfloat16()
    return (x[:, :hk * dk].view(rows, hk, dk), x[:, hk * dk:2 * hk * dk].view(rows, hk, dk),
            x[:, 2 * hk * dk:].view(rows, hv, dv))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    hv, dk, dv, lines = case["hv"], case["dk"], case["dv"], case["lines"]
    s = dict(case=case, scale=dk ** -0.5, state=torch.randn(lines, hv, dv, dk, device=DEV, generator=g) * 0.2)
    if case["op"] == "prefill":
        lens = _lengths(case)
        n, total = len(lens), sum(lens)
        s["qsl"] = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device=DEV)
        s["q"], s["k"], s["v"] = _qkv(total, case, g)
        s.update(_gates((total, hv), case, g))
        s["out"] = torch.zeros(total, hv, dv, dtype=torch.bfloat16, device=DEV)
        s["has_init"] = (torch.rand(n, generator=host) < 0.5).to(DEV)
        ci = torch.randperm(lines, generator=host)[:n].to(torch.int32)
        ci[_padded(case, n)] = -1
        s["cache_indices"] = ci.to(DEV)
    else:
        n, steps = case["batch"], case["seqlen"]
        q, k, v = _qkv(n * steps, case, g)
        s["q"], s["k"], s["v"] = (t.unflatten(0, (n, steps)) for t in (q, k, v))
        s.update(_gates((n, steps, hv), case, g))
        s["out"] = torch.zeros(n, steps, hv, dv, dtype=torch.bfloat16, device=DEV)
        order = torch.randperm(lines, generator=host).to(torch.int32)
        s["accepted"] = None
        if case["spec"]:
            ci = order[:n * steps].view(n, steps).clone()
            s["accepted"] = torch.randint(1, steps + 1, (n,), generator=host, dtype=torch.int32).to(DEV)
        else:
            ci = order[:n].clone()
        ci[_padded(case, n)] = -1
        s["cache_indices"] = ci.to(DEV)
    return s


def _prepare_verify(case, g):
    batch, vocab = case["batch"], case["vocab"]
    counts = _draft_counts(case)
    start = torch.tensor([0] + np.cumsum(counts).tolist(), dtype=torch.int32, device=DEV)
    nd = sum(counts)
    rows = nd + batch
    logits = torch.randn(rows, vocab, device=DEV, generator=g).mul_(3)
    # sampling filters leave most of the vocabulary of every other row at exactly zero
    logits[::2].masked_fill_(logits[::2] < 3, float("-inf"))
    logits[:, 0] = 1.0
    target = torch.softmax(logits, -1)
    of_draft = torch.cat([torch.arange(c, device=DEV) + int(o) + i for i, (c, o) in enumerate(zip(counts, start.tolist()))]
                         ) if nd else torch.zeros(0, dtype=torch.long, device=DEV)
    near = logits[of_draft]
    near.add_(torch.randn(near.shape, device=DEV, generator=g))
    if case["draft_probs"]:
        q = torch.softmax(near, -1)
        near.sub_(torch.log(-torch.log(torch.rand(near.shape, device=DEV, generator=g).clamp_(1e-20, 1 - 1e-7))))
    else:
        q = None
    tokens = near.argmax(-1).to(torch.int32) if nd else torch.zeros(0, dtype=torch.int32, device=DEV)
    return dict(case=case, draft_tokens=tokens, draft_start_loc=start, target_probs=target, draft_probs=q,
                accept_uniform=torch.rand(nd, device=DEV, generator=g), sample_uniform=torch.rand(batch, device=DEV, generator=g))


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "prefill":
        return _plain_prefill(state)
    if op == "decode":
        return _plain_decode(state)
    return _plain_verify(state)


def _own(s, op):
    import causal_depthwise_short_conv1d_amd as S
    if op == "verify":
        tokens, accepted = S.sconv_verify_drafts(s["draft_tokens"], s["draft_start_loc"], s["target_probs"], s["draft_probs"],
                                                 s["accept_uniform"], s["sample_uniform"], max_drafts=s["case"]["drafts"])
        return {"tokens": tokens, "accepted": accepted}
    opts = dict(A_log=s["A_log"], dt_bias=s["dt_bias"], scale=s["scale"], use_qk_l2norm=s["case"]["l2norm"], out=s["out"])
    if op == "prefill":
        S.gdr_fwd_varlen(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["qsl"], cache_indices=s["cache_indices"],
                         has_initial_state=s["has_init"], **opts)
    else:
        spec = s["case"]["spec"]
        S.gdr_update(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], cache_indices=s["cache_indices"],
                     num_accepted_tokens=s["accepted"], output_state_indices=s["cache_indices"] if spec else None, **opts)
    return {"out": s["out"], "state": s["state"]}


def _plain_inputs(s):
    """q, k, v, log decay and write strength in 32 bits (the decay in 64), key heads repeated over their value heads."""
    case = s["case"]
    rep = case["hv"] // case["hk"]
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    if case["l2norm"]:
        q, k = (t * torch.rsqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    q, k = (t.repeat_interleave(rep, dim=-2) for t in (q * s["scale"], k))
    if case["raw"]:
        x = s["g"].double() + s["dt_bias"].double()
        decay = -torch.exp(s["A_log"].double()) * torch.where(x > 20, x, torch.log1p(torch.exp(x)))
        beta = 1 / (1 + torch.exp(-s["beta"].float()))
    else:
        decay, beta = s["g"].double(), s["beta"]
    return q, k, v, decay, beta


def _plain_prefill(s):
    case = s["case"]
    qsl, ci = s["qsl"], s["cache_indices"].long()
    n, longest = case["nseq"], case["max_len"]
    nc = -(-longest // CHUNK)
    span = nc * CHUNK
    # the packed rows laid out (sequence, head, chunk, token); what lies behind a sequence's end has no key, value or decay
    t = torch.arange(span, device=DEV)
    row = qsl[:-1, None].long() + t
    live = ((row < qsl[1:, None]) & (ci >= 0)[:, None])
    row = torch.where(live, row, torch.zeros_like(row))

    def lay(x):
        x = x[row] * live.view(n, span, *([1] * (x.dim() - 1)))
        return x.view(n, nc, CHUNK, *x.shape[2:]).transpose(2, 3).transpose(1, 2)      # (n, head, chunk, token, ...)

    q, k, v, decay, beta = (lay(x) for x in _plain_inputs(s))
    G = decay.cumsum(-1)
    diff = G[..., :, None] - G[..., None, :]
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = torch.where(tri, diff, float("-inf")).exp().float()
    kT = k.transpose(-1, -2).contiguous()
    P = (q @ kT) * D
    A = (k @ kT) * D * beta[..., None] * tri.tril(-1)
    T = torch.eye(CHUNK, device=DEV).expand(A.shape).clone()
    for i in range(1, CHUNK):                          # (I + A)^-1, a row from those above it
        T[..., i, :i] = -(A[..., i:i + 1, :i] @ T[..., :i, :i].contiguous()).squeeze(-2)
    eG, eL = G.exp().float(), G[..., -1].exp().float()
    U = T @ (v * beta[..., None])
    W = T @ (k * (beta * eG)[..., None])
    qG = q * eG[..., None]
    kG = (k * (G[..., -1:] - G).exp().float()[..., None]).transpose(-1, -2).contiguous()
    line = ci.clamp(min=0)
    S = torch.where(s["has_init"].view(-1, 1, 1, 1), s["state"][line], 0.0).transpose(-1, -2).contiguous()    # (n, head, dk, dv)
    o = torch.empty(n, case["hv"], nc, CHUNK, case["dv"], device=DEV)
    for c in range(nc):
        vn = U[:, :, c] - W[:, :, c] @ S
        o[:, :, c] = qG[:, :, c] @ S + P[:, :, c] @ vn
        S = S * eL[:, :, c, None, None] + kG[:, :, c] @ vn
    o = o.transpose(1, 2).transpose(2, 3).reshape(n, span, case["hv"], case["dv"])
    s["out"][row[live]] = o[live].to(s["out"].dtype)
    s["state"][ci[ci >= 0]] = S.transpose(-1, -2)[ci >= 0]
    return {"out": s["out"], "state": s["state"]}


def _plain_decode(s):
    case = s["case"]
    ci = s["cache_indices"].long()
    spec = case["spec"]
    read = ci.gather(1, s["accepted"].long()[:, None] - 1)[:, 0] if spec else ci
    live = read >= 0
    q, k, v, decay, beta = (x[live] for x in _plain_inputs(s))
    e = decay.exp().float()
    S = s["state"][read[live]]
    for t in range(case["seqlen"]):
        S = S * e[:, t, :, None, None]
        u = (v[:, t] - (S * k[:, t, :, None, :]).sum(-1)) * beta[:, t, :, None]
        S = S + u[..., None] * k[:, t, :, None, :]
        s["out"][live, t] = (S * q[:, t, :, None, :]).sum(-1).to(s["out"].dtype)
        if spec:
            s["state"][ci[live, t]] = S
    if not spec:
        s["state"][ci[live]] = S
    return {"out": s["out"], "state": s["state"]}


def _plain_verify(s):
    case = s["case"]
    batch, most, vocab = case["batch"], case["drafts"], case["vocab"]
    start, x = s["draft_start_loc"].long(), s["draft_tokens"].long()
    p, q = s["target_probs"], s["draft_probs"]
    n = start[1:] - start[:-1]
    j = torch.arange(most, device=DEV)
    has = j < n[:, None]
    d = torch.where(has, start[:-1, None] + j, 0)
    row = d + torch.arange(batch, device=DEV)[:, None]
    if x.numel():
        tok = x[d]
        px = p[row, tok].double()
        qx = q[d, tok].double() if q is not None else torch.ones_like(px)
        ok = has & (s["accept_uniform"][d].double() * qx < px)
    else:
        tok, ok = d, has & False
    count = ok.long().cumprod(1).sum(1)                # accepted before the first refusal
    last = start[:-1] + torch.arange(batch, device=DEV) + count
    r = p[last].double()
    refused = count < n
    if x.numel():
        dr = torch.where(refused, start[:-1] + count, 0)
        if q is not None:
            take = q[dr].double()
        else:
            take = torch.zeros(batch, vocab, device=DEV, dtype=torch.float64).scatter_(1, x[dr][:, None], float("inf"))
        left = (r - take).clamp(min=0)
        left = torch.where((left.sum(1) > 0)[:, None], left, r)
        r = torch.where(refused[:, None], left, r)
    c = r.cumsum(1)
    pick = (c <= s["sample_uniform"].double()[:, None] * c[:, -1:]).sum(1)
    top = torch.where(r > 0, torch.arange(vocab, device=DEV), 0).amax(1)
    pick = torch.minimum(pick, top)
    tokens = torch.full((batch, most + 1), -1, dtype=torch.int32, device=DEV)
    k = torch.arange(most + 1, device=DEV)
    tokens[:, :most] = torch.where(j < count[:, None], tok, -1).to(torch.int32)
    tokens = torch.where(k == count[:, None], pick[:, None].to(torch.int32), tokens)
    return {"tokens": tokens, "accepted": (count + 1).to(torch.int32)}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_verify(s) if case["op"] == "verify" else _exact_delta(s)


def _exact_delta(s):
    """The recurrence, a token at a time, in 64 bits."""
    case = s["case"]
    f = torch.float64
    q, k, v = (s[n].to(f) for n in ("q", "k", "v"))
    if case["l2norm"]:
        q = q / torch.sqrt(q.square().sum(-1, keepdim=True) + 1e-6)
        k = k / torch.sqrt(k.square().sum(-1, keepdim=True) + 1e-6)
    if case["raw"]:
        z = s["g"].to(f) + s["dt_bias"].to(f)
        alpha = torch.exp(-torch.exp(s["A_log"].to(f)) * torch.logaddexp(z, torch.zeros_like(z)))
        beta = torch.sigmoid(s["beta"].to(f))
    else:
        alpha, beta = torch.exp(s["g"].to(f)), s["beta"].to(f)
    heads = torch.arange(case["hv"], device=DEV) // (case["hv"] // case["hk"])
    out, state = s["out"].to(f), s["state"].to(f)
    ci = s["cache_indices"].long().cpu()

    def step(S, qt, kt, vt, at, bt):
        qt, kt = qt[:, heads], kt[:, heads]
        S = S * at[..., None, None]
        seen = torch.matmul(S, kt.unsqueeze(-1)).squeeze(-1)
        S = S + ((vt - seen) * bt[..., None]).unsqueeze(-1) * kt.unsqueeze(-2)
        return S, torch.matmul(S, qt.unsqueeze(-1)).squeeze(-1) * s["scale"]

    if case["op"] == "decode":
        acc = s["accepted"].cpu().long() if case["spec"] else None
        src = ci[torch.arange(len(ci)), acc - 1] if case["spec"] else ci
        at = (src >= 0).nonzero()[:, 0].to(DEV)
        S = state[src[src >= 0].to(DEV)].clone()
        for t in range(case["seqlen"]):
            S, out[at, t] = step(S, q[at, t], k[at, t], v[at, t], alpha[at, t], beta[at, t])
            if case["spec"]:
                state[ci.to(DEV)[at, t]] = S
        if not case["spec"]:
            state[src[src >= 0].to(DEV)] = S
        return {"out": out, "state": state}
    first = s["qsl"].tolist()
    lens = [b - a for a, b in zip(first, first[1:])]
    order = sorted((i for i in range(len(lens)) if ci[i] >= 0), key=lambda i: -lens[i])
    ids = torch.tensor(order, device=DEV)
    begin = s["qsl"].long()[ids]
    line = ci.to(DEV)[ids]
    S = state[line] * s["has_init"][ids].to(f).view(-1, 1, 1, 1)
    live = len(order)
    for t in range(max(lens[i] for i in order)):
        while live and lens[order[live - 1]] <= t:
            live -= 1
        at = begin[:live] + t
        S[:live], out[at] = step(S[:live], q[at], k[at], v[at], alpha[at], beta[at])
    state[line] = S
    return {"out": out, "state": state}


def _exact_verify(s):
    """The definition on the host, a request at a time, in the host's longest floating type."""
    start = s["draft_start_loc"].tolist()
    x, ua, us = s["draft_tokens"].tolist(), s["accept_uniform"].tolist(), s["sample_uniform"].tolist()
    p, q = s["target_probs"].cpu().numpy(), None if s["draft_probs"] is None else s["draft_probs"].cpu().numpy()
    batch, most = s["case"]["batch"], s["case"]["drafts"]
    tokens = np.full((batch, most + 1), -1, dtype=np.int32)
    accepted = np.zeros(batch, dtype=np.int32)
    for i in range(batch):
        n, k = start[i + 1] - start[i], 0
        while k < n:
            d = start[i] + k
            if not ua[d] * (1.0 if q is None else float(q[d, x[d]])) < float(p[d + i, x[d]]):
                break
            tokens[i, k] = x[d]
            k += 1
        r = p[start[i] + i + k].astype(np.longdouble)
        if k < n:
            d = start[i] + k
            left = r.copy()
            if q is None:
                left[x[d]] = 0
            else:
                left = np.maximum(r - q[d].astype(np.longdouble), 0)
            if left.sum() > 0:
                r = left
        c = np.cumsum(r)
        over = np.flatnonzero(c > np.longdouble(us[i]) * c[-1])
        some = np.flatnonzero(r > 0)
        tokens[i, k] = over[0] if len(over) else (some[-1] if len(some) else 0)
        accepted[i] = k + 1
    return {"tokens": torch.from_numpy(tokens), "accepted": torch.from_numpy(accepted)}


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "verify":
        counts = _draft_counts(case)
        # a row of the target a request, one of the draft where one may be refused, and the drafts themselves
        rows = len(counts) + (sum(c > 0 for c in counts) if case["draft_probs"] else 0)
        return {"bytes": 4 * rows * case["vocab"] + 16 * sum(counts) + 4 * len(counts) * (case["drafts"] + 4),
                "flops": 3 * rows * case["vocab"]}
    hk, hv, dk, dv = (case[n] for n in ("hk", "hv", "dk", "dv"))
    gate = 4 if case["raw"] else 8
    if case["op"] == "prefill":
        lens = _lengths(case)
        pads = set(_padded(case, len(lens)))
        lens = [n for i, n in enumerate(lens) if i not in pads]
        tokens, states = sum(lens), 1.5 * len(lens)      # read for half of them, written for all
    else:
        live = case["batch"] - case["n_pad"]
        tokens, states = live * case["seqlen"], live * (1 + (case["seqlen"] if case["spec"] else 1))
    return {"bytes": tokens * (2 * (2 * hk * dk + 2 * hv * dv) + gate * hv) + 4 * states * hv * dv * dk,
            "flops": 7 * tokens * hv * dv * dk}
