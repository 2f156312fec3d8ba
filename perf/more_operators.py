"""Measured cases of the selective state space scan (prompts and decode) and of the gated group norm behind it.

Each case runs one operator: "prompt" (ssm_fwd_varlen), "decode" (ssm_update) or "norm" (sconv_group_norm), either as the
framework's call (own = True) or in its plain form in torch (own = False). The scan has two forms: one decay a head
(form "head": heads of head_dim channels) and one a channel and state (form "channel")."""
import math
import random

import torch

own = False

DEV = "cuda"
CHUNK = 64          # tokens a step of the plain scan


# ------------------------------------------------------------------ cases --

def _scan(name, **kw):
    return dict(dict(name=name, form="head", heads=128, head_dim=64, groups=8, state=128, gate=False, skip=True, raw=True, n_pad=0),
                **kw)


def _prompt(name, **kw):
    return _scan(name, **dict(dict(op="prompt", nseq=1, max_len=1, lens_seed=1, lines=1), **kw))


def _decode(name, **kw):
    return _scan(name, **dict(dict(op="decode", batch=1, seqlen=1, spec=False, lines=4), **kw))


def _norm(name, **kw):
    return dict(dict(name=name, op="norm", rows=1, channels=8192, group=1024, kind="rms", gate="first", activation="silu",
                     shared=False, bias=False), **kw)


def listed():
    return [
        # a short prompt: latency
        _prompt("prompt 128, 4096 channels", heads=64, max_len=128),
        # the benchmark's long prompts at 8192 channels
        _prompt("prompt 4195", max_len=4195),
        _prompt("prompt 14807", max_len=14807),
        # the varlen workload: 64 sequences of U[1, 2048] tokens, 256 cache lines, 4 padded entries
        _prompt("prompt 64 sequences, 4096 channels", heads=64, nseq=64, max_len=2048, lens_seed=7, n_pad=4, lines=256),
        # odd heads, one group, step sizes computed by the caller, gated output, small ragged batch
        _prompt("prompt ragged, heads 80 x 96", heads=12, head_dim=80, groups=1, state=96, nseq=17, max_len=301, lens_seed=3,
                n_pad=1, lines=20, raw=False, gate=True),
        # a decay for every channel and state, gated output, as layers without heads have it
        _prompt("prompt 4195, channel decays", form="channel", heads=1, head_dim=8192, groups=1, state=16, max_len=4195, gate=True),
        # one decoding request: latency
        _decode("decode 1, 4096 channels", heads=64),
        # a large serving batch
        _decode("decode 256", batch=256, lines=260, n_pad=2),
        # the speculative workload: 64 requests of 4 tokens, every token's state saved
        _decode("decode 64 x 4, states saved", batch=64, seqlen=4, spec=True, lines=256),
        # channel decays, a serving batch
        _decode("decode 64, channel decays", form="channel", heads=1, head_dim=8192, groups=1, state=16, batch=64, lines=80,
                gate=True),
        # behind the long prompt: gate, then the norm of eight groups
        _norm("norm 14807 x 8192", rows=14807),
        # behind the gated delta rule of the speculative batch: the norm of every head, weights shared by the heads, then the gate
        _norm("norm 256 rows, heads of 128", rows=256, channels=4096, group=128, gate="last", shared=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "decode", "decode", "norm"))
    if op == "norm":
        group = rng.choice((64, 128, 128, 256, 512, 1024, 2048, 4096, 8192, 80, 100, 1000))
        groups = rng.randint(1, max(1, min(64, 8192 // group)))
        c = _norm("", rows=_log_int(rng, 1, 14000), channels=group * groups, group=group, kind=rng.choice(("rms", "rms", "layer")),
                  gate=rng.choice(("first", "last", "none")), activation=rng.choice(("silu", "silu", "sigmoid")),
                  shared=rng.random() < 0.4, bias=rng.random() < 0.3)
        del c["name"]
        return c
    if rng.random() < 0.65:
        groups = rng.choice((1, 1, 2, 4, 8))
        dim = rng.choice((64, 64, 64, 128, 32, 80, 96))
        heads = groups * rng.randint(1, max(1, 8192 // dim // groups))
        sizes = dict(form="head", heads=heads, head_dim=dim, groups=groups, state=rng.choice((128, 128, 64, 96, 256, 40, 16)))
        if sizes["state"] > 128:
            sizes["heads"] = groups * max(1, heads // groups // 4)
    else:
        groups = rng.choice((1, 1, 1, 2))
        sizes = dict(form="channel", heads=groups, groups=groups, head_dim=rng.choice((64, 100, 1024, 1536, 2048, 4096, 8192)) // groups,
                     state=rng.choice((16, 16, 16, 8, 32)))
    sizes.update(gate=rng.random() < 0.4, skip=rng.random() < 0.8, raw=rng.random() < 0.6)
    if op == "prompt":
        nseq = 1 if rng.random() < 0.4 else _log_int(rng, 2, 64)
        wide = 1 if sizes["form"] == "head" and sizes["state"] <= 128 else 4
        max_len = _log_int(rng, 1, (14000 if nseq == 1 else min(4000, 64000 // nseq)) // wide)
        c = _prompt("", nseq=nseq, max_len=max_len, lens_seed=rng.randint(1, 1 << 20), n_pad=rng.randint(0, 2) if nseq > 4 else 0,
                    lines=nseq + rng.randint(0, 8), **sizes)
    else:
        batch = _log_int(rng, 1, 256)
        seqlen = rng.choice((1, 1, 2, 3, 4, 5))
        spec = seqlen > 1 and batch <= 48 and rng.random() < 0.7
        c = _decode("", batch=batch, seqlen=seqlen, spec=spec, n_pad=rng.randint(0, 2) if batch > 4 else 0,
                    lines=batch * (seqlen if spec else 1) + rng.randint(0, 8), **sizes)
    del c["name"]
    return c


def _lengths(case):
    """Sequence lengths of a prompt case: one of max_len, or U[1, max_len]."""
    if case["nseq"] == 1:
        return [case["max_len"]]
    r = random.Random(case["lens_seed"])
    return [r.randint(1, case["max_len"]) for _ in range(case["nseq"])]


def _padded(case, n):
    """Batch positions that are padded."""
    return random.Random(1000 + n).sample(range(n), case["n_pad"])


# ---------------------------------------------------------------- prepare --

def _layer(case, lead, g):
    """A scan's inputs with leading dimensions `lead`: x, B and C as views of one buffer (the convolution's output after its
    SiLU), the step sizes as the layer's bf16 projection or computed in fp32, and the layer's weights."""
    h, p, gr, n = (case[k] for k in ("heads", "head_dim", "groups", "state"))
    head = case["form"] == "head"
    rows = math.prod(lead)
    xbc = torch.randn(rows, h * p + 2 * gr * n, device=DEV, generator=g)
    xbc = (xbc * torch.sigmoid(xbc)).bfloat16()
    s = {"B": xbc[:, h * p:h * p + gr * n].view(*lead, gr, n), "C": xbc[:, h * p + gr * n:].view(*lead, gr, n)}
    s["x"] = xbc[:, :h * p].view(*lead, h, p) if head else xbc[:, :h * p].view(*lead, h * p)
    one = (h,) if head else (h * p,)                  # what has a step size
    dt = torch.exp(torch.rand(one, device=DEV, generator=g) * math.log(100) + math.log(0.001))
    bias = dt + torch.log(-torch.expm1(-dt))
    step = torch.randn(*lead, *one, device=DEV, generator=g).bfloat16()
    if case["raw"]:
        s.update(dt=step, dt_bias=bias)
    else:
        s.update(dt=torch.nn.functional.softplus(step.float() + bias), dt_bias=None)
    if head:
        s["A"] = -(torch.rand(h, device=DEV, generator=g) * 15 + 1)
    else:
        near = 1 + 0.1 * torch.randn(h * p, n, device=DEV, generator=g).clamp(-3, 3)
        s["A"] = -torch.arange(1, n + 1, device=DEV, dtype=torch.float32) * near
    s["D"] = 1 + 0.1 * torch.randn(one, device=DEV, generator=g) if case["skip"] else None
    s["z"] = torch.randn(s["x"].shape, device=DEV, generator=g).bfloat16() if case["gate"] else None
    s["out"] = torch.zeros(s["x"].shape, dtype=torch.bfloat16, device=DEV)
    shape = (case["lines"], h, p, n) if head else (case["lines"], h * p, n)
    s["state"] = torch.randn(shape, device=DEV, generator=g) * 0.2
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    if case["op"] == "norm":
        return _prepare_norm(case, g)
    lines = case["lines"]
    order = torch.randperm(lines, generator=host).to(torch.int32)
    if case["op"] == "prompt":
        lens = _lengths(case)
        n = len(lens)
        s = _layer(case, (sum(lens),), g)
        s["qsl"] = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
        s["has_init"] = (torch.rand(n, generator=host) < 0.5).to(DEV)
        ci = order[:n].clone()
    else:
        n, steps = case["batch"], case["seqlen"]
        s = _layer(case, (n, steps), g)
        s["accepted"] = None
        if case["spec"]:
            ci = order[:n * steps].view(n, steps).clone()
            s["accepted"] = torch.randint(1, steps + 1, (n,), generator=host, dtype=torch.int32).to(DEV)
        else:
            ci = order[:n].clone()
    ci[_padded(case, n)] = -1
    s.update(case=case, cache_indices=ci.to(DEV))
    return s


def _prepare_norm(case, g):
    rows, channels, group = case["rows"], case["channels"], case["group"]
    x = torch.randn(rows, channels, device=DEV, generator=g)
    x *= torch.exp(torch.randn(rows, 1, device=DEV, generator=g))      # rows of different size
    own_weights = group if case["shared"] else channels
    return dict(case=case, x=x.bfloat16(), out=torch.zeros(rows, channels, dtype=torch.bfloat16, device=DEV),
                z=torch.randn(rows, channels, device=DEV, generator=g).bfloat16() if case["gate"] != "none" else None,
                weight=(1 + 0.1 * torch.randn(own_weights, device=DEV, generator=g)).bfloat16(),
                bias=(0.1 * torch.randn(own_weights, device=DEV, generator=g)).bfloat16() if case["bias"] else None)


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "norm":
        return _plain_norm(state)
    if op == "prompt":
        return _plain_prompt(state)
    return _plain_decode(state)


def _own(s, op):
    import causal_depthwise_short_conv1d_amd as S
    case = s["case"]
    if op == "norm":
        return S.sconv_group_norm(s["x"], case["group"], weight=s["weight"], bias=s["bias"], z=s["z"], norm=case["kind"],
                                  activation=case["activation"], gate_first=case["gate"] == "first", out=s["out"])
    opts = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=case["raw"], out=s["out"])
    if op == "prompt":
        S.ssm_fwd_varlen(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], s["qsl"], cache_indices=s["cache_indices"],
                         has_initial_state=s["has_init"], **opts)
    else:
        S.ssm_update(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], cache_indices=s["cache_indices"],
                     num_accepted_tokens=s["accepted"], output_state_indices=s["cache_indices"] if case["spec"] else None, **opts)
    return {"out": s["out"], "state": s["state"]}


def _heads(case, t):
    """A tensor of channels as (heads, head_dim); with groups as heads in the channel form."""
    return t if case["form"] == "head" else t.unflatten(-1, (case["heads"], case["head_dim"]))


def _plain_inputs(s):
    """x, the step sizes (64 bits), B and C repeated over their heads, in 32 bits, and A; step sizes and A have a channel
    (and state) dimension, of one element in the head form."""
    case = s["case"]
    step = s["dt"].double()
    if case["raw"]:
        step = step + s["dt_bias"].double()
        step = torch.where(step > 20, step, torch.log1p(torch.exp(step)))
    rep = case["heads"] // case["groups"]
    B, C = (s[n].float().repeat_interleave(rep, dim=-2) for n in ("B", "C"))
    if case["form"] == "head":
        return s["x"].float(), step[..., None], B, C, s["A"].double()[:, None, None]
    return _heads(case, s["x"]).float(), _heads(case, step), B, C, s["A"].double().unflatten(0, (case["heads"], case["head_dim"]))


def _finish(s, y, at=None):
    """The skip and the gate, in 32 bits, on y (heads, head_dim last); `at`: those rows of x and z."""
    case = s["case"]
    pick = (lambda t: _heads(case, t if at is None else t[at]).float())
    if s["D"] is not None:
        y = y + pick(s["x"]) * (s["D"][:, None] if case["form"] == "head" else _heads(case, s["D"]))
    if s["z"] is not None:
        z = pick(s["z"])
        y = y * (z / (1 + torch.exp(-z)))
    return (y if case["form"] == "head" else y.flatten(-2)).to(s["out"].dtype)


def _plain_prompt(s):
    case = s["case"]
    qsl, ci = s["qsl"], s["cache_indices"].long()
    n, longest = case["nseq"], case["max_len"]
    nc = -(-longest // CHUNK)
    span = nc * CHUNK
    # the packed rows laid out (sequence, chunk, token); what lies behind a sequence's end has no step
    t = torch.arange(span, device=DEV)
    row = qsl[:-1, None].long() + t
    live = (row < qsl[1:, None]) & (ci >= 0)[:, None]
    row = torch.where(live, row, torch.zeros_like(row))
    x, step, B, C, A = _plain_inputs(s)

    def lay(v):
        v = v[row] * live.view(n, span, *([1] * (v.dim() - 1)))
        return v.view(n, nc, CHUNK, *v.shape[2:])

    heads, P, N = case["heads"], case["head_dim"], case["state"]
    line = ci.clamp(min=0)
    S = torch.where(s["has_init"].view(-1, 1, 1, 1), s["state"].view(-1, heads, P, N)[line], 0.0)
    form = _head_chunks if case["form"] == "head" else _channel_chunks
    y, S = form(lay(x), lay(step), lay(B), lay(C), A, S)
    y = y.reshape(n, span, heads, P)[live]
    s["out"][row[live]] = _finish(s, y, row[live])
    s["state"].view(-1, heads, P, N)[ci[ci >= 0]] = S[ci >= 0]
    return {"out": s["out"], "state": s["state"]}


def _head_chunks(x, step, B, C, A, S):
    """Chunks of tokens as products: (sequence, chunk, token, head, ...) in, y likewise, and the states after the last."""
    n, nc = x.shape[:2]
    x, B, C = (v.transpose(2, 3).contiguous() for v in (x, B, C))           # (n, nc, head, token, ...)
    step = step.squeeze(-1).transpose(2, 3)
    G = (step * A.view(-1, 1)).cumsum(-1)
    u = x * step[..., None].float()
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEV).tril()
    D = torch.where(tri, G[..., :, None] - G[..., None, :], float("-inf")).exp().float()
    y = ((C @ B.transpose(-1, -2).contiguous()) * D) @ u
    del D
    left = (G[..., -1:] - G).exp().float()
    add = (u * left[..., None]).transpose(-1, -2).contiguous() @ B          # (n, nc, head, head_dim, state)
    C = C * G.exp().float()[..., None]
    keep = G[..., -1].exp().float()
    for c in range(nc):
        y[:, c] += C[:, c] @ S.transpose(-1, -2).contiguous()
        S = S * keep[:, c, :, None, None] + add[:, c]
    return y.transpose(2, 3), S


def _channel_chunks(x, step, B, C, A, S):
    """The tokens of all chunks at once, one after the other, from empty states; then what the states before add."""
    n, nc, _, heads, P = x.shape
    G = (step.cumsum(2))                                                      # (n, nc, token, head, channel)
    u = x * step.float()
    h = torch.zeros(n, nc, heads, P, S.shape[-1], device=DEV)
    y = torch.empty_like(x)
    for t in range(CHUNK):
        h = h * (step[:, :, t, :, :, None].float() * A.float()).exp() + u[:, :, t, :, :, None] * B[:, :, t, :, None, :]
        y[:, :, t] = (h * C[:, :, t, :, None, :]).sum(-1)
    before = torch.empty_like(h)
    keep = (G[:, :, -1, :, :, None] * A).exp().float()
    for c in range(nc):
        before[:, c] = S
        S = S * keep[:, c] + h[:, c]
    for t in range(CHUNK):
        y[:, :, t] += (before * (G[:, :, t, :, :, None].float() * A.float()).exp() * C[:, :, t, :, None, :]).sum(-1)
    return y, S


def _plain_decode(s):
    case = s["case"]
    ci = s["cache_indices"].long()
    spec = case["spec"]
    read = ci.gather(1, s["accepted"].long()[:, None] - 1)[:, 0] if spec else ci
    live = read >= 0
    x, step, B, C, A = _plain_inputs(s)
    x, step, B, C = (v[live] for v in (x, step, B, C))
    state = s["state"].view(-1, case["heads"], case["head_dim"], case["state"])
    S = state[read[live]]
    ys = []
    for t in range(case["seqlen"]):
        S = S * (step[:, t, :, :, None] * A).exp().float() + (x[:, t] * step[:, t].float())[..., None] * B[:, t, :, None, :]
        ys.append((S * C[:, t, :, None, :]).sum(-1))
        if spec:
            state[ci[live, t]] = S
    s["out"][live] = _finish(s, torch.stack(ys, 1), live)
    if not spec:
        state[ci[live]] = S
    return {"out": s["out"], "state": s["state"]}


def _plain_norm(s):
    case = s["case"]
    rows, group = case["rows"], case["group"]
    x = s["x"].float().view(rows, -1, group)
    w = s["weight"].float()
    w = w if case["shared"] else w.view(-1, group)
    gate = None
    if s["z"] is not None:
        z = s["z"].float().view(rows, -1, group)
        gate = 1 / (1 + torch.exp(-z))
        gate = z * gate if case["activation"] == "silu" else gate
        if case["gate"] == "first":
            x = x * gate
    if case["kind"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w
    if s["bias"] is not None:
        b = s["bias"].float()
        y = y + (b if case["shared"] else b.view(-1, group))
    if gate is None:
        e = 1 / (1 + torch.exp(-y))
        y = y * e if case["activation"] == "silu" else e
    elif case["gate"] == "last":
        y = y * gate
    s["out"].copy_(y.view(rows, -1))
    return s["out"]


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] == "norm" else _exact_scan(s)


def _exact_norm(s):
    case = s["case"]
    f = torch.float64
    groups = case["channels"] // case["group"]
    cut = (lambda t: torch.stack(t.to(f).chunk(groups, dim=-1), dim=-2))         # (..., group, channel)
    wide = (lambda t: None if t is None else cut(t.repeat(groups) if case["shared"] else t))
    act = (lambda t: t * torch.sigmoid(t)) if case["activation"] == "silu" else torch.sigmoid
    v, w, b = cut(s["x"]), wide(s["weight"]), wide(s["bias"])
    if case["gate"] == "first":
        v = v * act(cut(s["z"]))
    off = v.mean(-1, keepdim=True) if case["kind"] == "layer" else 0.0
    v = (v - off) / torch.sqrt(torch.square(v - off).mean(-1, keepdim=True) + 1e-5) * w
    v = v if b is None else v + b
    v = act(v) if case["gate"] == "none" else v * act(cut(s["z"])) if case["gate"] == "last" else v
    return v.flatten(-2)


def _exact_scan(s):
    """The recurrence, a token at a time, in 64 bits."""
    case = s["case"]
    f = torch.float64
    H, P, N = case["heads"], case["head_dim"], case["state"]
    per_head = case["form"] == "head"
    of_head = torch.arange(H, device=DEV) // (H // case["groups"])
    lead = s["x"].shape[:1 if case["op"] == "prompt" else 2]
    x = s["x"].reshape(*lead, H, P)
    z = None if s["z"] is None else s["z"].reshape(*lead, H, P)
    wide = (lambda t: t[..., None].expand(*t.shape, P) if per_head else t.unflatten(-1, (H, P)))
    A = (s["A"].to(f)[:, None, None] if per_head else s["A"].to(f).view(H, P, N))
    D = None if s["D"] is None else wide(s["D"].to(f))
    bias = None if s["dt_bias"] is None else wide(s["dt_bias"].to(f))
    dt = s["dt"]
    out = s["out"].to(f).reshape(*lead, H, P)
    state = s["state"].to(f).view(-1, H, P, N)
    ci = s["cache_indices"].long().cpu()

    def step(S, at):
        d = wide(dt[at].to(f))
        if bias is not None:
            d = torch.logaddexp(d + bias, torch.zeros_like(d))
        xt = x[at].to(f)
        S = S * torch.exp(d[..., None] * A) + (d * xt)[..., None] * s["B"][at].to(f)[:, of_head].unsqueeze(-2)
        y = torch.matmul(S, s["C"][at].to(f)[:, of_head].unsqueeze(-1)).squeeze(-1)
        if D is not None:
            y = y + D * xt
        if z is not None:
            y = y * torch.nn.functional.silu(z[at].to(f))
        return S, y

    if case["op"] == "decode":
        acc = s["accepted"].cpu().long() if case["spec"] else None
        src = ci[torch.arange(len(ci)), acc - 1] if case["spec"] else ci
        at = (src >= 0).nonzero()[:, 0].to(DEV)
        S = state[src[src >= 0].to(DEV)].clone()
        for t in range(case["seqlen"]):
            S, out[at, t] = step(S, (at, t))
            if case["spec"]:
                state[ci.to(DEV)[at, t]] = S
        if not case["spec"]:
            state[src[src >= 0].to(DEV)] = S
        return {"out": out.view(s["out"].shape), "state": state.view(s["state"].shape)}
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
        S[:live], out[at] = step(S[:live], at)
    state[line] = S
    return {"out": out.view(s["out"].shape), "state": state.view(s["state"].shape)}


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["channels"]
        weights = (1 + case["bias"]) * (case["group"] if case["shared"] else case["channels"])
        return {"bytes": 2 * n * (3 if case["gate"] != "none" else 2) + 2 * weights, "flops": 10 * n}
    H, P, G, N = (case[k] for k in ("heads", "head_dim", "groups", "state"))
    steps = H if case["form"] == "head" else H * P
    decays = H if case["form"] == "head" else H * P * N
    if case["op"] == "prompt":
        lens = _lengths(case)
        pads = set(_padded(case, len(lens)))
        lens = [n for i, n in enumerate(lens) if i not in pads]
        tokens, states = sum(lens), 1.5 * len(lens)      # read for half of them, written for all
    else:
        live = case["batch"] - case["n_pad"]
        tokens, states = live * case["seqlen"], live * (1 + (case["seqlen"] if case["spec"] else 1))
    row = 2 * ((3 if case["gate"] else 2) * H * P + 2 * G * N) + (2 if case["raw"] else 4) * steps
    return {"bytes": tokens * row + 4 * states * H * P * N + 4 * decays, "flops": 6 * tokens * H * P * N}
