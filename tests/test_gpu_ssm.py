"""GPU parity of the selective state space scan (prefill and decode, both
forms) with the 64-bit recurrence, within the running bound of ssm_ref."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FILL = -3.0


def put(t):
    return None if t is None else t.to(DEV)


def call_fwd(g, st, qsl, ci, has, out=None):
    return S.ssm_fwd_varlen(g["x"], g["dt"], g["A"], g["B"], g["C"], st, put(qsl), put(ci), put(has), D=g["D"], z=g["z"],
                            dt_bias=g["dt_bias"], dt_softplus=g["dt_softplus"], dt_limit=g["dt_limit"], out=out)


def call_update(g, st, ci=None, acc=None, osi=None, out=None):
    return S.ssm_update(g["x"], g["dt"], g["A"], g["B"], g["C"], st, put(ci), put(acc), put(osi), D=g["D"], z=g["z"],
                        dt_bias=g["dt_bias"], dt_softplus=g["dt_softplus"], dt_limit=g["dt_limit"], out=out)


def lines_for(n, extra, seed, pads=()):
    order = torch.randperm(n + extra, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    for i in pads:
        order[i] = -1
    return order


def state_of(d, lines, lead, seed, scale=0.3):
    H, _, P, N = R.sizes(d["x"], d["A"], d["B"], lead)
    shape = (lines, H, P, N) if d["A"].dim() == 1 else (lines, H * P, N)
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale


def prefill(lens, form, heads, head_dim, groups, n, seed=0, pads=(), init=None, tail=0, edit=None, strided=None, **kw):
    """Runs prefill on the GPU and the reference; compares outputs, states and what must stay untouched."""
    total = sum(lens)
    d = R.draw((total + tail,), form, heads, head_dim, groups, n, seed, **kw)
    if edit:
        edit(d)
    state = state_of(d, len(lens) + 3, 1, seed + 1)
    qsl = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    ci = lines_for(len(lens), 3, seed + 2, pads)
    has = torch.rand(len(lens), generator=torch.Generator().manual_seed(seed + 3)) < 0.5 if init is None else torch.tensor(init)
    o, otol, s, stol, live = R.fwd(d, state, qsl, ci, has)
    g, st = R.on(d, DEV), state.to(DEV)
    out = torch.full(d["x"].shape, FILL, dtype=BF, device=DEV)
    if strided:
        g, st, out = strided(g, st, out)
    assert call_fwd(g, st, qsl, ci, has, out) is out
    torch.cuda.synchronize()
    got = out.cpu()
    R.check(got[live], o[live], otol[live], f"out {lens}")
    assert (got[~live] == FILL).all()
    R.check_state(st, s, stol)


FORMS = [("head", 2, 64, 1, 128), ("head", 4, 32, 2, 64), ("channel", 1, 96, 1, 16), ("channel", 2, 32, 2, 8)]


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 333])
@pytest.mark.parametrize("form", FORMS)
def test_prefill_lengths(n, form):
    prefill([n], *form, seed=n)


@pytest.mark.parametrize("p,n", [(64, 128), (64, 64), (128, 128), (32, 32), (96, 80), (80, 96), (100, 40), (8, 8), (1, 1), (5, 3),
                                 (64, 16), (64, 256), (130, 200), (16, 4), (65, 130), (64, 129), (256, 8)])
def test_prefill_head_sizes(p, n):
    prefill([70, 5, 130], "head", 4, p, 2, n, seed=p + n, pads=(1,), gate=p % 3 == 0)


@pytest.mark.parametrize("p,n", [(64, 16), (1, 16), (3, 1), (100, 16), (128, 32), (96, 5), (1000, 16), (257, 64), (64, 256), (33, 100)])
def test_prefill_channel_sizes(p, n):
    prefill([70, 5, 130], "channel", 2, p, 2, n, seed=p + n, pads=(1,), gate=p % 2 == 0)


@pytest.mark.parametrize("h,g", [(1, 1), (4, 1), (3, 3), (6, 2), (24, 8), (7, 1), (10, 2)])
def test_prefill_head_groups(h, g):
    prefill([67, 30], "head", h, 64, g, 64, seed=h)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kw", [dict(raw=False), dict(gate=True), dict(skip=False), dict(bias=False), dict(dt_limit=(0.01, 0.05)),
                                dict(slow=1e-3), dict(slow=50.0), dict(raw=False, gate=True, skip=False)])
def test_prefill_options(form, kw):
    prefill([150, 64], *form, seed=7, **kw)


@pytest.mark.parametrize("form", FORMS)
def test_prefill_ragged_batch_with_empty_and_padded_sequences(form):
    prefill([0, 1, 64, 0, 3, 129, 2, 63, 65, 1, 0, 7], *form, seed=3, pads=(2, 6), tail=9)


@pytest.mark.parametrize("form", [("head", 6, 64, 2, 128), ("head", 6, 40, 1, 100), ("channel", 1, 200, 1, 16)])
def test_prefill_many_sequences(form):
    lens = [1 + (37 * i) % 90 for i in range(44)]
    lens[7], lens[9], lens[30] = 0, 200, 64
    prefill(lens, *form, seed=5, pads=(3, 40))


@pytest.mark.parametrize("form", FORMS)
def test_prefill_steps_of_zero_and_of_all(form):
    """No step keeps the state and writes nothing; a huge one forgets everything; a decay above 0 counts as 0."""
    def edit(d):
        d["dt"][:20] = 0.0
        d["dt"][20:40:3] = 1e3
        d["dt"][50] = 1e6
        d["dt"][60:64] = -0.5
        d["dt"][100:] *= 1e-4
    prefill([140], *form, seed=11, raw=False, edit=edit)


@pytest.mark.parametrize("form", FORMS)
def test_prefill_magnitudes(form):
    def edit(d):
        d["x"][:70] *= 1e-6
        d["x"][70:90] *= 3e6
        d["B"][::3] *= 2.0 ** -40
        d["B"][1::3] *= 2.0 ** 30
        d["C"][5] = 0
        d["x"][100:110] = 0
    prefill([130, 40], *form, seed=13, edit=edit)


@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 2, 64, 2, 16)])
@pytest.mark.parametrize("which", ["pitched", "offset", "token_contiguous", "broadcast", "state_t", "heads_apart"])
def test_prefill_layouts(form, which):
    head = form[0] == "head"

    def strided(g, st, out):
        def pitched(t, extra, off):
            b = torch.full((*t.shape[:-1], t.shape[-1] + extra), 7.0, dtype=t.dtype, device=DEV)
            w = b[..., off:off + t.shape[-1]]
            w.copy_(t)
            return w
        names = ("x", "B", "C", "z", "dt")
        if which == "pitched":
            for n in names:
                g[n] = pitched(g[n], 8, 0)
            out = pitched(out, 16, 8)
        elif which == "offset":
            for n in names:
                g[n] = pitched(g[n], 3, 1)
            out = pitched(out, 5, 3)
        elif which == "token_contiguous":
            for n in names:
                g[n] = g[n].movedim(0, -1).contiguous().movedim(-1, 0)
            out = out.movedim(0, -1).contiguous().movedim(-1, 0)
        elif which == "state_t":
            st = st.transpose(-1, -2).contiguous().transpose(-1, -2)
        elif which == "heads_apart" and head:
            for n in ("x", "B", "C", "z"):
                g[n] = g[n].transpose(1, 2).contiguous().transpose(1, 2)
            out = out.transpose(0, 1).contiguous().transpose(0, 1)
        return g, st, out

    def edit(d):
        if which == "broadcast":                       # every group has the first one's B, every channel one D
            d["B"] = d["B"][:, :1].expand(-1, 2, -1)
            d["D"] = d["D"][:1].expand(d["D"].shape)
    prefill([100, 37], *form, seed=21, gate=True, strided=strided, edit=edit)


def test_prefill_skip_of_every_channel():
    """D (heads, head_dim)."""
    def edit(d):
        d["D"] = torch.randn(3, 64, generator=torch.Generator().manual_seed(1))
    prefill([100, 70], "head", 3, 64, 1, 64, seed=23, edit=edit, gate=True)


@pytest.mark.parametrize("form", FORMS)
def test_prefill_without_state(form):
    d = R.draw((90,), *form, 31)
    qsl = torch.tensor([0, 60, 90], dtype=torch.int32)
    ref = R.fwd(d, None, qsl, None, None)
    out = call_fwd(R.on(d, DEV), None, qsl, None, None)
    R.check(out, ref[0], ref[1], "out")


@pytest.mark.parametrize("form", FORMS)
def test_prefill_bad_lines_and_offsets_stay_inside(form):
    """Lines outside the cache skip their sequence; offsets outside the rows are clamped."""
    d = R.draw((80,), *form, 32)
    state = state_of(d, 3, 1, 1)
    ci = torch.tensor([7, 1, -5], dtype=torch.int32)
    has = torch.ones(3, dtype=torch.bool)
    st, out = state.to(DEV), torch.full(d["x"].shape, FILL, dtype=BF, device=DEV)
    call_fwd(R.on(d, DEV), st, torch.tensor([0, 20, 50, 500], dtype=torch.int32), ci, has, out)
    ref = R.fwd(d, state, [0, 20, 50, 80], ci, has)
    R.check(out.cpu()[20:50], ref[0][20:50], ref[1][20:50], "out")
    assert (out.cpu()[:20] == FILL).all() and (out.cpu()[50:] == FILL).all()
    R.check_state(st, ref[2], ref[3])


@pytest.mark.parametrize("form", [("head", 2, 64, 2, 64), ("channel", 2, 64, 2, 16)])
def test_prefill_nan_and_inf_stay_in_their_sequence_and_head(form):
    d = R.draw((192,), *form, 33)
    x = d["x"].view(192, 2, 64)
    x[70, 0] = float("nan")
    x[71, 0, 3] = float("inf")
    state = state_of(d, 3, 1, 1)
    qsl = torch.tensor([0, 64, 128, 192], dtype=torch.int32)
    has = torch.ones(3, dtype=torch.bool)
    st = state.to(DEV)
    out = call_fwd(R.on(d, DEV), st, qsl, None, has).cpu().view(192, 2, 64)
    ref = R.fwd(d, state, qsl, None, has)
    ok = torch.ones(192, 2, dtype=torch.bool)
    ok[64:128, 0] = False
    R.check(out[ok], ref[0].view(192, 2, 64)[ok], ref[1].view(192, 2, 64)[ok], "out")
    assert torch.isnan(out[72:128, 0]).all()
    n = form[4]
    st, want, tol = st.view(3, 2, 64, n), ref[2].view(3, 2, 64, n), ref[3].view(3, 2, 64, n)
    for line, head in ((0, 0), (0, 1), (1, 1), (2, 0), (2, 1)):
        R.check_state(st[line, head], want[line, head], tol[line, head])


@pytest.mark.parametrize("form", FORMS)
def test_prefill_is_deterministic_and_splits(form):
    """Twice the same bits; and 400 tokens at once are 90 and then 310 continued."""
    d = R.draw((400,), *form, 34)
    g = R.on(d, DEV)
    has = torch.ones(1, dtype=torch.bool)
    state = state_of(d, 1, 1, 1)

    def go(a, b, st):
        part = {k: v[a:b] if k in ("x", "dt", "B", "C") else v for k, v in g.items()}
        return call_fwd(part, st, torch.tensor([0, b - a], dtype=torch.int32), None, has)
    s1, s2, s3 = (state.to(DEV) for _ in range(3))
    o1, o2 = go(0, 400, s1), go(0, 400, s2)
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(s1, s2)
    o3 = torch.cat([go(0, 90, s3), go(90, 400, s3)])
    ref = R.fwd(d, state, [0, 400], None, [True])
    for o, s in ((o1, s1), (o3, s3)):
        R.check(o, ref[0], ref[1], "out")
        R.check_state(s, ref[2], ref[3])


# ----------------------------------------------------------------- decode --

def decode(n, steps, form, heads, head_dim, groups, N, seed=0, spec=None, pads=(), flat=False, strided=None, ci=None,
           accepted=None, osi=None, lines=None, **kw):
    d = R.draw((n, steps), form, heads, head_dim, groups, N, seed, **kw)
    lines = lines or n * (steps if spec else 1) + 3
    state = state_of(d, lines, 2, seed + 1)
    gen = torch.Generator().manual_seed(seed + 2)
    if ci is None:
        order = torch.randperm(lines, generator=gen).to(torch.int32)
        ci = order[:n * steps].view(n, steps).clone() if spec else order[:n].clone()
        for i in pads:
            ci[i] = -1
    if spec:
        accepted = torch.randint(1, steps + 1, (n,), generator=gen, dtype=torch.int32) if accepted is None else accepted
        osi = ci if osi is None else osi
    o, otol, s, stol, live = R.update(d, state, ci, accepted, osi)
    g, st = R.on(d, DEV), state.to(DEV)
    out = torch.full(d["x"].shape, FILL, dtype=BF, device=DEV)
    if strided:
        g, st, out = strided(g, st, out)
    oo = out
    if flat:
        g = {k: v[:, 0] if k in ("x", "dt", "B", "C", "z") and v is not None else v for k, v in g.items()}
        oo = out[:, 0]
    assert call_update(g, st, ci, accepted, osi, oo) is oo
    torch.cuda.synchronize()
    got = out.cpu()
    R.check(got[live], o[live], otol[live], "out")
    assert (got[~live] == FILL).all()
    R.check_state(st, s, stol)


@pytest.mark.parametrize("n", [1, 2, 7, 64])
@pytest.mark.parametrize("form", FORMS)
def test_decode_batches(n, form):
    decode(n, 1, *form, seed=n, pads=(1,) if n > 2 else (), flat=True, gate=n == 7)


def test_decode_large_batch():
    decode(70, 1, "head", 32, 64, 2, 32, seed=5)
    decode(20, 1, "channel", 1, 3000, 1, 16, seed=6)


@pytest.mark.parametrize("p,n", [(1, 1), (3, 9), (31, 33), (32, 7), (96, 80), (100, 40), (127, 17), (160, 24), (200, 16), (64, 256),
                                 (64, 128), (9, 160), (12, 66)])
@pytest.mark.parametrize("form", ["head", "channel"])
def test_decode_sizes(p, n, form):
    heads, groups = (4, 2) if form == "head" else (2, 2)
    decode(3, 2, form, heads, p, groups, n, seed=p, gate=n % 2 == 0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kw", [dict(raw=False), dict(gate=True), dict(skip=False), dict(bias=False), dict(dt_limit=(0.01, 0.05))])
def test_decode_options(form, kw):
    decode(5, 3, *form, seed=9, **kw)


@pytest.mark.parametrize("steps", [1, 2, 4, 5])
@pytest.mark.parametrize("form", FORMS)
def test_decode_speculative(steps, form):
    decode(6, steps, *form, seed=steps, spec=True, pads=(2,))


@pytest.mark.parametrize("form", FORMS)
def test_decode_speculative_skips_and_partial_lines(form):
    ci = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 99], [7, 8]], dtype=torch.int32)
    osi = torch.tensor([[0, -1], [2, 3], [5, 5], [6, 6], [9, 200]], dtype=torch.int32)   # the same line twice: the later step
    acc = torch.tensor([2, 0, 1, 2, 3], dtype=torch.int32)                               # 0, 3: outside; 99: no line
    decode(5, 2, *form, seed=40, spec=True, ci=ci, osi=osi, accepted=acc, lines=12)


@pytest.mark.parametrize("form", FORMS)
def test_decode_saves_without_accepted_counts(form):
    osi = torch.tensor([[3, 4], [5, -7]], dtype=torch.int32)
    decode(2, 2, *form, seed=41, ci=torch.tensor([0, 1], dtype=torch.int32), osi=osi, lines=6)


@pytest.mark.parametrize("form", [("head", 4, 24, 2, 64), ("channel", 2, 24, 2, 16)])
@pytest.mark.parametrize("which", ["pitched", "offset", "state_t", "state_pitched"])
def test_decode_layouts(form, which):
    def strided(g, st, out):
        if which in ("pitched", "offset"):
            off, extra = (0, 8) if which == "pitched" else (1, 3)

            def wide(t, fill):
                return torch.full((*t.shape[:-1], t.shape[-1] + extra), fill, dtype=t.dtype, device=DEV)[..., off:off + t.shape[-1]]
            for n in ("x", "B", "C", "z", "dt"):
                g[n] = wide(g[n], 7.0).copy_(g[n])
            out = wide(out, FILL)
        elif which == "state_t":
            st = st.transpose(-1, -2).contiguous().transpose(-1, -2)
        else:
            st = torch.full((*st.shape[:-1], st.shape[-1] + 1), 7.0, device=DEV)[..., 1:].copy_(st)
        return g, st, out
    decode(4, 2, *form, seed=50, strided=strided, gate=True)


# ------------------------------------------------------- graphs, streams --

@pytest.mark.parametrize("op", ["prefill", "decode"])
@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 1, 512, 1, 16)])
def test_graph_replays_match_eager(op, form):
    n, steps = 3, 240
    d = R.on(R.draw((n * steps,) if op == "prefill" else (n, 5), *form, 60), DEV)
    state = state_of(d, n, 1 if op == "prefill" else 2, 1).to(DEV)
    qsl = torch.tensor([0, 240, 241, 720], dtype=torch.int32, device=DEV)
    has = torch.ones(n, dtype=torch.bool, device=DEV)

    def call(st, out):
        if op == "prefill":
            call_fwd(d, st, qsl, None, has, out)
        else:
            call_update(d, st, out=out)
    st, out = state.clone(), torch.zeros_like(d["x"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(st, out)                                  # a stream of its own, before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(st, out)
    st.copy_(state)
    want, wout = state.clone(), torch.zeros_like(out)
    for i in range(4):
        d["x"].mul_(0.9)                               # new inputs between the replays
        graph.replay()
        call(want, wout)
        torch.cuda.synchronize()
        assert torch.equal(st, want) and torch.equal(out, wout), i


@pytest.mark.parametrize("nseq,T", [(1, 1500), (60, 40)])
@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 1, 512, 1, 16)])
def test_two_streams_at_once(nseq, T, form):
    """Calls in flight together give what they give alone."""
    qsl = torch.arange(nseq + 1, dtype=torch.int32, device=DEV) * T
    has = torch.ones(nseq, dtype=torch.bool, device=DEV)
    cases = []
    for seed in (80, 81):
        d = R.draw((nseq * T,), *form, seed)
        cases.append((R.on(d, DEV), state_of(d, nseq, 1, seed).to(DEV)))
    alone = []
    for d, st in cases:
        s = st.clone()
        alone.append((call_fwd(d, s, qsl, None, has), s))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = [None, None]
        states = [st.clone() for _, st in cases]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = call_fwd(cases[i][0], states[i], qsl, None, has)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], alone[i][0]) and torch.equal(states[i], alone[i][1])


def test_state_offsets_past_32_bits():
    """A cache of more than 2^31 elements; only its last line is touched."""
    H, P, N = 128, 64, 128
    lines = (1 << 31) // (H * P * N) + 3
    st = torch.zeros(lines, H, P, N, device=DEV)
    d = R.draw((1, 1), "head", H, P, 8, N, 70)
    s0 = state_of(d, 1, 2, 1)
    st[-1] = s0[0].to(DEV)
    g = R.on(d, DEV)
    ci = torch.tensor([lines - 1], dtype=torch.int32)
    out = call_update(g, st, ci)
    ref = R.update(d, s0, None, None, None)
    R.check(out, ref[0], ref[1], "out")
    R.check_state(st[-1:], ref[2], ref[3])
    one = {k: v[0] if k in ("x", "dt", "B", "C") else v for k, v in d.items()}
    out = call_fwd(R.on(one, DEV), st, torch.tensor([0, 1], dtype=torch.int32), ci, torch.zeros(1, dtype=torch.bool))
    ref = R.fwd(one, s0, [0, 1], None, None)
    R.check(out, ref[0], ref[1], "out")
    R.check_state(st[-1:], ref[2], ref[3])
    assert not st[:-1].any()
