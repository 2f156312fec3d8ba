"""GPU parity of the gated delta rule (prefill and decode) with the 64-bit
recurrence, within the running bound of gdr_ref."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import gdr_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FILL = -3.0


def lines_for(n, extra, seed, pads=()):
    order = torch.randperm(n + extra, generator=torch.Generator().manual_seed(seed))[:n].to(torch.int32)
    for i in pads:
        order[i] = -1
    return order


def prefill(lens, hk, hv, dk, dv, seed=0, raw=True, l2norm=True, pads=(), init=None, decay=1.0, scale=None, tail=0,
            edit=None, strided=None, state_scale=0.3):
    """Runs prefill on the GPU and the reference; compares outputs, states and what must stay untouched."""
    n, total = len(lens), sum(lens)
    d = R.draw_inputs((total + tail,), hk, hv, dk, dv, seed, raw=raw, normed=not l2norm, decay=decay)
    if edit:
        edit(d)
    gen = torch.Generator().manual_seed(seed + 1)
    state = torch.randn(n + 3, hv, dv, dk, generator=gen) * state_scale
    qsl = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    ci = lines_for(n, 3, seed + 2, pads)
    has = (torch.rand(n, generator=gen) < 0.5) if init is None else torch.tensor(init)
    sc = dk ** -0.5 if scale is None else scale
    ref = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, qsl, ci, has, d["A_log"], d["dt_bias"], sc, l2norm,
                R.C_CHUNK, R.F_CHUNK)
    g = R.on(d, DEV)
    st = state.to(DEV)
    out = torch.full((total + tail, hv, dv), FILL, dtype=BF, device=DEV)
    if strided:
        g, st, out = strided(g, st, out)
    S.gdr_fwd_varlen(g["q"], g["k"], g["v"], g["g"], g["beta"], st, qsl.to(DEV), ci.to(DEV), has.to(DEV), A_log=g["A_log"],
                     dt_bias=g["dt_bias"], scale=sc, use_qk_l2norm=l2norm, out=out)
    torch.cuda.synchronize()
    o, otol, s, stol, live = ref
    got = out.cpu()
    R.check(got[live], o[live], otol[live], f"out {lens} {hk, hv, dk, dv}")
    assert (got[~live] == FILL).all()
    R.check_state(st, s, stol)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [63], [64], [65], [127], [128], [129], [200], [333]])
def test_prefill_lengths(lens):
    prefill(lens, 1, 2, 128, 128, seed=lens[0])


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64), (64, 128), (32, 32), (96, 80), (100, 40), (8, 8), (1, 1), (5, 3),
                                   (127, 129), (72, 16), (128, 17), (130, 20), (256, 32), (192, 48), (33, 200)])
def test_prefill_head_sizes(dk, dv):
    prefill([70, 5, 130], 2, 4, dk, dv, seed=dk + dv, pads=(1,))


@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 4), (3, 3), (2, 6), (16, 32)])
def test_prefill_head_groups(hk, hv):
    prefill([67, 30], hk, hv, 64, 64, seed=hk)


@pytest.mark.parametrize("raw,l2norm,decay", [(True, True, 1.0), (False, True, 1.0), (False, False, 0.1), (True, False, 1.0),
                                              (False, True, 20.0)])
def test_prefill_gates_and_norms(raw, l2norm, decay):
    prefill([150, 64], 2, 2, 128, 64, seed=7, raw=raw, l2norm=l2norm, decay=decay, scale=0.7)


def test_prefill_ragged_batch_with_empty_and_padded_sequences():
    prefill([0, 1, 64, 0, 3, 129, 2, 63, 65, 1, 0, 7], 2, 4, 64, 64, seed=3, pads=(2, 6), tail=9)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (96, 80), (128, 200), (8, 16), (36, 24)])
def test_prefill_many_heads(dk, dv):
    """Batches whose heads fill the chip by themselves: one kernel (two for 36 channels, which have no vector loads)."""
    lens = [1 + (37 * i) % 90 for i in range(44)]
    lens[7], lens[9], lens[30] = 0, 200, 64
    prefill(lens, 2, 6, dk, dv, seed=dk + dv, pads=(3, 40))


def test_prefill_without_workspace(monkeypatch):
    """The C entry with no workspace: one kernel for layouts with vector loads, a token at a time for others."""
    real = S._launch_packed
    monkeypatch.setattr(S, "_launch_packed", lambda fn, dev, args: real(fn, dev, (*args[:-2], 0, 0)))
    prefill([70, 5, 130], 2, 4, 128, 128, seed=1)
    prefill([70, 5, 130], 2, 4, 64, 100, seed=2)
    prefill([70, 5, 130], 2, 4, 36, 24, seed=3)


def test_prefill_no_decay_and_full_decay():
    def edit(d):
        d["g"][:20] = 0.0                              # nothing is forgotten
        d["g"][20:40:3] = float("-inf")                # everything is
        d["g"][50] = -1e30
        d["g"][60:70] = 5.0                            # above 0 counts as 0
        d["beta"][70:80] = 0.0                         # nothing is written
        d["beta"][90:100] = 1.0
    prefill([140], 2, 2, 64, 64, seed=11, raw=False, edit=edit)


def test_prefill_zero_keys_and_repeated_keys():
    def edit(d):
        d["k"][3:9] = 0
        d["q"][5] = 0
        d["k"][64:] = d["k"][10]                       # one key over and over: A is full
    prefill([150], 1, 2, 128, 64, seed=12, edit=edit)


def test_prefill_value_magnitudes():
    def edit(d):
        d["v"][:70] *= 1e-4
        d["v"][70:90] *= 3e4
        d["k"][::3] *= 2.0 ** -20                      # l2norm's eps decides what is left of these
        d["k"][1::3] *= 2.0 ** 12
    prefill([130, 40], 2, 2, 64, 64, seed=13, edit=edit)


@pytest.mark.parametrize("which", ["pitched", "offset", "transposed", "token_contiguous", "broadcast", "state_t"])
def test_prefill_layouts(which):
    def strided(g, st, out):
        def pitched(t, extra, off):
            b = torch.full((t.shape[0], t.shape[1], t.shape[2] + extra), 7.0, dtype=t.dtype, device=DEV)
            w = b[:, :, off:off + t.shape[2]]
            w.copy_(t)
            return w
        if which == "pitched":
            for x in "qkv":
                g[x] = pitched(g[x], 8, 0)
            out = pitched(out, 16, 8)
        elif which == "offset":
            for x in "qkv":
                g[x] = pitched(g[x], 3, 1)
            out = pitched(out, 5, 3)
        elif which == "transposed":
            for x in "qkv":
                g[x] = g[x].transpose(1, 2).contiguous().transpose(1, 2)
            g["g"] = g["g"].t().contiguous().t()
            g["beta"] = g["beta"].t().contiguous().t()
        elif which == "token_contiguous":
            for x in "qkv":
                g[x] = g[x].permute(1, 2, 0).contiguous().permute(2, 0, 1)
            out = out.permute(1, 2, 0).contiguous().permute(2, 0, 1)
        elif which == "broadcast":
            assert g["k"].shape[1] == 2
        elif which == "state_t":
            st = st.transpose(2, 3).contiguous().transpose(2, 3)
        return g, st, out

    def edit(d):
        if which == "broadcast":                       # every head has the first one's key
            d["k"] = d["k"][:, :1].expand(-1, 2, -1)
    prefill([100, 37], 2, 4, 64, 64, seed=21, strided=strided, edit=edit)


def test_prefill_without_state_and_default_scale():
    d = R.draw_inputs((90,), 2, 4, 64, 64, 31)
    qsl = torch.tensor([0, 60, 90], dtype=torch.int32)
    ref = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], None, qsl, None, None, d["A_log"], d["dt_bias"], 0.125, True,
                R.C_CHUNK, R.F_CHUNK)
    g = R.on(d, DEV)
    out = S.gdr_fwd_varlen(g["q"], g["k"], g["v"], g["g"], g["beta"], None, qsl.to(DEV), A_log=g["A_log"],
                           dt_bias=g["dt_bias"], use_qk_l2norm=True)
    R.check(out, ref[0], ref[1], "out")


def test_prefill_bad_lines_and_offsets_stay_inside():
    """Lines outside the cache skip their sequence; offsets outside the rows are clamped."""
    d = R.draw_inputs((80,), 1, 2, 64, 64, 32)
    g = R.on(d, DEV)
    state = torch.randn(3, 2, 64, 64) * 0.3
    qsl = torch.tensor([0, 20, 50, 500], dtype=torch.int32)
    ci = torch.tensor([7, 1, -5], dtype=torch.int32)
    has = torch.ones(3, dtype=torch.bool)
    st, out = state.to(DEV), torch.full((80, 2, 64), FILL, dtype=BF, device=DEV)
    S.gdr_fwd_varlen(g["q"], g["k"], g["v"], g["g"], g["beta"], st, qsl.to(DEV), ci.to(DEV), has.to(DEV), A_log=g["A_log"],
                     dt_bias=g["dt_bias"], scale=1.0, use_qk_l2norm=True, out=out)
    ref = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, [0, 20, 50, 80], ci, has, d["A_log"], d["dt_bias"], 1.0,
                True, R.C_CHUNK, R.F_CHUNK)
    R.check(out.cpu()[20:50], ref[0][20:50], ref[1][20:50], "out")
    assert (out.cpu()[:20] == FILL).all() and (out.cpu()[50:] == FILL).all()
    R.check_state(st, ref[2], ref[3])


def test_prefill_nan_and_inf_stay_in_their_sequence_and_head():
    d = R.draw_inputs((192,), 2, 2, 64, 64, 33)
    d["v"][70, 0] = float("nan")
    d["k"][71, 0, 3] = float("inf")
    state = torch.randn(3, 2, 64, 64) * 0.3
    qsl = torch.tensor([0, 64, 128, 192], dtype=torch.int32)
    has = torch.ones(3, dtype=torch.bool)
    g = R.on(d, DEV)
    st = state.to(DEV)
    out = S.gdr_fwd_varlen(g["q"], g["k"], g["v"], g["g"], g["beta"], st, qsl.to(DEV), None, has.to(DEV),
                           A_log=g["A_log"], dt_bias=g["dt_bias"], scale=1.0, use_qk_l2norm=True)
    ref = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, qsl, None, has, d["A_log"], d["dt_bias"], 1.0, True,
                R.C_CHUNK, R.F_CHUNK)
    ok = torch.ones(192, 2, dtype=torch.bool)
    ok[64:128, 0] = False
    R.check(out.cpu()[ok], ref[0][ok], ref[1][ok], "out")
    assert torch.isnan(out.cpu()[72:128, 0]).all()
    for line, head in ((0, 0), (0, 1), (1, 1), (2, 0), (2, 1)):
        R.check_state(st[line, head], ref[2][line, head], ref[3][line, head])


def test_prefill_is_deterministic_and_splits():
    """Twice the same bits; and 200 tokens at once are 90 and then 110 continued."""
    d = R.draw_inputs((200,), 2, 4, 128, 128, 34)
    g = R.on(d, DEV)
    has = torch.ones(1, dtype=torch.bool, device=DEV)
    state = (torch.randn(1, 4, 128, 128) * 0.3)

    def go(a, b, st):
        return S.gdr_fwd_varlen(g["q"][a:b], g["k"][a:b], g["v"][a:b], g["g"][a:b], g["beta"][a:b], st,
                                torch.tensor([0, b - a], dtype=torch.int32, device=DEV), None, has, A_log=g["A_log"],
                                dt_bias=g["dt_bias"], use_qk_l2norm=True)
    s1, s2, s3 = (state.to(DEV) for _ in range(3))
    o1, o2 = go(0, 200, s1), go(0, 200, s2)
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(s1, s2)
    o3 = torch.cat([go(0, 90, s3), go(90, 200, s3)])
    ref = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, [0, 200], None, [True], d["A_log"], d["dt_bias"],
                128 ** -0.5, True, R.C_CHUNK, R.F_CHUNK)
    for o, s in ((o1, s1), (o3, s3)):
        R.check(o, ref[0], ref[1], "out")
        R.check_state(s, ref[2], ref[3])


# ----------------------------------------------------------------- decode --

def decode(n, steps, hk, hv, dk, dv, seed=0, raw=True, l2norm=True, spec=None, pads=(), three_d=False, strided=None,
           ci=None, accepted=None, osi=None, lines=None):
    d = R.draw_inputs((n, steps), hk, hv, dk, dv, seed, raw=raw, normed=not l2norm)
    gen = torch.Generator().manual_seed(seed + 1)
    lines = lines or n * (steps if spec else 1) + 3
    state = torch.randn(lines, hv, dv, dk, generator=gen) * 0.3
    if ci is None:
        order = torch.randperm(lines, generator=gen).to(torch.int32)
        ci = order[:n * steps].view(n, steps).clone() if spec else order[:n].clone()
        for i in pads:
            ci[i] = -1
    if spec:
        accepted = torch.randint(1, steps + 1, (n,), generator=gen, dtype=torch.int32) if accepted is None else accepted
        osi = ci if osi is None else osi
    o, otol, s, stol, live = R.update(d["q"], d["k"], d["v"], d["g"], d["beta"], state, ci, accepted, osi, d["A_log"],
                                      d["dt_bias"], 0.2, l2norm)
    g = R.on(d, DEV)
    st = state.to(DEV)
    out = torch.full((n, steps, hv, dv), FILL, dtype=BF, device=DEV)
    if strided:
        g, st, out = strided(g, st, out)
    a = {x: g[x] for x in ("q", "k", "v", "g", "beta")}
    oo = out
    if three_d:
        a = {x: t[:, 0] for x, t in a.items()}
        oo = out[:, 0]
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    r = S.gdr_update(**a, state=st, cache_indices=put(ci), num_accepted_tokens=put(accepted),
                     output_state_indices=put(osi), A_log=g["A_log"], dt_bias=g["dt_bias"], scale=0.2,
                     use_qk_l2norm=l2norm, out=oo)
    assert r is oo
    torch.cuda.synchronize()
    got = out.cpu()
    R.check(got[live], o[live], otol[live], "out")
    assert (got[~live] == FILL).all()
    R.check_state(st, s, stol)


@pytest.mark.parametrize("n", [1, 2, 7, 64])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64)])
def test_decode_batches(n, dk, dv):
    decode(n, 1, 2, 4, dk, dv, seed=n, pads=(1,) if n > 2 else (), three_d=True)


def test_decode_large_batch_of_many_heads():
    decode(40, 1, 16, 32, 32, 64, seed=5)


@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 9), (31, 33), (32, 7), (96, 80), (100, 40), (127, 17), (160, 24), (200, 16),
                                   (256, 256)])
def test_decode_head_sizes(dk, dv):
    decode(3, 2, 2, 4, dk, dv, seed=dk)


@pytest.mark.parametrize("raw,l2norm", [(False, True), (False, False), (True, False)])
def test_decode_gates_and_norms(raw, l2norm):
    decode(5, 3, 2, 4, 64, 32, seed=9, raw=raw, l2norm=l2norm)


@pytest.mark.parametrize("steps", [1, 2, 4, 5])
def test_decode_speculative(steps):
    decode(6, steps, 2, 4, 64, 64, seed=steps, spec=True, pads=(2,))


def test_decode_speculative_skips_and_partial_lines():
    ci = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 99], [7, 8]], dtype=torch.int32)
    osi = torch.tensor([[0, -1], [2, 3], [5, 5], [6, 6], [9, 200]], dtype=torch.int32)   # the same line twice: the later step
    acc = torch.tensor([2, 0, 1, 2, 3], dtype=torch.int32)                               # 0, 3: outside; 99: no line
    decode(5, 2, 1, 2, 32, 32, seed=40, spec=True, ci=ci, osi=osi, accepted=acc, lines=12)


def test_decode_saves_without_accepted_counts():
    osi = torch.tensor([[3, 4], [5, -7]], dtype=torch.int32)
    decode(2, 2, 1, 2, 64, 64, seed=41, ci=torch.tensor([0, 1], dtype=torch.int32), osi=osi, lines=6)


@pytest.mark.parametrize("which", ["pitched", "offset", "state_t", "state_pitched"])
def test_decode_layouts(which):
    def strided(g, st, out):
        if which in ("pitched", "offset"):
            off, extra = (0, 8) if which == "pitched" else (1, 3)
            for x in "qkv":
                b = torch.full((*g[x].shape[:3], g[x].shape[3] + extra), 7.0, dtype=BF, device=DEV)
                w = b[..., off:off + g[x].shape[3]]
                w.copy_(g[x])
                g[x] = w
            out = torch.full((*out.shape[:3], out.shape[3] + extra), FILL, dtype=BF, device=DEV)[..., off:off + out.shape[3]]
        elif which == "state_t":
            st = st.transpose(2, 3).contiguous().transpose(2, 3)
        else:
            b = torch.full((*st.shape[:3], st.shape[3] + 1), 7.0, device=DEV)
            w = b[..., 1:]
            w.copy_(st)
            st = w
        return g, st, out
    decode(4, 2, 2, 4, 64, 24, seed=50, strided=strided)


# ------------------------------------------------------- graphs, streams --

@pytest.mark.parametrize("op", ["prefill", "decode"])
def test_graph_replays_match_eager(op):
    n, steps, hk, hv, dk, dv = 3, 40, 2, 4, 64, 64
    d = R.on(R.draw_inputs((n * steps,) if op == "prefill" else (n, steps), hk, hv, dk, dv, 60), DEV)
    state = torch.randn(n, hv, dv, dk, device=DEV) * 0.3
    qsl = torch.tensor([0, 40, 41, 120], dtype=torch.int32, device=DEV)
    has = torch.ones(n, dtype=torch.bool, device=DEV)

    def call(st, out):
        kw = dict(A_log=d["A_log"], dt_bias=d["dt_bias"], use_qk_l2norm=True, out=out)
        if op == "prefill":
            S.gdr_fwd_varlen(d["q"], d["k"], d["v"], d["g"], d["beta"], st, qsl, None, has, **kw)
        else:
            S.gdr_update(d["q"], d["k"], d["v"], d["g"], d["beta"], st, **kw)
    st, out = state.clone(), torch.zeros_like(d["v"])
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
        d["v"].mul_(0.9)                               # new inputs between the replays
        graph.replay()
        call(want, wout)
        torch.cuda.synchronize()
        assert torch.equal(st, want) and torch.equal(out, wout), i


@pytest.mark.parametrize("nseq,T", [(1, 300), (60, 40)])
def test_two_streams_at_once(nseq, T):
    """Calls in flight together, each with its own workspace (one sequence) or none (many heads), give what they give alone."""
    qsl = torch.arange(nseq + 1, dtype=torch.int32, device=DEV) * T
    cases = []
    for seed in (80, 81):
        d = R.on(R.draw_inputs((nseq * T,), 2, 4, 64, 64, seed), DEV)
        cases.append((d, torch.randn(nseq, 4, 64, 64, device=DEV) * 0.3))
    has = torch.ones(nseq, dtype=torch.bool, device=DEV)

    def call(d, st):
        return S.gdr_fwd_varlen(d["q"], d["k"], d["v"], d["g"], d["beta"], st, qsl, None, has, A_log=d["A_log"],
                                dt_bias=d["dt_bias"], use_qk_l2norm=True)
    alone = []
    for d, st in cases:
        s = st.clone()
        alone.append((call(d, s), s))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = [None, None]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        states = [st.clone() for _, st in cases]
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = call(cases[i][0], states[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(got[i], alone[i][0]) and torch.equal(states[i], alone[i][1])


def test_prefill_short_sequences_by_elements():
    """Odd sizes and short sequences: a token at a time, without a workspace."""
    prefill([1 + i % 7 for i in range(40)], 1, 2, 36, 20, seed=90, pads=(5,))


def test_one_kernel_and_two_agree():
    """The same sequences alone (two kernels) and among many (one kernel)."""
    d = R.on(R.draw_inputs((40 * 200,), 2, 8, 64, 64, 91), DEV)
    st = torch.randn(40, 8, 64, 64, device=DEV) * 0.3
    many, few = st.clone(), st[:1].clone()
    kw = dict(A_log=d["A_log"], dt_bias=d["dt_bias"], use_qk_l2norm=True)
    has = torch.ones(40, dtype=torch.bool, device=DEV)
    a = S.gdr_fwd_varlen(d["q"], d["k"], d["v"], d["g"], d["beta"], many,
                         torch.arange(41, dtype=torch.int32, device=DEV) * 200, None, has, **kw)
    b = S.gdr_fwd_varlen(*(d[x][:200] for x in ("q", "k", "v", "g", "beta")), few,
                         torch.tensor([0, 200], dtype=torch.int32, device=DEV), None, has[:1], **kw)
    # the same products in the same order: the state to fp32's last bits, the output to a bf16 step
    assert ((a[:200].float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-6).all()
    assert ((many[0] - few[0]).abs() <= 2.0 ** -20 * few[0].abs().amax(-1, keepdim=True)).all()


def test_state_offsets_past_32_bits():
    """A cache of more than 2^31 elements; only its last line is touched."""
    hv, dv, dk = 32, 128, 128
    lines = (1 << 31) // (hv * dv * dk) + 3
    st = torch.zeros(lines, hv, dv, dk, device=DEV)
    d = R.draw_inputs((1, 1), 2, hv, dk, dv, 70)
    s0 = torch.randn(1, hv, dv, dk) * 0.3
    st[-1] = s0[0].to(DEV)
    g = R.on(d, DEV)
    ci = torch.tensor([lines - 1], dtype=torch.int32, device=DEV)
    out = S.gdr_update(g["q"], g["k"], g["v"], g["g"], g["beta"], st, ci, A_log=g["A_log"], dt_bias=g["dt_bias"], scale=0.2,
                       use_qk_l2norm=True)
    ref = R.update(d["q"], d["k"], d["v"], d["g"], d["beta"], s0, None, None, None, d["A_log"], d["dt_bias"], 0.2, True)
    R.check(out, ref[0], ref[1], "out")
    R.check_state(st[-1:], ref[2], ref[3])
    out = S.gdr_fwd_varlen(g["q"][0], g["k"][0], g["v"][0], g["g"][0], g["beta"][0], st,
                           torch.tensor([0, 1], dtype=torch.int32, device=DEV), ci, torch.zeros(1, dtype=torch.bool, device=DEV),
                           A_log=g["A_log"], dt_bias=g["dt_bias"], scale=0.2, use_qk_l2norm=True)
    ref = R.fwd(d["q"][0], d["k"][0], d["v"][0], d["g"][0], d["beta"][0], s0, [0, 1], None, None, d["A_log"], d["dt_bias"],
                0.2, True, R.C_CHUNK, R.F_CHUNK)
    R.check(out, ref[0], ref[1], "out")
    R.check_state(st[-1:], ref[2], ref[3])
    assert not st[:-1].any()


def test_decode_without_a_token_dimension():
    """(batch, heads, head_dim) inputs, sliced and transposed too, as (batch, 1, heads, head_dim) ones."""
    d = R.on(R.draw_inputs((6, 1), 2, 4, 64, 48, 95), DEV)
    kw = dict(A_log=d["A_log"], dt_bias=d["dt_bias"], use_qk_l2norm=True)
    st = torch.randn(6, 4, 48, 64, device=DEV)
    want_st = st.clone()
    want = S.gdr_update(d["q"], d["k"], d["v"], d["g"], d["beta"], want_st, **kw)
    flat = [d[x][:, 0] for x in ("q", "k", "v", "g", "beta")]
    odd = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in flat]
    for ins in (flat, odd):
        got_st = st.clone()
        got = S.gdr_update(*ins, got_st, **kw)
        assert got.shape == (6, 4, 48) and torch.equal(got, want[:, 0]) and torch.equal(got_st, want_st)
    with pytest.raises(ValueError):
        S.gdr_update(flat[0], flat[1], d["v"], flat[3], flat[4], st, **kw)
    with pytest.raises(ValueError):
        S.gdr_update(flat[0], flat[1], flat[2], d["g"], flat[4], st, **kw)


@pytest.mark.parametrize("hk,hv,lens", [(1, 8, [130]), (1, 6, [4100]), (2, 12, [700, 500]), (1, 3, [12000]), (1, 7, [90])])
def test_prefill_head_groups_prepared_together(hk, hv, lens):
    """Few and many chunks of groups of 2, 3, 6, 7 and 8 value heads."""
    prefill(lens, hk, hv, 64, 16, seed=hv)
