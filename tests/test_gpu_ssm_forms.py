"""Which kernel takes a call of the selective state space scan must not show:
segments, few heads, many, without a workspace, short sequences, against the
64-bit recurrence; and a layer's run of convolution, scan, norm and drafts."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R
from tests.test_gpu_ssm import BF, DEV, call_fwd, call_update, prefill, put, state_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[1300], [700, 1, 0, 900], [640], [3000]])
@pytest.mark.parametrize("form", [("head", 2, 64, 1, 32), ("head", 1, 32, 1, 64), ("head", 3, 8, 1, 128), ("channel", 1, 70, 1, 16),
                                  ("channel", 2, 8, 2, 20)])
def test_segments(lens, form):
    prefill(lens, *form, seed=lens[0], gate=form[1] == 3, slow=0.05)


@pytest.mark.parametrize("form", [("head", 2, 64, 1, 32), ("channel", 1, 70, 1, 16)])
def test_segments_of_a_decay_that_leaves_nothing(form):
    """A segment forgets all of what was before, or nothing."""
    def edit(d):
        d["dt"][200:400] = 30.0
        d["dt"][500:1100] = 0.0
    prefill([1300], *form, seed=1, raw=False, edit=edit, init=[True])


def test_segments_of_growing_decays():
    """Decays of both signs, and steps of both: what would grow stays."""
    def edit(d):
        d["A"][:, ::3] *= -1
        d["dt"][::5] *= -1
    prefill([900], "channel", 1, 70, 1, 16, seed=2, raw=False, edit=edit, init=[True])


@pytest.mark.parametrize("form", [("head", 2, 64, 1, 32), ("channel", 1, 70, 1, 16)])
def test_without_workspace(form, monkeypatch):
    real = S._launch_packed
    monkeypatch.setattr(S, "_launch_packed", lambda fn, dev, args: real(fn, dev, (*args[:-2], 0, 0)))
    prefill([1300, 5], *form, seed=3)


def test_short_of_memory_takes_no_workspace(monkeypatch):
    real = torch.empty_strided

    def empty(shape, *a, **kw):
        if kw.get("dtype") is torch.uint8:
            raise torch.OutOfMemoryError("none left")
        return real(shape, *a, **kw)
    monkeypatch.setattr(torch, "empty_strided", empty)
    prefill([1300], "head", 2, 64, 1, 32, seed=4)


@pytest.mark.parametrize("heads,head_dim,nseq", [(1, 64, 1), (3, 64, 30), (5, 64, 60), (4, 96, 20), (40, 64, 20), (9, 32, 50),
                                                 (12, 130, 9)])
def test_workgroups_of_two_four_and_eight_waves(heads, head_dim, nseq):
    prefill([7 + (i * 29) % 90 for i in range(nseq)], "head", heads, head_dim, 1, 64, seed=heads, pads=(0,) if nseq > 1 else ())


@pytest.mark.parametrize("mean", [3, 5, 6, 8, 9])
@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 1, 100, 1, 16)])
def test_short_sequences(mean, form):
    prefill([mean - 2, mean + 2, mean, mean], *form, seed=mean)


@pytest.mark.parametrize("kw", [dict(raw=False), dict(gate=True)])
def test_many_short_sequences_past_what_is_ranked(kw):
    prefill([6 + i % 9 for i in range(300)], "head", 2, 16, 1, 16, seed=5, **kw)


def test_step_sizes_that_underflow_and_saturate():
    """softplus from e^-90 to the identity."""
    def edit(d):
        d["dt"][:] = torch.linspace(-90, 90, d["dt"].shape[0])[:, None].bfloat16()
        d["dt_bias"] = torch.zeros_like(d["dt_bias"])
    for form in (("head", 2, 64, 1, 32), ("channel", 1, 70, 1, 16)):
        prefill([180], *form, seed=6, edit=edit, slow=1e-3)


@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 2, 64, 2, 16)])
def test_layer(form):
    """A prompt, then speculative steps: the convolution's output as x, B and C, the scan, the gated norm; the state and the
    windows of the accepted step go on.  Against the same kernels fed the whole sequence at once, and the recurrence."""
    head = form[0] == "head"
    H, P, G, N = form[1:]
    dim, cd, T, K, steps = H * P, H * P + 2 * G * N, 70, 3, 4
    g = torch.Generator().manual_seed(9)
    total = T + K * steps
    xbc = torch.randn(total, cd, generator=g).bfloat16()
    w = (torch.randn(cd, 4, generator=g) * 0.4).bfloat16().to(DEV)
    d = R.draw((total,), *form, 10, gate=True)
    nw = (1 + 0.1 * torch.randn(dim, generator=g)).bfloat16().to(DEV)
    dd = R.on(d, DEV)

    def parts(y, lead, lo, hi):
        x, B, C = y[..., :dim], y[..., dim:dim + G * N], y[..., dim + G * N:]
        q = dict(dd)
        q.update(x=x.unflatten(-1, (H, P)) if head else x, B=B.unflatten(-1, (G, N)), C=C.unflatten(-1, (G, N)),
                 dt=dd["dt"][lo:hi].view(*lead, *dd["dt"].shape[1:]), z=None)
        return q

    def norm(y, lo, hi):
        z = dd["z"][lo:hi].reshape(hi - lo, dim)
        return S.sconv_group_norm(y.reshape(hi - lo, dim), dim // 2, weight=nw, z=z, activation="silu", gate_first=True)

    def prompt(n):
        cs = torch.zeros(8, cd, 3, dtype=BF, device=DEV)
        st = torch.zeros((8, H, P, N) if head else (8, dim, N), device=DEV)
        qsl = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        line = torch.tensor([5], dtype=torch.int32, device=DEV)
        xin = xbc[:n].to(DEV)
        y = S.conv1d_fwd_varlen(xin.t(), w, None, cs, qsl, cache_indices=line,
                                has_initial_state=torch.zeros(1, dtype=torch.bool, device=DEV)).t()
        q = parts(y, (n,), 0, n)
        o = call_fwd(q, st, qsl, line, None)
        return y, norm(o, 0, n), cs, st, q, o
    y_all, want, _, st_all, q_all, o_all = prompt(total)
    ref = R.fwd({k: (v.cpu() if isinstance(v, torch.Tensor) else v) for k, v in q_all.items()}, st_all.cpu() * 0, [0, total],
                torch.tensor([5]), None)
    R.check(o_all, ref[0], ref[1], "out")
    R.check_state(st_all, ref[2], ref[3])
    _, got, cs, st, _, _ = prompt(T)
    outs, pos = [got], T
    ci = torch.tensor([[0, 1, 2, 3]], dtype=torch.int32, device=DEV)
    st[0], cs[0] = st[5], cs[5]
    acc = torch.tensor([1], dtype=torch.int32, device=DEV)
    for k in range(K):
        xin = xbc[pos:pos + steps].to(DEV).t().unsqueeze(0).contiguous()
        hist = cs[ci[0, acc.item() - 1]].unsqueeze(0).clone()      # the window of the accepted step
        new = torch.zeros(1, steps, cd, 3, dtype=BF, device=DEV)
        y = S.conv1d_update(xin, hist, w, activation="silu", intermediate=new)
        q = parts(y.transpose(1, 2), (1, steps), pos, pos + steps)
        o = call_update(q, st, ci, acc, ci)
        outs.append(norm(o, pos, pos + steps))
        cs[ci[0].long()] = new[0]
        acc = put(torch.tensor([steps], dtype=torch.int32))
        pos += steps
    both = torch.cat(outs).float()
    # two ways to the same values: states to 2^-18 of their sums, y rounded to bf16 by each, and so is the norm
    assert ((both - want.float()).abs() <= 2.0 ** -6 * want.float().abs() + 2.0 ** -6 * want.float().abs().mean()).all()


@pytest.mark.parametrize("form", [("head", 2, 64, 1, 64), ("channel", 1, 300, 1, 16)])
def test_graphs_of_segments_replay(form):
    """Two captured calls, each with a workspace of its own, replayed in turn with eager calls between them."""
    has = torch.ones(1, dtype=torch.bool, device=DEV)
    runs = []
    for T in (1400, 900):
        d = R.on(R.draw((T,), *form, T, slow=0.05), DEV)
        qsl = torch.tensor([0, T], dtype=torch.int32, device=DEV)
        state = state_of(d, 1, 1, T).to(DEV)
        st, out = state.clone(), torch.zeros_like(d["x"])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call_fwd(d, st, qsl, None, has, out)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call_fwd(d, st, qsl, None, has, out)
        st.copy_(state)
        runs.append((d, qsl, state.clone(), st, out, graph))
    for i in range(3):
        for d, qsl, want, st, out, graph in runs:
            d["x"].mul_(0.9)
            graph.replay()
            wout = call_fwd(d, want, qsl, None, has)
            torch.cuda.synchronize()
            assert torch.equal(st, want) and torch.equal(out, wout), i


@pytest.mark.parametrize("form", [("head", 2, 64, 1, 64), ("channel", 1, 300, 1, 16)])
def test_empty_calls(form):
    d = R.on(R.draw((0,), *form, 1), DEV)
    st = state_of(d, 2, 1, 1).to(DEV)
    before = st.clone()
    out = call_fwd(d, st, torch.tensor([0, 0, 0], dtype=torch.int32), None, torch.ones(2, dtype=torch.bool))
    assert out.shape == d["x"].shape and torch.equal(st, before)
    d = R.on(R.draw((0, 1), *form, 1), DEV)
    assert call_update(d, st).shape == d["x"].shape
    assert torch.equal(st, before)


@pytest.mark.parametrize("lens,form", [([769] * 20, ("head", 2, 64, 1, 64)), ([257] * 40, ("channel", 1, 70, 1, 20))])
def test_segments_whose_last_one_ends_first(lens, form):
    """Last segments of one token, which write their lines while the first ones are at work, on lines that hold a state."""
    prefill(lens, *form, seed=12, init=[True] * len(lens), slow=0.05)
