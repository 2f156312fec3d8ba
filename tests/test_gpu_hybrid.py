"""A linear-attention layer's serving steps with the operators together: the
convolution feeds the gated delta rule its q, k and v (views of one output),
over a packed prefill and then speculative steps, in which the verification's
num_accepted_tokens tells both caches what stood.  Against the oracle's
convolution and the 64-bit recurrence of the tokens that were accepted."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
import oracle
from tests import gdr_ref as R
from tests.parity import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
HK, HV, D, W = 2, 4, 32, 4
DIM = 2 * HK * D + HV * D
LENS, DRAFTS, VOCAB = [70, 3, 140, 1], 3, 50
N, STEPS = len(LENS), DRAFTS + 1


def views(rows):
    """q, k and v of (.., DIM) convolution outputs."""
    lead = rows.shape[:-1]
    return (rows[..., :HK * D].view(*lead, HK, D), rows[..., HK * D:2 * HK * D].view(*lead, HK, D),
            rows[..., 2 * HK * D:].view(*lead, HV, D))


@pytest.mark.parametrize("graph", [False, True])
def test_prefill_then_speculative_steps(graph):
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    total = sum(LENS)
    w, bias = (rnd(DIM, W) * 0.5).to(BF).to(DEV), (rnd(DIM) * 0.1).to(BF).to(DEV)
    A_log, dt_bias = torch.rand(HV, generator=gen).to(DEV), (rnd(HV) - 3).to(DEV)
    opts = dict(A_log=A_log, dt_bias=dt_bias, use_qk_l2norm=True)
    qsl = torch.tensor([0] + torch.tensor(LENS).cumsum(0).tolist(), dtype=torch.int32)

    # lines: the convolution's rolling windows; one state a request and step
    conv = torch.zeros(N + 2, DIM, W - 2 + STEPS, dtype=BF, device=DEV)
    state = torch.zeros(N * STEPS + 3, HV, D, D, device=DEV)
    conv_line = torch.randperm(N + 2, generator=gen)[:N].to(torch.int32)
    lines = torch.randperm(N * STEPS + 3, generator=gen)[:N * STEPS].to(torch.int32).view(N, STEPS).contiguous()

    x = rnd(total, DIM).to(BF)
    a, b = rnd(total, HV).to(BF), rnd(total, HV).to(BF)
    y = S.conv1d_fwd_varlen(x.to(DEV).t(), w, bias, conv[:, :, :W - 1], qsl.to(DEV), conv_line.to(DEV), None)
    q, k, v = views(y.t())
    out = S.gdr_fwd_varlen(q, k, v, a.to(DEV), b.to(DEV), state, qsl.to(DEV), lines[:, 0].contiguous().to(DEV), None, **opts)

    # what each request has taken in so far, for the reference
    took = [dict(x=[x[qsl[i]:qsl[i + 1]]], y=[y.t()[qsl[i]:qsl[i + 1]].cpu()], a=[a[qsl[i]:qsl[i + 1]]],
                 b=[b[qsl[i]:qsl[i + 1]]], o=[out[qsl[i]:qsl[i + 1]].cpu()]) for i in range(N)]

    xs, ys = torch.zeros(N, STEPS, DIM, dtype=BF, device=DEV), torch.zeros(N, STEPS, DIM, dtype=BF, device=DEV)
    ga, gb = torch.zeros(N, STEPS, HV, dtype=BF, device=DEV), torch.zeros(N, STEPS, HV, dtype=BF, device=DEV)
    out = torch.zeros(N, STEPS, HV, D, dtype=BF, device=DEV)
    accepted = torch.ones(N, dtype=torch.int32, device=DEV)          # prefill left one state, and a window of one step
    tokens = torch.zeros(N, DRAFTS + 1, dtype=torch.int32, device=DEV)
    start = (torch.arange(N + 1) * DRAFTS).to(torch.int32).to(DEV)
    p, qd = torch.zeros(N * STEPS, VOCAB, device=DEV), torch.zeros(N * DRAFTS, VOCAB, device=DEV)
    drafts = torch.zeros(N * DRAFTS, dtype=torch.int32, device=DEV)
    ua, us = torch.zeros(N * DRAFTS, device=DEV), torch.zeros(N, device=DEV)
    cl, ll = conv_line.to(DEV), lines.to(DEV)

    def step():
        S.conv1d_update(xs.transpose(1, 2), conv, w, bias, "silu", cl, num_accepted_tokens=accepted,
                        out=ys.transpose(1, 2))
        q, k, v = views(ys)
        S.gdr_update(q, k, v, ga, gb, state, ll, accepted, ll, out=out, **opts)
        S.sconv_verify_drafts(drafts, start, p, qd, ua, us, DRAFTS, tokens, accepted)

    def fill():
        xs.copy_(rnd(N, STEPS, DIM))
        ga.copy_(rnd(N, STEPS, HV))
        gb.copy_(rnd(N, STEPS, HV))
        lp = rnd(N * STEPS, VOCAB)
        own = torch.tensor([i for i in range(N * STEPS) if i % STEPS < DRAFTS])
        lq = lp[own] + 0.7 * rnd(len(own), VOCAB)
        p.copy_(torch.softmax(lp, -1))
        qd.copy_(torch.softmax(lq, -1))
        drafts.copy_(torch.multinomial(torch.softmax(lq, -1), 1, generator=gen)[:, 0])
        ua.copy_(torch.rand(N * DRAFTS, generator=gen))
        us.copy_(torch.rand(N, generator=gen))

    if graph:
        keep = [t.clone() for t in (conv, state, accepted)]
        fill()
        step()                                         # (what the step does to the caches is taken back)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for t, s in zip((conv, state, accepted), keep):
            t.copy_(s)
    counts = []
    for _ in range(5):
        fill()
        if graph:
            g.replay()
        else:
            step()
        torch.cuda.synchronize()
        want = R.verify(drafts.cpu(), start.cpu(), p.cpu(), qd.cpu(), ua.cpu(), us.cpu(), DRAFTS)
        assert torch.equal(tokens.cpu(), want[0]) and torch.equal(accepted.cpu(), want[1])
        counts += want[1].tolist()
        for i, n in enumerate(want[1].tolist()):
            for name, t in (("x", xs), ("y", ys), ("a", ga), ("b", gb), ("o", out)):
                took[i][name].append(t[i, :n].cpu())
    assert 1 in counts and max(counts) > 1

    final = accepted.cpu()
    for i, t in enumerate(took):
        x, y, a, b, o = (torch.cat(t[n]) for n in "xyabo")
        ref = torch.empty(DIM, len(x), dtype=BF)
        oracle.fwd_varlen(x.t().contiguous(), w.cpu(), bias.cpu(), None, torch.tensor([0, len(x)], dtype=torch.int32), ref)
        assert_close(y.t(), ref, f"convolution of request {i}")
        q, k, v = views(y)
        zero = torch.zeros(1, HV, D, D)
        ro, rtol, rs, rst, _ = R.fwd(q, k, v, a, b, zero, [0, len(x)], None, None, A_log.cpu(), dt_bias.cpu(), D ** -0.5, True,
                                     R.C_CHUNK, R.F_CHUNK)
        R.check(o, ro, rtol, f"output of request {i}")
        R.check_state(state[lines[i, final[i] - 1].item()].cpu()[None], rs, rst, f"state of request {i}")
