"""The step sizes: how exact the softplus is, and what a step of 0 does."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
F64 = torch.float64
U = 2.0 ** -24


def scan(form, x, dt, A, B, C, state, T=None, **kw):
    """ssm_fwd_varlen over sequences of T tokens, or (T None) ssm_update; everything on the CPU, the state too."""
    st = state.to(DEV)
    if T is None:
        out = S.ssm_update(*(t.to(DEV) for t in (x, dt, A, B, C)), st, **kw)
    else:
        n = x.shape[0] // T
        qsl = (torch.arange(n + 1) * T).to(torch.int32).to(DEV)
        out = S.ssm_fwd_varlen(*(t.to(DEV) for t in (x, dt, A, B, C)), st, qsl, None, torch.ones(n, dtype=torch.bool, device=DEV), **kw)
    return out.cpu(), st.cpu()


# a token at a time (decode, a prompt of one token), in chunks, a thread a channel
KERNELS = [("head", None), ("head", 1), ("head", 70), ("channel", None), ("channel", 1), ("channel", 24)]


def inputs(form, T, n, H, P, N):
    """x and B of 1 in the last token and of 0 before it, C of 0; (n T, ..), or (n, ..) for decode."""
    rows = n * (T or 1)
    last = torch.zeros(n, T or 1, dtype=BF)
    last[:, -1] = 1
    last = last.view(rows, 1, 1)
    if form == "head":
        return last.expand(rows, H, P).contiguous(), last.expand(rows, 1, N).contiguous(), torch.zeros(rows, 1, N, dtype=BF)
    return last[:, 0].expand(rows, H * P).contiguous(), last.expand(rows, 1, N).contiguous(), torch.zeros(rows, 1, N, dtype=BF)


@pytest.mark.parametrize("form,T", KERNELS)
def test_softplus(form, T):
    """The state after one written token of x = B = 1 is the step size itself.

    Roundings of u = 2^-24, relative to log(1 + e^v): 3 of e^-|v| (two of the exponential, one of what its argument's second part
    adds), 1 of 2 + e, 2 of its reciprocal, 1 of the quotient, 2 of the series, 1 of the sum; what lies below 2^-126 may be 0."""
    H, P, N, n = (64, 4, 8, 40) if form == "head" else (1, 256, 8, 10)
    v = torch.linspace(-87, 30, 2560)
    x, B, C = inputs(form, T, n, H, P, N)
    k = 2560 // n
    dt = torch.zeros(n, T or 1, k)
    dt[:, -1] = v.view(n, k)
    dt = dt.view(-1, k)
    A = -torch.ones(H) if form == "head" else -torch.ones(P, N)
    shape = (n, H, P, N) if form == "head" else (n, P, N)
    _, st = scan(form, x, dt, A, B, C, torch.zeros(shape), T, dt_softplus=True)
    want = torch.logaddexp(v.to(F64), torch.zeros(2560, dtype=F64)).view((n, H, 1, 1) if form == "head" else (n, P, 1)).expand(shape)
    R.check(st, want, 10 * U * want + 2.0 ** -126, "step")


@pytest.mark.parametrize("form,T", KERNELS)
def test_softplus_far_out(form, T):
    H, P, N, n = (4, 4, 8, 1) if form == "head" else (1, 4, 8, 1)
    v = torch.tensor([-float("inf"), -1e30, 1e30, 3e38])
    x, B, C = inputs(form, T, n, H, P, N)
    dt = torch.zeros(T or 1, 4)
    dt[-1] = v
    A = -torch.ones(H) if form == "head" else -torch.ones(P, N)
    shape = (n, H, P, N) if form == "head" else (n, P, N)
    _, st = scan(form, x, dt, A, B, C, torch.zeros(shape), T, dt_softplus=True)
    assert torch.equal(st, v.clamp(min=0).view((n, H, 1, 1) if form == "head" else (n, P, 1)).expand(shape))
    dt[-1] = float("nan")
    _, st = scan(form, x, dt, A, B, C, torch.zeros(shape), T, dt_softplus=True)
    assert torch.isnan(st).all()


# (form, lengths or None for decode): a token at a time, chunks of which a part is empty, segments some of which have no step
# at all, a thread a channel, its segments
FORGETFUL = [("head", 3, 64, 1, 32, None), ("head", 3, 64, 1, 32, [2, 3, 1]), ("head", 3, 64, 1, 32, [70, 5, 129]), ("head", 2, 32, 1, 64, [90]),
             ("head", 2, 64, 1, 32, [1300]), ("head", 2, 16, 1, 160, [40]), ("channel", 1, 70, 1, 16, None),
             ("channel", 2, 20, 2, 20, [2, 1]), ("channel", 1, 70, 1, 16, [70, 5, 129]), ("channel", 1, 70, 1, 5, [1300])]


@pytest.mark.parametrize("form,H,P,G,N,lens", FORGETFUL)
def test_decays_of_minus_infinity(form, H, P, G, N, lens):
    """A step forgets everything, a step of 0 (and what lies behind a sequence's end) nothing.  In 64 bits e^(-10^6 d) is 0 as well
    for every other step here, which is 0.01 or more."""
    rows = (5, 2) if lens is None else (sum(lens),)
    d = R.draw(rows, form, H, P, G, N, 7, raw=False)
    g = torch.Generator().manual_seed(8)
    d["dt"] = torch.where(torch.rand(d["dt"].shape, generator=g) < 0.4, 0.0, d["dt"].clamp(min=0.01))
    if lens and lens[0] > 500:
        d["dt"][150:450] = 0
    d["A"].view(-1)[::3] = -1e6
    shape = (5 if lens is None else len(lens), H, P, N) if form == "head" else (5 if lens is None else len(lens), H * P, N)
    state = torch.randn(shape, generator=g)
    st = state.to(DEV)
    k = R.on(d, DEV)
    k["A"].view(-1)[::3] = -float("inf")
    args = (k["x"], k["dt"], k["A"], k["B"], k["C"], st)
    if lens is None:
        o, otol, s, stol, _ = R.update(d, state, None, None, None)
        out = S.ssm_update(*args, D=k["D"])
    else:
        qsl = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
        has = torch.ones(len(lens), dtype=torch.bool)
        o, otol, s, stol, _ = R.fwd(d, state, qsl, None, has)
        out = S.ssm_fwd_varlen(*args, qsl.to(DEV), None, has.to(DEV), D=k["D"])
    R.check(out, o, otol, "out")
    R.check_state(st, s, stol)
