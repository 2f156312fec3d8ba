"""How many bits the head form's chunks keep on the way to the outputs.

Terms of nearly equal size and opposite sign leave an output that is small
beside them (2^-11 of them or less), so its own rounding to bf16 does not hide
what its terms were rounded to.  u = 2^-24; M: the terms' magnitudes."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
F64 = torch.float64
U = 2.0 ** -24
T = 64                       # one chunk a sequence

# (heads, head_dim, state_dim, sequences): two waves a head in workgroups of two, four and eight; a wave a head
SHAPES = [(4, 64, 128, 2), (16, 64, 128, 20), (16, 64, 128, 34), (16, 64, 64, 34), (16, 64, 32, 34), (6, 32, 128, 3), (5, 32, 64, 2),
          (6, 96, 48, 3)]


def rand(g, *shape):
    return torch.rand(shape, generator=g)


def signs(g, *shape):
    return 1.0 - 2.0 * torch.randint(0, 2, shape, generator=g)


def call(x, dt, A, B, C, state, nseq, pitch):
    """x .. on the CPU; pitch: rows `pitch` elements longer than what they hold, from an odd place on."""
    def place(t):
        if not pitch:
            return t.to(DEV)
        w = torch.zeros((*t.shape[:-1], t.shape[-1] + pitch), dtype=t.dtype, device=DEV)[..., 1:1 + t.shape[-1]]
        return w.copy_(t)
    qsl = (torch.arange(nseq + 1) * T).to(torch.int32).to(DEV)
    has = torch.ones(nseq, dtype=torch.bool, device=DEV)
    return S.ssm_fwd_varlen(place(x), dt.to(DEV), A.to(DEV), place(B), place(C), state.to(DEV), qsl, None, has).cpu()


@pytest.mark.parametrize("pitch", [0, 3])
@pytest.mark.parametrize("H,P,N,nseq", SHAPES)
def test_states_keep_their_bits_in_the_outputs(H, P, N, nseq, pitch):
    """y = e^G c (S_a + S_b) with S_b = -(1 + t) S_a, t below 2^-12.

    c times a bf16 part of S is exact in fp32, and so are the zeros between them: S's parts, three each if they hold all of its
    24 bits, are at most 6 terms, whose sums are off by 2 u M each at most: 12 u M.  e^G and its product: by 2^-16 of y."""
    g = torch.Generator().manual_seed(H + P + N + nseq)
    rows = nseq * T
    first = (rand(g, nseq, H, P) + 1) * signs(g, nseq, H, P)
    state = torch.zeros(nseq, H, P, N)
    a = torch.randint(0, N, (nseq, H, P, 1), generator=g)
    b = (a + torch.randint(1, N, (nseq, H, P, 1), generator=g)) % N
    state.scatter_(3, a, first[..., None])
    state.scatter_(3, b, -(first * (1 + rand(g, nseq, H, P) * 2.0 ** -12))[..., None])
    c = ((rand(g, rows, 1, 1) + 1) * signs(g, rows, 1, 1)).to(BF).expand(rows, 1, N).contiguous()
    x = torch.randn(rows, H, P, generator=g).to(BF)
    dt = rand(g, rows, H) * 2.0 ** -6
    A = -rand(g, H) - 0.5
    out = call(x, dt, A, torch.zeros(rows, 1, N, dtype=BF), c, state, nseq, pitch)
    e = torch.exp((dt.to(F64) * A.to(F64)).view(nseq, T, H).cumsum(1))[..., None]
    s = state.to(F64)[:, None]
    cc = c.to(F64)[:, 0, 0].view(nseq, T, 1, 1)
    y, M = e * cc * s.sum(-1), e * cc.abs() * s.abs().sum(-1)
    assert (y.abs() < 2.0 ** -12 * M).all()
    R.check(out.view(y.shape), y, 16 * U * M + (2.0 ** -8 + 2.0 ** -16) * y.abs(), "out")


@pytest.mark.parametrize("pitch", [0, 3])
@pytest.mark.parametrize("first,second", [(0, 1), (30, 31), (3, 40), (31, 32), (33, 37)])
@pytest.mark.parametrize("H,P,N,nseq", SHAPES)
def test_scores_keep_their_bits_in_the_outputs(H, P, N, nseq, first, second, pitch):
    """y_i = b c_i v (e^(G_i - G_a) d_a - e^(G_i - G_b) d_b) from two tokens a < b with x of v and -v.

    A score b c is exact (16 bits).  Its factors e^(G_i - R) and e^(R - G_j) d, |G| below 2^-4: an exponential is off by 2 u and
    |G| u, the product with d and the two with the score by u each: 8 u of the term in all.  The parts of a weighted score times
    v are exact, 6 at most, whose sums are off by 2 u M each: 12 u M.  (G is summed in 64 bits of d A rounded to 32: u |G|.)"""
    g = torch.Generator().manual_seed(H + P + N + nseq + first)
    rows = nseq * T
    n = int(torch.randint(0, N, (1,), generator=g))
    B, C = (torch.zeros(rows, 1, N, dtype=BF) for _ in range(2))
    B[:, 0, n] = 1.375
    C[:, 0, n] = ((rand(g, rows) + 1) * signs(g, rows)).to(BF)
    x = torch.zeros(nseq, T, H, P, dtype=BF)
    x[:, first] = ((rand(g, nseq, H, P) + 1) * signs(g, nseq, H, P)).to(BF)
    x[:, second] = -x[:, first]
    d = rand(g, nseq, 1, H) * 2.0 ** -3 + 2.0 ** -3
    dt = d.expand(nseq, T, H) * (1 + rand(g, nseq, T, H) * 2.0 ** -14)
    A = -(rand(g, H) + 0.5) * 2.0 ** -11 / (second - first + 63)
    state = torch.zeros(nseq, H, P, N)
    out = call(x.view(rows, H, P), dt.reshape(rows, H), A, B, C, state, nseq, pitch)
    G = (dt.to(F64) * A.to(F64)).cumsum(1)
    w = torch.exp(G[:, :, None] - G[:, None]) * dt.to(F64)[:, None]              # (sequence, i, j, head)
    w = w * torch.ones(T, T, dtype=F64).tril()[None, :, :, None]
    t = [w[:, :, j, :, None] * x.to(F64)[:, j][:, None] for j in (first, second)]
    cc = 1.375 * C.to(F64)[:, 0, n].view(nseq, T, 1, 1)
    y, M = cc * (t[0] + t[1]), cc.abs() * (t[0].abs() + t[1].abs())
    assert (y.abs() < 2.0 ** -11 * M)[:, second:].all()
    R.check(out.view(y.shape), y, 24 * U * M + (2.0 ** -8 + 2.0 ** -16) * y.abs(), "out")
