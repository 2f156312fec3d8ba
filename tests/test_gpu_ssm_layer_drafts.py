"""A layer whose drafts stand only in part: every step goes on from the state and the window of its last standing token."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.mark.parametrize("form", [("head", 4, 64, 2, 64), ("channel", 2, 64, 2, 16)])
@pytest.mark.parametrize("stand", [[1, 3, 2, 4], [2, 1, 1, 4, 3]])
def test_steps_go_on_from_the_accepted_one(form, stand):
    """Two requests of 4 drafted tokens a step, of which `stand` (the other: the list backwards) are kept.  What the steps gave for the
    kept tokens against one pass over them in 64 bits: the convolution within half a bf16 step (2^-8) and a few u of its
    terms, the scan within the recurrence's bound on the convolution's own outputs."""
    head = form[0] == "head"
    H, P, G, N = form[1:]
    dim, cd, steps, n = H * P, H * P + 2 * G * N, 4, 2
    g = torch.Generator().manual_seed(len(stand))
    w = (torch.randn(cd, 4, generator=g) * 0.4).to(BF).to(DEV)
    kept = [stand, stand[::-1]]
    total = max(sum(k) for k in kept)
    xbc = torch.randn(n, total + steps, cd, generator=g).to(BF)       # what the requests' kept tokens bring
    junk = torch.randn(n, steps, cd, generator=g).to(BF)              # and the drafts that do not stand
    d = R.on(R.draw((n, total + steps), *form, 10, gate=True), DEV)

    def parts(y, dt, z):
        x, B, C = y[..., :dim], y[..., dim:dim + G * N], y[..., dim + G * N:]
        q = dict(d)
        q.update(x=x.unflatten(-1, (H, P)) if head else x, B=B.unflatten(-1, (G, N)), C=C.unflatten(-1, (G, N)), dt=dt, z=z)
        return q
    lines = torch.arange(n * steps, dtype=torch.int32, device=DEV).view(n, steps)
    st = torch.randn((n * steps, H, P, N) if head else (n * steps, dim, N), generator=g).to(DEV)
    first = st[::steps].clone()
    window = torch.zeros(n * steps, cd, 3, dtype=BF, device=DEV)
    acc = torch.ones(n, dtype=torch.int32, device=DEV)                # the first step reads each request's first line
    outs, convs, at = [[], []], [[], []], [0, 0]
    for k in range(len(stand)):
        now = [kept[b][k] for b in range(n)]
        x = torch.stack([torch.where(torch.arange(steps)[:, None] < now[b], xbc[b, at[b]:at[b] + steps], junk[b]) for b in range(n)]).to(DEV)
        hist = window[lines.gather(1, acc.long()[:, None] - 1)[:, 0].long()]
        new = torch.zeros(n, steps, cd, 3, dtype=BF, device=DEV)
        y = S.conv1d_update(x.transpose(1, 2).contiguous(), hist, w, intermediate=new).transpose(1, 2)
        dt, z = (torch.stack([d[t][b, at[b]:at[b] + steps] for b in range(n)]) for t in ("dt", "z"))
        q = parts(y, dt, z)
        o = S.ssm_update(q["x"], q["dt"], q["A"], q["B"], q["C"], st, lines, acc, lines, D=q["D"], z=q["z"], dt_bias=q["dt_bias"],
                         dt_softplus=True)
        window[lines.long()] = new
        for b in range(n):
            outs[b].append(o[b, :now[b]])
            convs[b].append(y[b, :now[b]])
            at[b] += now[b]
        acc = torch.tensor(now, dtype=torch.int32, device=DEV)
    for b in range(n):
        T = sum(kept[b])
        assert T == at[b]
        y = torch.cat(convs[b])
        past = torch.cat([torch.zeros(3, cd, dtype=torch.float64), xbc[b, :T].double()])
        terms = torch.stack([past[j:j + T] * w.double().cpu()[:, j] for j in range(4)])
        want = terms.sum(0)
        R.check(y, want, 2.0 ** -8 * want.abs() + 8 * 2.0 ** -24 * terms.abs().sum(0), "convolution")
        q = parts(y, d["dt"][b, :T], d["z"][b, :T])
        ref = R.fwd({m: v.cpu() if isinstance(v, torch.Tensor) else v for m, v in q.items()}, first[b:b + 1].cpu(), [0, T], None, [True])
        R.check(torch.cat(outs[b]), ref[0], ref[1], "out")
        R.check_state(st[b * steps + kept[b][-1] - 1][None], ref[2], ref[3])
