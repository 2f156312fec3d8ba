"""The kernels that long and large prompts take, against the 64-bit recurrence: workgroups of eight waves, several to a place,
several groups; segments of more than the least length, with empty, short and padded sequences between them, in every layout."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FILL = -3.0


def workspace(lens, form, H, P, G, N):
    need = S.load_library().ssm_fwd_workspace_bytes
    return need(len(lens), sum(lens), H, G, P, N, 0) if form == "head" else need(len(lens), sum(lens), G, G, H * P // G, N, 1)


def run(lens, form, H, P, G, N, seed=0, pads=(), layout=None, tail=0, **kw):
    """As test_gpu_ssm.prefill, with the recurrence on the GPU."""
    d = R.draw((sum(lens) + tail,), form, H, P, G, N, seed, **kw)
    gen = torch.Generator().manual_seed(seed + 1)
    lines = len(lens) + 3
    state = torch.randn((lines, H, P, N) if form == "head" else (lines, H * P, N), generator=gen) * 0.3
    qsl = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    ci = torch.randperm(lines, generator=gen)[:len(lens)].to(torch.int32)
    ci[list(pads)] = -1
    has = torch.rand(len(lens), generator=gen) < 0.7
    g, st = R.on(d, DEV), state.to(DEV)
    with torch.device(DEV):
        o, otol, s, stol, live = (t.cpu() for t in R.fwd(g, st, qsl, ci, has))
    out = torch.full(d["x"].shape, FILL, dtype=BF, device=DEV)
    if layout == "offset":                             # rows from odd places on, read by elements
        def wide(t):
            return torch.full((*t.shape[:-1], t.shape[-1] + 3), 7.0, dtype=t.dtype, device=DEV)[..., 1:1 + t.shape[-1]].copy_(t)
        for n in ("x", "B", "C", "z", "dt"):
            g[n] = None if g[n] is None else wide(g[n])
        out = wide(out)
    elif layout == "state_t":
        st = st.transpose(-1, -2).contiguous().transpose(-1, -2)
    S.ssm_fwd_varlen(g["x"], g["dt"], g["A"], g["B"], g["C"], st, qsl.to(DEV), ci.to(DEV), has.to(DEV), D=g["D"], z=g["z"],
                     dt_bias=g["dt_bias"], dt_softplus=g["dt_softplus"], out=out)
    got = out.cpu()
    R.check(got[live], o[live], otol[live], "out")
    assert (got[~live] == FILL).all()
    R.check_state(st, s, stol)


# no segments, eight waves a workgroup: (sequences, heads, head_dim, groups, states)
@pytest.mark.parametrize("n,H,P,G,N", [(17, 32, 64, 2, 128), (33, 16, 64, 2, 128), (9, 64, 64, 8, 128), (20, 16, 128, 2, 64), (34, 16, 64, 1, 32)])
@pytest.mark.parametrize("layout,gate", [(None, False), (None, True), ("offset", True), ("state_t", False)])
def test_large_batches(n, H, P, G, N, layout, gate):
    lens = [1 + (i * 53) % 140 for i in range(n)]
    lens[3] = 0
    assert workspace(lens, "head", H, P, G, N) == 0
    run(lens, "head", H, P, G, N, seed=n, pads=(1, n - 2), layout=layout, tail=3, gate=gate)


SEGMENTED = [([1344], "head", 128, 64, 8, 128),                     # segments of 3 chunks, 32 workgroups a place
             ([4300], "head", 32, 64, 2, 128),                      # of 3
             ([2000, 1, 0, 2100, 64], "head", 32, 64, 2, 128),
             ([1700, 0, 1400, 5], "head", 16, 64, 1, 64), ([1100, 1, 900], "head", 12, 32, 3, 128), ([1500, 0, 900], "head", 8, 130, 2, 32),
             ([1300], "channel", 1, 8192, 1, 16),                   # of 48 tokens
             ([3000, 1, 0, 1900, 9], "channel", 2, 2048, 2, 16),
             ([700, 0, 900], "channel", 1, 300, 1, 33), ([1111], "channel", 2, 100, 2, 64), ([900, 3, 0, 500], "channel", 1, 1000, 1, 24)]


@pytest.mark.parametrize("lens,form,H,P,G,N", SEGMENTED)
@pytest.mark.parametrize("layout", [None, "offset", "state_t"])
def test_segments(lens, form, H, P, G, N, layout):
    assert workspace(lens, form, H, P, G, N) > 0
    run(lens, form, H, P, G, N, seed=lens[0], layout=layout, slow=0.05, tail=2)


@pytest.mark.parametrize("lens,form,H,P,G,N", [c for c in SEGMENTED if len(c[0]) > 2])
@pytest.mark.parametrize("gate", [False, True])
def test_segments_beside_padded_sequences(lens, form, H, P, G, N, gate):
    """Each of the long ones in turn is padded, and so is a short one."""
    long = [i for i, n in enumerate(lens) if n > 400]
    short = [i for i, n in enumerate(lens) if n <= 400]
    assert workspace(lens, form, H, P, G, N) > 0
    for i in long:
        run(lens, form, H, P, G, N, seed=i, pads=(i, short[-1]), slow=0.05, gate=gate)
