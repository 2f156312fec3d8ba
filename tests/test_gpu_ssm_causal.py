"""What is not finite in a token's B or C reaches no earlier token, and no other group."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [("head", 4, 64, 2, 64), ("head", 6, 32, 2, 128), ("head", 4, 24, 2, 200), ("channel", 2, 64, 2, 16)]


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("slow", [1.0, 200.0])
@pytest.mark.parametrize("at", [3, 31, 32, 63, 64, 100])
@pytest.mark.parametrize("which", ["B", "C"])
@pytest.mark.parametrize("form", FORMS)
def test_stays_with_its_token_and_those_behind_it(form, which, at, slow, value):
    """B reaches the token and those behind it, C the token alone; heads of the other group neither.  slow 200: decays past 2^-64
    within half a chunk, whose factors are taken another way."""
    T, P = 130, form[2]
    d = R.draw((T,), *form, at, slow=slow)
    state = torch.randn((1, *d["A"].shape, P, form[4]) if form[0] == "head" else (1, *d["A"].shape),
                        generator=torch.Generator().manual_seed(1))
    qsl, has = torch.tensor([0, T], dtype=torch.int32), torch.ones(1, dtype=torch.bool)
    o, otol, s, stol, _ = R.fwd(d, state, qsl, None, has)
    g, st = R.on(d, DEV), state.to(DEV)
    g[which] = g[which].clone()
    g[which][at, 1, 2] = value
    out = S.ssm_fwd_varlen(g["x"], g["dt"], g["A"], g["B"], g["C"], st, qsl.to(DEV), None, has.to(DEV), D=g["D"],
                           dt_bias=g["dt_bias"], dt_softplus=True).cpu()
    # by groups
    got, o, otol = (t.reshape(T, 2, -1) for t in (out, o, otol))
    R.check(got[:, 0], o[:, 0], otol[:, 0], "the other group")
    R.check(got[:at, 1], o[:at, 1], otol[:at, 1], "before")
    assert not torch.isfinite(got[at, 1]).any()
    got, s, stol = (t.cpu().reshape(2, -1, form[4]) for t in (st, s, stol))
    if which == "C":
        R.check(out.reshape(T, 2, -1)[at + 1:, 1], o[at + 1:, 1], otol[at + 1:, 1], "behind")
        R.check_state(got, s, stol)
    else:
        rest = torch.arange(form[4]) != 2
        R.check_state(got[0], s[0], stol[0])
        R.check_state(got[1][:, rest], s[1][:, rest], stol[1][:, rest])
