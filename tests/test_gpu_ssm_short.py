"""Prompts of a few tokens go as decode does, to the last bit."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import ssm_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("form", [("head", 16, 64, 2, 128), ("head", 3, 80, 1, 96), ("channel", 1, 300, 1, 16)])
def test_a_few_tokens_are_a_decode_step(form, n, T):
    d = R.on(R.draw((n, T), *form, 5 + T), DEV)
    state = torch.randn((n, *((form[1], form[2]) if form[0] == "head" else (form[1] * form[2],)), form[4]), device=DEV)
    opts = dict(D=d["D"], dt_bias=d["dt_bias"], dt_softplus=True)
    s1, s2 = state.clone(), state.clone()
    want = S.ssm_update(d["x"], d["dt"], d["A"], d["B"], d["C"], s1, **opts)
    flat = {k: v.flatten(0, 1) for k, v in d.items() if k in ("x", "dt", "B", "C")}
    qsl = torch.arange(n + 1, dtype=torch.int32, device=DEV) * T
    got = S.ssm_fwd_varlen(flat["x"], flat["dt"], d["A"], flat["B"], flat["C"], s2, qsl, None, torch.ones(n, dtype=torch.bool, device=DEV),
                           **opts)
    assert torch.equal(got.view(want.shape), want) and torch.equal(s1, s2)
