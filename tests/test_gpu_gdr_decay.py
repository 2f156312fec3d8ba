"""States and outputs that decay inside one chunk: what is left at its end is
held to 2^-26 of the channel's largest value in the chunk, beside the relative
roundings of the tokens' own sums (gdr_ref's bound without its floor)."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import gdr_ref as R
from tests.test_gpu_gdr import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["two_kernels", "one_kernel"])
@pytest.mark.parametrize("dk,dv", [(64, 32), (128, 128)])
@pytest.mark.parametrize("values,decay", [(20, -0.3), (20, -1.0), (40, -0.7), (5, -0.2), (1, -0.25)])
def test_decay_within_a_chunk(monkeypatch, form, dk, dv, values, decay):
    if form == "one_kernel":
        real = S._launch_packed
        monkeypatch.setattr(S, "_launch_packed", lambda fn, dev, args: real(fn, dev, (*args[:-2], 0, 0)))
    n, hk, hv, scale = 128, 1, 2, dk ** -0.5
    d = R.draw_inputs((n,), hk, hv, dk, dv, seed=values, raw=False)
    for a in (0, 64):                                  # values at the start of a chunk, then nothing but decay
        d["v"][a + values:a + 64] = 0.0
        d["g"][a + values:a + 64] = decay
    d["v"][64:] = 0.0
    d["v"][64:64 + values] = d["v"][:values]
    state = torch.zeros(1, hv, dv, dk)
    # (a factor that is not C_CHUNK: no floor)
    o, otol, s, stol, _ = R.fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], state, [0, n], None, None, None, None, scale, True,
                                R.C_CHUNK * 1.0001, R.F_CHUNK)
    g, st = R.on(d, DEV), state.to(DEV)
    out = S.gdr_fwd_varlen(g["q"], g["k"], g["v"], g["g"], g["beta"], st, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                           scale=scale, use_qk_l2norm=True)
    largest = d["v"].double().abs().amax(0)            # per head and channel, the same in both chunks
    R.check_state(st, s, stol + 2.0 ** -26 * largest)
    qn = R.norm_qk(d["q"], d["k"], scale, True, hv)[0].norm(dim=-1)
    R.check(out, o, otol + 2.0 ** -26 * largest * qn[..., None], "out")
