"""The chunked delta rule holds each value channel's state in a power-of-two
unit of its own.  Here the unit has to follow what the channel goes through:
chunks that write nothing, states decayed to nothing, tiny states before
ordinary values.  Against the 64-bit recurrence, in both kernel forms."""
import pytest
import torch

import causal_depthwise_short_conv1d_amd as S
from tests import gdr_ref as R
from tests.test_gpu_gdr import prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["two_kernels", "one_kernel"])
def form(request, monkeypatch):
    """A call of few heads and more than 64 tokens a sequence takes two kernels with its workspace, one without."""
    if request.param == "one_kernel":
        real = S._launch_packed
        monkeypatch.setattr(S, "_launch_packed", lambda fn, dev, args: real(fn, dev, (*args[:-2], 0, 0)))
    return request.param


def run(n, edit, **kw):
    prefill([n], 1, 2, 64, 32, seed=n, raw=False, edit=edit, **kw)


@pytest.mark.parametrize("size", [1.0, 1e3])
@pytest.mark.parametrize("zeros", [64, 128, 192])
@pytest.mark.parametrize("at,decay", [(0, 0.0), (0, -2.0), (64, 0.0), (64, -1.0), (70, -0.5), (70, -2.0)])
@pytest.mark.parametrize("what", ["v", "beta"])
def test_chunks_that_write_nothing(form, what, at, decay, zeros, size):
    """Zero values or zero write strength for whole chunks (a masked or padded prefix, or in mid-sequence), then values."""
    def edit(d):
        d[what][at:at + zeros] = 0.0
        d["g"][at:at + zeros] = decay
        d["v"][at + zeros:] *= size
    run(at + zeros + 75, edit, init=[at > 0])


def test_zero_channels_beside_live_ones(form):
    def edit(d):
        d["v"][:200, :, ::3] = 0.0
        d["v"][70:260, :, 1] = 0.0
        d["v"][:, :, 31] = 0.0
    run(290, edit, init=[False])


@pytest.mark.parametrize("decay", [-1.0, -30.0, float("-inf")])
def test_full_decay_over_two_chunks_then_values(form, decay):
    def edit(d):
        d["v"][64:192] = 0.0
        d["g"][64:192] = decay
        d["v"][192:] *= 100.0
    run(270, edit, init=[True])


@pytest.mark.parametrize("scale", [1e-12, 1e-30, 1e-34, 1e-37])
@pytest.mark.parametrize("size", [0.0, 1e-30, 1.0, 1e3])
def test_tiny_initial_states(form, scale, size):
    """Nothing but the state (size 0), values like it, and ordinary ones after a tiny state."""
    def edit(d):
        d["v"] *= size
        d["g"] *= 0.02                                 # some of the state is left at the end
        if size > 1:
            d["v"][:64] = 0.0
    run(150, edit, init=[True], state_scale=scale)


@pytest.mark.parametrize("exponent", [20, 50, 70, 76])
def test_large_values_after_nothing(form, exponent):
    """Values of up to 2^79 (draws reach six) in a channel whose unit is as high as it gets."""
    def edit(d):
        d["v"][:128] = 0.0
        d["g"][:128] = -0.7
        d["v"][128:] *= 2.0 ** exponent
    run(260, edit, init=[True])


def test_large_state_that_goes_and_small_values(form):
    def edit(d):
        d["g"][64:128] = float("-inf")
        d["v"][64:] *= 2.0 ** -30
    run(200, edit, init=[True], state_scale=1e20)
