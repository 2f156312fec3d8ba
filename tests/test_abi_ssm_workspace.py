"""The scan's workspace: what a caller that reserves the stated maximum may rely on (no GPU needed)."""
import itertools
import random

import pytest

import causal_depthwise_short_conv1d_amd as S

MB = 10 ** 6
# stated in sconv.h, by states a channel
HEADS = {128: 51 * MB}
CHANNELS = {16: 24 * MB, 32: 45 * MB, 64: 87 * MB}


@pytest.fixture(scope="module")
def need():
    return S.load_library().ssm_fwd_workspace_bytes


def tokens(batch):
    """Lengths around every step of the plans' segment counts, and far out."""
    r = random.Random(batch)
    yield from (640 * batch, 641 * batch, 704 * batch, 128 * batch, 4096, 14807, 16384, (1 << 31) - 257)
    for _ in range(60):
        yield batch * int(2 ** r.uniform(7, 24))


def test_stated_maxima_hold(need):
    most = dict.fromkeys(("head", 16, 32, 64), 0)
    for batch in (1, 2, 3, 4, 7, 8, 16, 31, 32, 63, 64, 65, 127, 128):
        for T in tokens(batch):
            if T > (1 << 31) - 257:
                continue
            for G, H, P in itertools.chain(((1, h, 64) for h in (1, 4, 8, 63, 64, 128, 252, 256)),
                                           ((g, 8 * g, 64) for g in (2, 8, 32, 63, 64)), ((1, 8, 32), (8, 64, 32), (4, 12, 200)),
                                           ((g, g, 8) for g in (1, 7, 64))):
                for N in (8, 32, 64, 128):
                    most["head"] = max(most["head"], need(batch, T, H, G, P, N, 0))
            for G, P in ((1, 1), (1, 256), (1, 8192), (1, 16384), (1, 32768), (1, 32512), (3, 8192), (7, 1000), (64, 512), (128, 256),
                         (128, 3), (31, 1025)):
                for N in (16, 32, 64):
                    most[N] = max(most[N], need(batch, T, G, G, P, N, 1))
    assert 0.9 * HEADS[128] < most["head"] <= HEADS[128]
    for n, limit in CHANNELS.items():
        assert 0.9 * limit < most[n] <= limit, n


@pytest.mark.parametrize("dims", [(1, 4096, 252, 1, 64, 128, 0), (1, 640, 1, 1, 32768, 64, 1), (1, 640, 1, 1, 32768, 16, 1),
                                  (1, 16384, 1, 1, 8192, 16, 1)])
def test_calls_near_the_maxima(need, dims):
    limit = HEADS[128] if not dims[-1] else CHANNELS[dims[5]]
    assert 0.8 * limit < need(*dims) <= limit


def test_a_workspace_for_channels_serves_heads(need):
    """A (dim, state_dim) whose channels and states share a decay by strides takes the head form's kernel: with what was asked for
    by channels (or none, and then without segments)."""
    r = random.Random(3)
    for _ in range(4000):
        G, P, N = r.choice((1, 1, 2, 8, 64)), r.choice((1, 8, 33, 64, 256, 1000, 8192, 16384)), r.choice((1, 8, 16, 33, 64))
        batch = r.choice((1, 2, 5, 30, 64, 100))
        T = batch * int(2 ** r.uniform(5, 18))
        channels, heads = need(batch, T, G, G, P, N, 1), need(batch, T, G, G, P, N, 0)
        assert channels == 0 or channels >= heads, (batch, T, G, P, N)
