"""Prefill at sizes and values that the other tests leave out: batches around
the longest one that is ordered by length, keys of a wide spread in one row."""
import pytest
import torch

from tests.test_gpu_gdr import prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [511, 512, 513, 700])
def test_many_sequences(n):
    """One kernel; up to 512 sequences start in the order of their lengths, more as they come."""
    lens = [(7 * i) % 5 for i in range(n)]             # empty ones among them
    lens[n - 1], lens[3], lens[n // 2] = 130, 66, 64
    prefill(lens, 1, 2, 8, 8, seed=n, pads=(0, 1, n - 2))


@pytest.mark.parametrize("n", [512, 513])
def test_many_equal_sequences(n):
    prefill([2] * n, 1, 1, 16, 8, seed=n, pads=(n - 1,))


@pytest.mark.parametrize("lens", [[150], [20, 7, 64]])
@pytest.mark.parametrize("l2norm", [True, False])
def test_keys_of_a_wide_spread(lens, l2norm):
    """Elements of a key and query from their norm down to 2^-40 of it: in fp16, 2^-24 of the norm is the last step."""
    def edit(d):
        gen = torch.Generator().manual_seed(3)
        for x in "qk":
            e = torch.randint(0, 41, d[x].shape, generator=gen)
            d[x].mul_(2.0 ** -e.float())
            d[x][..., ::16] = 2.0 ** -4                # (so that no row is all small)
    prefill(lens, 2, 2, 64, 32, seed=17, l2norm=l2norm, edit=edit)
