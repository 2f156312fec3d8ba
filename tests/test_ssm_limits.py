"""Step size limits past fp32, as programs give them that mean none (no GPU needed)."""
import ctypes
import sys

import pytest
import torch

import causal_depthwise_short_conv1d_amd as S

INF = float("inf")


@pytest.mark.parametrize("given,want", [(None, (-INF, INF)), ((0.0, sys.float_info.max), (0.0, INF)), ((-1e300, 0.5), (-INF, 0.5)),
                                        ((0, INF), (0.0, INF)), ((0.125, torch.finfo(torch.float32).max), (0.125, 3.4028234663852886e38))])
def test_limits_are_packed(monkeypatch, given, want):
    """They reach the library as fp32; what fp32 does not have is no limit."""
    S.load_library()
    pack, _ = S._packed["ssm_update"]
    got = []
    monkeypatch.setattr(S, "_launch_packed", lambda fn, dev, args: got.append(pack(*args, 0)))
    for name in ("_dev", "_ptr"):
        monkeypatch.setattr(S, name, lambda t, *a: 0 if t is None else t.data_ptr())
    bf = torch.bfloat16
    S.ssm_update(torch.zeros(3, 4, 8, dtype=bf), torch.zeros(3, 4), torch.zeros(4), torch.zeros(3, 2, 16, dtype=bf),
                 torch.zeros(3, 2, 16, dtype=bf), torch.zeros(3, 4, 8, 16), dt_limit=given)
    lo = S.load_library().ssm_update.argtypes.index(ctypes.c_float)
    words = torch.frombuffer(bytearray(got[0]), dtype=torch.float32)[::2]
    assert (float(words[lo]), float(words[lo + 1])) == want
