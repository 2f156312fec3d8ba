"""Prefill whose workspace cannot be had: the forms that need none answer it."""
import pytest
import torch

from tests.test_gpu_gdr import prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv", [(128, 64), (36, 20)])
def test_prefill_when_the_workspace_does_not_fit(monkeypatch, dk, dv):
    """Vector layouts take one kernel, others go a token at a time."""
    real, asked = torch.empty_strided, []

    def empty_strided(size, stride, **kw):
        if kw.get("dtype") is torch.uint8:
            asked.append(size[0])
            raise torch.OutOfMemoryError("no memory for the workspace")
        return real(size, stride, **kw)
    monkeypatch.setattr(torch, "empty_strided", empty_strided)
    prefill([200, 70], 1, 2, dk, dv, seed=dk)
    assert asked and asked[0] > 0
