"""Calls that the binding refuses before it reads an operand; none needs a device."""
import pytest
import torch

from rank_residual_w4a4_b200 import _build, twq


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    twq.load()


def test_experts_need_their_weights(monkeypatch):
    """moe_experts reads the slots' weights. Left out, they would be a new buffer that nothing has
    written."""
    made = []
    monkeypatch.setattr(twq, "_moe_buffers", lambda *a: pytest.fail("went on without weights"))
    monkeypatch.setattr(twq, "_empty", lambda *a: made.append(a))
    for weights in (None, 1.0, [1.0]):
        with pytest.raises(TypeError, match="weights"):
            twq.moe_experts(torch.zeros((2, 128), dtype=torch.bfloat16), torch.zeros((2, 1), dtype=torch.int32),
                            weights, None)
    assert not made
