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


def test_a_matrix_elsewhere_is_named_with_both_devices(monkeypatch):
    """Adapters, layers and experts share the check of their matrices; its message is none of theirs."""
    monkeypatch.setattr(twq, "_dev", lambda t, name, dtype: 16)
    with pytest.raises(ValueError, match="^ids must be on cuda:1, got cpu$"):
        twq._mat(torch.zeros((2, 3), dtype=torch.int32), "ids", torch.int32, 2, 3, torch.device("cuda", 1))
