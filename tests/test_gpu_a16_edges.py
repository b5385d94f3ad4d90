"""The operators on BF16 activations where test_gpu_a16.py does not go: blocks that outlast one
another, sizes at the limits, one expert that takes all tokens, and the precision that the header
states for the experts' products."""
import time

import pytest
import torch

import a16_ref as ref
from test_gpu_a16 import BF, make_experts, make_layer, make_x, normal, twq  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["linear", "experts"])
@pytest.mark.parametrize("b", [1, 9, 40])
def test_blocks_that_outlast_one_another(twq, device, b, call):
    """Long sums of few columns: a cluster's blocks share one job, and each of them gives up later
    than the block that gets its part. That one still is there when the part comes: the status
    tells, the context stays usable, and the next calls are right."""
    gen = torch.Generator().manual_seed(20 + b)
    if call == "linear":
        x, w = make_x(gen, b, 8192).to(device), make_layer(twq, gen, 8192, 256, 64, device)
        f = lambda: twq.fused_linear_a16(x, w)
    else:
        x, ex = make_x(gen, b, 2048).to(device), make_experts(twq, gen, 2, 2048, 2048, 16, 16, device)
        logits = normal(gen, b, 2).to(device)
        f = lambda: twq.moe_layer(x, logits, 1, ex)[0]
    want = f()
    assert twq.device_status() == 0
    for _ in range(3):
        twq.selftest_a16_stall(100000)
        try:
            t0 = time.perf_counter()
            f()
            code = twq.device_status()
            spent = time.perf_counter() - t0
        finally:
            twq.selftest_a16_stall(0)
        assert 71 <= code <= 76 and spent < 1.0, (code, spent)
        assert twq.device_status() == 0
        assert torch.equal(f(), want) and twq.device_status() == 0


def test_a_block_outwaits_its_peers(twq, device):
    """The last blocks of a cluster of eight give up after 2.8 s, the first, which gets their parts,
    after 0.35 s: it is there when they come."""
    gen = torch.Generator().manual_seed(23)
    x, w = make_x(gen, 1, 8192).to(device), make_layer(twq, gen, 8192, 256, 0, device)
    want = twq.fused_linear_a16(x, w)
    twq.selftest_a16_stall(350000000)
    try:
        t0 = time.perf_counter()
        twq.fused_linear_a16(x, w)
        code = twq.device_status()
        spent = time.perf_counter() - t0
    finally:
        twq.selftest_a16_stall(0)
    assert code == 74 and 0.35 <= spent < 4.0, (code, spent)  # 74: activations that did not come
    assert twq.device_status() == 0 and torch.equal(twq.fused_linear_a16(x, w), want)
