"""What the host computes for launches on BF16 activations, from the kernel's own translation unit."""
import ctypes
import hashlib
import os
import random
import subprocess

import pytest

from test_a16_plan import CSRC, DEPS, ROOT, _nvcc

HARNESS = os.path.join(ROOT, "tests", "a16_host_harness.cu")


@pytest.fixture(scope="module")
def harness():
    h = hashlib.sha256()
    for d in [HARNESS] + DEPS[1:]:
        with open(d, "rb") as fh:
            h.update(fh.read())
    out_dir = os.path.join(ROOT, "tests", "_build")
    os.makedirs(out_dir, exist_ok=True)
    path = os.path.join(out_dir, "liba16host_%s.so" % h.hexdigest()[:16])
    if not os.path.exists(path):
        # PTX only for the device side: the harness runs host code alone. What launches call in other
        # files may stay unresolved.
        tmp = path + ".tmp%d" % os.getpid()
        cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=compute_100a", "-std=c++17", "-O1",
               "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
               HARNESS, "-o", tmp]
        try:
            subprocess.run(cmd, check=True, capture_output=True, timeout=900)
        except FileNotFoundError:
            pytest.skip("nvcc is not available")
        os.replace(tmp, path)
    return ctypes.CDLL(path, mode=os.RTLD_LAZY)


@pytest.mark.parametrize("ns,stall", [(2000000000, 0), (1000, 1), (200000, 1), (1000000000, 1)])
def test_a_block_outwaits_every_peer_that_sends_to_it(harness, ns, stall):
    """A block that began a job waits for the parts of the blocks that go on with it, from the end of its
    own steps. Whenever theirs run into their limits, in any step and in as many as there are before
    one runs out, they have sent before its limit is over: a store may not meet a block that left."""
    wait, parts = harness.twq_test_a16_wait_limit, harness.twq_test_a16_parts_limit
    wait.restype = parts.restype = ctypes.c_uint64
    wait.argtypes = [ctypes.c_uint64, ctypes.c_int, ctypes.c_int]
    parts.argtypes = [ctypes.c_uint64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    step_ns = 2000  # what is not waiting: 240 to 707 cycles a group of 32 columns, two groups a step, twofold
    rng = random.Random(ns)
    for _ in range(2000):
        split_log = rng.choice([1, 2, 3])
        split, steps, jobs = 1 << split_log, rng.randint(1, 200), rng.randint(1, 4)
        total = steps * jobs
        begin = [total * r >> split_log for r in range(split + 1)]
        for r in range(split):
            lo, hi = begin[r], begin[r + 1]
            if lo == hi or hi % steps == 0:
                continue
            for q in range(r + 1, split):
                mine = begin[q + 1] - begin[q]
                if begin[q] >= hi - hi % steps + steps or not mine:
                    continue
                longest = 2 * mine * wait(ns, stall, q) + mine * step_ns
                assert parts(ns, stall, split, hi - lo) > longest


def test_every_device_is_asked_once(harness):
    """How many clusters run at once is asked once for each kernel, device and number of blocks on an SM,
    on as many devices as a machine has and in any order; the answers are each device's own."""
    out = (ctypes.c_int64 * 2)()

    def plans(dev):
        harness.twq_test_a16_plans(ctypes.c_int(dev), out)
        return out[0], out[1]

    first = [plans(d) for d in range(16)]
    assert len({asked for asked, _ in first}) == 1 and first[0][0] % 4 == 0
    assert first[0][0] // 4 <= 27 * 3
    assert len({s for _, s in first}) > 1  # other devices, other plans
    for d in reversed(range(16)):
        assert plans(d) == (0, first[d][1])
    # a device beyond the places for answers is asked again, and gets its own plan all the same
    far = plans(1000)
    assert far[0] > 0 and plans(1000) == far and far[1] != first[0][1]


@pytest.mark.parametrize("all_there", [True, False])
def test_the_kernels_shares_fit_together(harness, all_there):
    """The kernel's own walk: each step of each job is one block's; a block that goes on with a job sends its
    part to the block that began it, to a place that is there; and that one waits for exactly those."""
    shares = harness.twq_test_a16_shares
    shares.restype = ctypes.c_int64
    out = (ctypes.c_int64 * 3)()
    begin, owner, others = (ctypes.c_int * 9)(), (ctypes.c_int * 8)(), (ctypes.c_int * 8)()
    rng = random.Random(7 + all_there)
    for _ in range(600):
        jobs, per = int(rng.choice([1, 2, 5, 40, 150, 700]) * rng.uniform(1, 2)), rng.choice([1, 2, 3, rng.randint(1, 60)])
        room, per_sm = rng.choice([((148, 74, 36, 15), 1), ((296, 148, 71, 33), 2), ((444, 222, 107, 48), 3)])
        harness.twq_test_a16_plan(ctypes.c_int64(jobs), ctypes.c_int64(per), (ctypes.c_int * 4)(*room), per_sm,
                                  rng.choice([4, 8]), int(all_there), out)
        clusters, log, room_for = out
        blocks = 1 << log
        there = jobs if all_there else rng.choice([0, 1, rng.randint(0, jobs), jobs, 2 * jobs])
        done = 0
        for c in range(clusters):
            both = shares(there, clusters, c, per, log, begin, owner, others)
            first, last = both & 0xFFFFFFFF, both >> 32
            assert first == done and begin[0] == 0 and begin[blocks] == (last - first) * per
            done = last
            sends = {r: [] for r in range(blocks)}
            for r in range(blocks):
                assert begin[r] <= begin[r + 1]
                if owner[r] >= 0:
                    o = owner[r]
                    job = begin[r] // per * per
                    assert begin[o] <= job < begin[o + 1] and 0 <= r - o - 1 < room_for
                    sends[o].append(r)
            for r in range(blocks):
                waits = [q for q in range(r + 1, r + 1 + others[r]) if begin[q] < begin[q + 1]]
                assert waits == sends[r]
        assert done == there
