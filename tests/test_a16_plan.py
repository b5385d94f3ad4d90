"""How the host divides a launch on BF16 activations, checked on the CPU.

Clusters of blocks take equal numbers of jobs, and a cluster's blocks equal shares of their jobs'
steps, one job after the other. A block that ends a job which an earlier one began sends its part
there, to the (its rank - the owner's - 1)-th place of a buffer of `parts` places; the owner waits for
exactly the parts that are sent. Every block's walk is repeated here as the kernel makes it, for jobs
that the host knows and for such as only the GPU knows (the experts that were chosen), from none to
more than were planned for.
"""
import ctypes
import hashlib
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_residual_w4a4_b200", "csrc")
HARNESS = os.path.join(ROOT, "tests", "a16_plan_harness.cu")
DEPS = [HARNESS] + [os.path.join(CSRC, f) for f in
                    ("twq_a16_sm100.cu", "sm100_ptx.cuh", "twq_a16.h", "twq_adapter.h",
                     "twq_internal.h")] + [os.path.join(ROOT, "include", "twq.h")]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


@pytest.fixture(scope="module")
def plan():
    h = hashlib.sha256()
    for d in DEPS:
        with open(d, "rb") as fh:
            h.update(fh.read())
    out_dir = os.path.join(ROOT, "tests", "_build")
    os.makedirs(out_dir, exist_ok=True)
    path = os.path.join(out_dir, "liba16plan_%s.so" % h.hexdigest()[:16])
    if not os.path.exists(path):
        # PTX only for the device side: the harness runs host code alone. Launches are not called;
        # what they call in other files may stay unresolved.
        cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=compute_100a", "-std=c++17", "-O1",
               "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
               HARNESS, "-o", path + ".tmp"]
        try:
            subprocess.run(cmd, check=True, capture_output=True, timeout=900)
        except FileNotFoundError:
            pytest.skip("nvcc is not available")
        os.replace(path + ".tmp", path)
    fn = ctypes.CDLL(path, mode=os.RTLD_LAZY).twq_test_a16_plan
    I, L = ctypes.c_int, ctypes.c_int64
    fn.argtypes = [L, L, ctypes.POINTER(I), I, I, I, I, ctypes.POINTER(L)]

    def call(jobs, steps, room, per_sm, warps, all_there, most):
        out = (L * 4)()
        assert fn(jobs, steps, (I * 4)(*room), per_sm, warps, all_there, most, out) == 0
        return tuple(out)
    return call


def walk(jobs, steps, clusters, split_log, parts):
    """The steps of the busiest block; fails where the blocks' walks do not fit together."""
    blocks, busiest, seen = 1 << split_log, 0, 0
    each, more = divmod(jobs, clusters)
    for c in range(clusters):
        first = each * c + min(c, more)
        last = first + each + (c < more)
        assert first == seen
        seen = last
        total = (last - first) * steps
        begin = [total * r >> split_log for r in range(blocks + 1)]
        assert begin[0] == 0 and begin[-1] == total
        sent = {r: set() for r in range(blocks)}
        for r in range(blocks):
            lo, hi = begin[r], begin[r + 1]
            busiest = max(busiest, hi - lo)
            if lo < hi and lo % steps:  # goes on with a job of an earlier block's
                owner = r - 1
                while begin[owner] > lo - lo % steps:
                    owner -= 1
                assert begin[owner] < begin[owner + 1] and 0 <= r - owner - 1 < parts
                sent[owner].add(r - owner - 1)
        for r in range(blocks):
            lo, hi = begin[r], begin[r + 1]
            rest = hi % steps if lo < hi else 0
            awaited = set()
            if rest and hi - rest >= lo:  # begins a job that others go on with
                q = r + 1
                while q < blocks and begin[q] < hi - rest + steps:
                    if begin[q] < begin[q + 1]:
                        awaited.add(q - r - 1)
                    q += 1
            assert awaited == sent[r]
    assert seen == jobs
    return busiest


ROOMS = {1: (148, 74, 36, 15), 2: (296, 148, 71, 33), 3: (444, 222, 107, 48)}


@pytest.mark.parametrize("all_there", [True, False])
@pytest.mark.parametrize("per_sm", [1, 2, 3])
def test_blocks_fit_together(plan, per_sm, all_there):
    rng = random.Random(100 * per_sm + all_there)
    for _ in range(3000):
        jobs = int(rng.choice([1, 1, 2, 3, 5, 10, 40, 150, 500, 2000]) * rng.uniform(1, 2))
        steps = rng.choice([1, 2, 3, rng.randint(1, 60)])
        warps, most = rng.choice([4, 8]), rng.choice([3, 3, 3, 2, 1, 0])
        clusters, split_log, parts, mine = plan(jobs, steps, ROOMS[per_sm], per_sm, warps, all_there, most)
        assert 1 <= clusters <= jobs and clusters <= ROOMS[per_sm][split_log] and split_log <= most
        assert walk(jobs, steps, clusters, split_log, parts) <= mine
        if not all_there:
            for there in (0, 1, rng.randint(0, jobs), rng.randint(jobs, 2 * jobs)):
                walk(there, steps, clusters, split_log, parts)
