"""Rules of the kernels on BF16 activations that no run shows: what a block may do only after
what, read in the kernel's source. Each is a short piece of it, found by name."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rank_residual_w4a4_b200", "csrc")


def source(name="twq_a16_sm100.cu"):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


def body(text, head):
    """The braces' contents after the first place that `head` matches."""
    at = text.index("{", re.search(head, text).end())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced braces")


def test_parts_of_peers_are_acquired_at_the_clusters_scope():
    """Peers' stores complete on this block's barrier with a release at the cluster's scope; a wait
    whose acquire is the block's own would not be ordered behind them."""
    text = source()
    waits = re.findall(r"(\w+)\(&s_recv, 0\)", text)
    assert waits and set(waits) == {"mbar_try_wait_cluster"}
    assert "acquire.cluster" in body(source("sm100_ptx.cuh"), r"bool mbar_try_wait_cluster\(")


def test_early_reads_do_not_come_from_l1():
    """ids and activations may be read before the kernel's own wait, on the ground that the kernel in
    front has waited for their writer. Visibility is promised at the wait alone; loads that are strong at
    the GPU's scope, and loads behind an acquire there, do not find an older line in an SM's L1."""
    text = source()
    assert "ld.relaxed.gpu.global" in body(text, r"ld4_early\(const void\* p\)")
    assert "ld.acquire.gpu.global" in body(text, r"acquire_early\(const uint16_t\* p\)")
    loads = re.findall(r"(\w+)\(ids \+", body(text, r"int make_chunks\("))
    assert loads and set(loads) == {"ld4_early"}
    kernel = body(text, r"a16_kernel\(const __grid_constant__ A16Args a\)")
    # the warps that load activations: wait or acquire, before the first load and on every way to it
    ready = re.search(r"if \(a\.x_ready\)\s*acquire_early\(a\.x\);\s*else\s*pdl_wait\(\);", kernel)
    assert ready and ready.end() < re.search(r"\bld16\(", kernel).start()
    # h, which the kernel in front writes, behind the wait
    assert kernel.index("if (!waited) pdl_wait();") < kernel.index("ld16(a.h")
    assert len(re.findall(r"\bld\d+\(", kernel)) == 2
