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
    the GPU's scope do not find an older line in an SM's L1."""
    text = source()
    for name in ("ld16_early", "ld4_early"):
        assert "ld.relaxed.gpu.global" in body(text, r"%s\(const \w+\* p\)" % name)
    loads = re.findall(r"(\w+)\(ids \+", body(text, r"int make_chunks\("))
    assert loads and set(loads) == {"ld4_early"}
    kernel = body(text, r"a16_kernel\(const __grid_constant__ A16Args a\)")
    load = body(kernel, r"auto load = \[&\]\(int n0\)")
    assert set(re.findall(r"\bld\d+\w*", load)) == {"ld16_early"}
    # h alone is read by plain loads, behind the wait
    rest = re.findall(r"\bld\d+\w*\(([^)]*)\)", kernel.replace(load, "").replace("ld16_early", "early"))
    assert rest and all("a.h" in r for r in rest)
    assert kernel.index("if (!waited) pdl_wait();") < kernel.index("ld16(a.h")
