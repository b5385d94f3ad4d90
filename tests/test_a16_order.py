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


def test_no_block_leaves_before_its_peers_have_sent():
    """A peer's own waits may end later than any limit of the block that gets its part. So past the
    limit the block meets all others at the cluster's barrier, at which each arrives after its
    sending, and only then gives up."""
    text = source()
    wait = body(text, r"auto wait_parts = \[&\]")
    arrive, meet = wait.index("cluster_arrive_relaxed"), wait.index("cluster_wait_acquire")
    assert arrive < meet < wait.index("g_a16_status")
    # one arrival of every thread where the cluster starts, one after the roles, each round waited for
    # before the next: by the products ahead of their steps, by the others at the end
    kernel = body(text, r"a16_kernel\(const __grid_constant__ A16Args a\)")
    end = kernel[kernel.rindex("if (split > 1)"):]
    assert re.search(r"if \(warp >= kWarps\) cluster_wait_acquire\(\);\s*cluster_arrive_relaxed\(\);", end)
    products = kernel.index("float acc[2][NT][4]")
    first = kernel.index("if (split > 1) cluster_wait_acquire();")
    assert products < first < kernel.index("for (int v = lo; v < hi;)", products)
    assert "cluster_wait" not in body(kernel, r"auto send_part = \[&\]\(int rows\)")


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
