"""Run as a program, without torch: adapter and layer calls, a cudaDeviceReset, twq_release_cache,
and the same calls on new buffers. Exits 0 if every call succeeds and the outputs are equal."""
import ctypes
import importlib.util
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I = ctypes.c_void_p, ctypes.c_int64


class Groups(ctypes.Structure):
    _fields_ = [("b", I), ("count", I), ("order", P), ("offsets", P), ("tiles", P)]


class Weights(ctypes.Structure):
    _fields_ = [("m", I), ("n", I), ("r", I), ("rq", P), ("sr", P), ("l1q", P), ("sl1", P), ("l2t", P)]


class Adapters(ctypes.Structure):
    _fields_ = [("m", I), ("n", I), ("r", I), ("count", I), ("a", P), ("b", P), ("scale", P)]


def cudart():
    spec = importlib.util.find_spec("nvidia.cuda_runtime")
    dirs = [os.path.join(d, "lib") for d in spec.submodule_search_locations] if spec else []
    for d in dirs + ["/usr/local/cuda/lib64"]:
        path = os.path.join(d, "libcudart.so.12")
        if os.path.exists(path):
            return ctypes.CDLL(path)
    raise OSError("libcudart.so.12 not found")


def alloc_on(rt):
    def alloc(nbytes, byte=0):
        p = P()
        assert rt.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(max(nbytes, 256))) == 0
        assert rt.cudaMemset(p, byte, ctypes.c_size_t(max(nbytes, 256))) == 0
        return p.value
    return alloc


def fetch(rt, p, nbytes):
    host = ctypes.create_string_buffer(nbytes)
    assert rt.cudaMemcpy(host, P(p), ctypes.c_size_t(nbytes), 2) == 0
    return host.raw


def run_layer(rt, lib, b):
    m, n, r = 512, 512, 32
    alloc = alloc_on(rt)
    w = Weights(m, n, r, alloc(n * m // 2, 0x11), alloc(m // 128 * n * 4, 0x3c), alloc(r * m // 2, 0x11),
                alloc(m // 128 * r * 4, 0x3c), alloc(n * r * 2, 0x3c))
    y = alloc(b * n * 2)
    status = lib.twq_fused_linear(P(alloc(b * m // 2, 0x11)), P(alloc(b * m // 128 * 4, 0x3c)), I(b),
                                  ctypes.byref(w), P(y), None)
    assert status == 0, status
    out = fetch(rt, y, b * n * 2)
    assert any(out)
    return out


def run(rt, lib, b):
    m, n, r, count = 512, 256, 16, 2
    alloc = alloc_on(rt)
    sizes = (ctypes.c_size_t * 3)()
    assert lib.twq_row_groups_sizes(I(b), I(count), sizes) == 0
    g = Groups(b, count, *[alloc(s) for s in sizes])
    # every BF16 0x3c3c = 0.0115; every scale 0x3f3f3f3f = 0.747; every id 0
    ad = Adapters(m, n, r, count, alloc(count * r * m * 2, 0x3c), alloc(count * n * r * 2, 0x3c),
                  alloc(count * 4, 0x3f))
    x, h, y = alloc(b * m * 2, 0x3c), alloc(b * r * 2), alloc(b * n * 2)
    dx, da, db = alloc(b * m * 2), alloc(count * r * m * 2), alloc(count * n * r * 2)
    lib.twq_adapter_backward_workspace_bytes.restype = ctypes.c_size_t
    need = lib.twq_adapter_backward_workspace_bytes(I(b), I(m), I(n), I(r), I(count))
    ws = alloc(need)
    status = [
        lib.twq_group_rows(P(alloc(b * 4)), ctypes.byref(g), None),
        lib.twq_adapter_linear(P(x), I(m), I(b), ctypes.byref(ad), ctypes.byref(g), None, P(h), P(y), None),
        lib.twq_adapter_backward(P(y), P(x), I(m), P(h), I(b), ctypes.byref(ad), ctypes.byref(g), None, P(dx),
                                 P(da), P(db), P(ws), ctypes.c_size_t(need), None),
    ]
    assert status == [0, 0, 0], status
    assert rt.cudaDeviceSynchronize() == 0
    out = [fetch(rt, p, nbytes) for p, nbytes in ((y, b * n * 2), (dx, b * m * 2), (da, count * r * m * 2),
                                                  (db, count * n * r * 2))]
    assert any(out[0])
    return out


def main():
    rt = cudart()
    lib = ctypes.CDLL(os.path.join(ROOT, "rank_residual_w4a4_b200", "libtwq.so"))

    def calls():
        return [run(rt, lib, b) for b in (40, 2000)] + [run_layer(rt, lib, b) for b in (4, 300)]

    before = calls()
    assert rt.cudaDeviceReset() == 0
    lib.twq_release_cache()
    assert calls() == before


if __name__ == "__main__":
    sys.exit(main())
