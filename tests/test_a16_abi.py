"""The entry points on BF16 activations on the host: sizes, and every refusal before a launch."""
import ctypes

import pytest

from rank_residual_w4a4_b200 import _build, twq

A = 0x100000  # 16-byte aligned fake device address (never dereferenced on these paths)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return twq.load()


def weights(m=512, n=256, r=16, rq=A, sr=A, l1q=A, sl1=A, l2t=A):
    return twq._Weights(m, n, r, rq, sr, l1q, sl1, l2t)


def experts(count=4, up=None, down=None):
    return twq._Experts(count, up or weights(256, 1024, 16), down or weights(512, 256, 0))


def test_linear_refused(lib):
    def f(w=weights(), x=A, ldx=512, b=4, h=A, y=A):
        return lib.twq_fused_linear_a16(x, ldx, b, None if w is None else ctypes.byref(w), h, y, None)

    assert f(w=None) == 1 and f(x=None) == 1 and f(h=None) == 1 and f(y=None) == 1
    assert f(b=-1) == 1 and f(b=65) == 2 and f(ldx=504) == 1 and f(ldx=516) == 3
    for k in ("x", "h", "y"):
        assert f(**{k: A + 8}) == 3
    assert f(w=weights(m=500)) == 1 and f(w=weights(n=200)) == 1 and f(w=weights(m=0)) == 1
    assert f(w=weights(r=8)) == 1 and f(w=weights(r=272)) == 2 and f(w=weights(r=-16)) == 1
    assert f(w=weights(m=(1 << 20) + 128), ldx=1 << 21) == 2 and f(w=weights(n=(1 << 20) + 128)) == 2
    for k in ("rq", "sr", "l1q", "sl1", "l2t"):
        assert f(w=weights(**{k: None})) == 1 and f(w=weights(**{k: A + 8})) == 3
    assert f(b=0, x=None, h=None, y=None) == 0  # nothing to do


@pytest.mark.parametrize("name", ["twq_moe_route", "twq_moe_route_bf16"])
def test_route_refused(lib, name):
    def f(logits=A, ld=64, b=5, count=64, k=8, ids=A, w=A):
        return getattr(lib, name)(logits, ld, b, count, k, 1, ids, w, None)

    assert f(logits=None) == 1 and f(ids=None) == 1 and f(w=None) == 1
    assert f(b=-1) == 1 and f(b=(1 << 24) + 1) == 2
    assert f(count=0) == 1 and f(count=1025, ld=1025) == 2 and f(ld=63) == 1
    assert f(k=0) == 1 and f(k=17) == 2 and f(k=65) == 1 and f(count=4, k=5) == 1
    assert f(logits=A + 1) == 3 and f(ids=A + 2) == 3 and f(w=A + 1) == 3
    assert f(b=0, logits=None, ids=None, w=None) == 0


@pytest.mark.parametrize("name", ["twq_moe_experts", "twq_moe_layer", "twq_moe_layer_bf16"])
def test_experts_refused(lib, name):
    need = lib.twq_moe_workspace_bytes(4, 2, ctypes.byref(experts()))
    assert need >= 4 * 2 * (2 * 512 * 2 + 16 * 2)

    def f(e=experts(), x=A, ldx=256, b=4, ids=A, w=A, k=2, base=A, y=A, ws=A, nb=need, logits=A, ld=4):
        e = None if e is None else ctypes.byref(e)
        if name == "twq_moe_experts":
            return lib.twq_moe_experts(x, ldx, b, ids, w, k, e, base, y, ws, nb, None)
        return getattr(lib, name)(x, ldx, b, logits, ld, k, 1, e, base, ids, w, y, ws, nb, None)

    for k in ("x", "ids", "w", "y", "ws"):
        assert f(**{k: None}) == 1, k
    for k in ("x", "base", "y", "ws"):
        assert f(**{k: A + 8}) == 3, k
    assert f(ids=A + 2) == 3 and f(w=A + 2) == 3
    assert f(e=None) == 1 and f(nb=need - 1) == 1 and f(ldx=248) == 1 and f(ldx=260) == 3
    assert f(b=-1) == 1 and f(b=65, nb=1 << 30) == 2 and f(k=0) == 1 and f(k=17, nb=1 << 30) == 2
    assert f(e=experts(count=0)) == 1 and f(e=experts(count=1025), ld=1025) == 2
    assert f(e=experts(up=weights(256, 1152, 16))) == 1           # not twice the down product's rows
    assert f(e=experts(down=weights(512, 384, 0))) == 1           # not x's width
    assert f(e=experts(up=weights(256, 1000, 16))) == 1 and f(e=experts(up=weights(256, 1024, 8))) == 1
    assert f(e=experts(up=weights(256, 1024, 272))) == 2
    assert f(e=experts(up=weights(256, 1 << 21, 0), down=weights(1 << 20, 256, 0)), nb=1 << 40) == 2
    for k in ("rq", "sr", "l1q", "sl1", "l2t"):
        assert f(e=experts(up=weights(256, 1024, 16, **{k: None}))) == 1
        assert f(e=experts(up=weights(256, 1024, 16, **{k: A + 8}))) == 3
    for k in ("rq", "sr"):
        assert f(e=experts(down=weights(512, 256, 0, **{k: None}))) == 1
    if name != "twq_moe_experts":
        assert f(logits=None) == 1 and f(ld=3) == 1 and f(k=5, nb=1 << 30) == 1
        assert f(logits=A + 1) == 3
    assert f(b=0, x=None, ids=None, w=None, y=None, ws=None, nb=0, logits=None) == 0


@pytest.mark.parametrize("args", [(-1, 2, {}), (65, 2, {}), (4, 0, {}), (4, 17, {}), (4, 2, {"count": 0}),
                                  (4, 2, {"up": weights(256, 900, 0)})])
def test_workspace_of_a_refused_shape_is_zero(lib, args):
    b, k, e = args
    assert lib.twq_moe_workspace_bytes(b, k, ctypes.byref(experts(**e))) == 0


def test_stall_selftest_validation(lib):
    f = lib.twq_selftest_a16_stall
    assert f(-1) == 1 and f(999) == 1 and f(1000000001) == 1
    assert f(1000) == 0 and f(1000000000) == 0 and f(0) == 0


def test_launch_accounting(lib):
    assert twq.launches_per_call("twq_fused_linear_a16") == 2
    assert twq.launches_per_call("twq_moe_route") == 1 and twq.launches_per_call("twq_moe_experts") == 5
    assert twq.launches_per_call("twq_moe_layer") == 6 and twq.launches_per_call("twq_moe_layer_bf16") == 6


def test_binding_refuses_the_host(lib):
    import torch
    with pytest.raises((ValueError, RuntimeError)):
        twq.moe_route(torch.zeros((2, 4)), 2)
    with pytest.raises(TypeError):
        twq.moe_route(torch.zeros(4), 2)
    with pytest.raises(ValueError):
        twq.Experts.empty(2, 256, 128, 0, "cpu")
