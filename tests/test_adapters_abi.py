"""The adapter entry points on the host: sizes, and every refusal before a launch."""
import ctypes

import pytest
import torch

from rank_residual_w4a4_b200 import _build, twq

A = 0x100000  # 16-byte aligned fake device address (never dereferenced on these paths)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return twq.load()


def groups(b=40, count=3, order=A, offsets=A, tiles=A):
    return ctypes.byref(twq._RowGroups(b, count, order, offsets, tiles))


def adapters(m=512, n=256, r=16, count=3, a=A, b=A, scale=A):
    return ctypes.byref(twq._Adapters(m, n, r, count, a, b, scale))


@pytest.mark.parametrize("b,count,want", [(-1, 1, 1), (1, 0, 1), ((1 << 20) + 1, 1, 2), (1, 4097, 2)])
def test_group_sizes_refused(lib, b, count, want):
    arr = (ctypes.c_size_t * 3)()
    assert lib.twq_row_groups_sizes(b, count, arr) == want
    assert lib.twq_group_rows(A, groups(b, count), None) == want


@pytest.mark.parametrize("b,count", [(0, 1), (1, 1), (5, 4096), (1000, 7), (1 << 20, 4096)])
def test_group_sizes_hold_every_tile(lib, b, count):
    """The tile lists have room for the worst split: every key has rows, all but one of
    them one row only."""
    arr = (ctypes.c_size_t * 3)()
    assert lib.twq_row_groups_sizes(b, count, arr) == 0
    assert arr[0] == 4 * b and arr[1] == 4 * (count + 1)
    need = 1
    for rows in (16, 128):
        if rows == 16 and b > 768:  # no forward pass takes the small tiles then
            continue
        keys = min(b, count + 1)
        need += (keys - 1) + -(-(b - keys + 1) // rows) if b else 0
    assert arr[2] >= 16 * need
    assert lib.twq_row_groups_sizes(1, 1, None) == 1


def test_group_rows_refused(lib):
    f = lib.twq_group_rows
    assert f(A, None, None) == 1
    assert f(None, groups(), None) == 1
    assert f(A, groups(order=None), None) == 1
    assert f(A, groups(offsets=None), None) == 1
    assert f(A, groups(tiles=None), None) == 1
    assert f(A + 2, groups(), None) == 3
    for k in ("order", "offsets", "tiles"):
        assert f(A, groups(**{k: A + 4}), None) == 3


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_linear_refused(lib, codes):
    def f(ad=adapters(), g=groups(), b=40, x=A, x2=None, base=A, h=A, y=A):
        if codes:
            return lib.twq_adapter_linear_i8(x, A if x2 is None else x2, b, ad, g, base, h, y, None)
        return lib.twq_adapter_linear(x, 512 if x2 is None else x2, b, ad, g, base, h, y, None)

    assert f(ad=None) == 1 and f(g=None) == 1
    assert f(x=None) == 1 and f(h=None) == 1 and f(y=None) == 1
    assert f(x=A + 8) == 3 and f(h=A + 8) == 3 and f(y=A + 2) == 3 and f(base=A + 4) == 3
    if codes:
        assert f(x2=0) == 1 and f(x2=A + 4) == 3
    else:
        assert f(x2=504) == 1 and f(x2=516) == 3     # row stride below m; breaks 16 bytes
    assert f(ad=adapters(m=500)) == 1 and f(ad=adapters(n=200)) == 1 and f(ad=adapters(m=0)) == 1
    assert f(ad=adapters(r=12)) == 1 and f(ad=adapters(r=0)) == 1 and f(ad=adapters(r=-8)) == 1
    assert f(ad=adapters(r=136)) == 2 and f(ad=adapters(n=(1 << 20) + 128)) == 2
    assert f(ad=adapters(count=0)) == 1 and f(ad=adapters(count=4097)) == 2
    for k in ("a", "b", "scale"):
        assert f(ad=adapters(**{k: None})) == 1 and f(ad=adapters(**{k: A + 8})) == 3
    for k in ("order", "offsets", "tiles"):
        assert f(g=groups(**{k: None})) == 1 and f(g=groups(**{k: A + 8})) == 3
    assert f(g=groups(b=39)) == 1 and f(g=groups(count=2)) == 1   # another batch's grouping
    assert f(b=-1, g=groups(b=-1)) == 1 and f(b=(1 << 20) + 1, g=groups(b=(1 << 20) + 1)) == 2
    assert f(b=0, g=groups(b=0), x=None, h=None, y=None) == 0     # nothing to do


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_backward_refused(lib, codes):
    need = lib.twq_adapter_backward_workspace_bytes(40, 512, 256, 16, 3)
    assert need > 0

    def f(ad=adapters(), g=groups(), b=40, dy=A, x=A, x2=None, h=A, base=A, dx=A, da=A, db=A, ws=A,
          nb=need):
        if codes:
            return lib.twq_adapter_backward_i8(dy, x, A if x2 is None else x2, h, b, ad, g, base, dx,
                                               da, db, ws, nb, None)
        return lib.twq_adapter_backward(dy, x, 512 if x2 is None else x2, h, b, ad, g, base, dx, da,
                                        db, ws, nb, None)

    for k in ("dy", "x", "h", "dx", "da", "db", "ws"):
        assert f(**{k: None}) == 1, k
        assert f(**{k: A + 8}) == 3, k
    assert f(base=A + 4) == 3 and f(nb=need - 1) == 1
    assert f(ad=adapters(r=136)) == 2 and f(ad=adapters(m=100)) == 1
    assert f(g=groups(b=41)) == 1 and f(g=groups(count=4)) == 1
    if codes:
        assert f(x2=0) == 1
    else:
        assert f(x2=256) == 1 and f(x2=520 + 4) == 3


@pytest.mark.parametrize("args", [(-1, 128, 128, 8, 1), (1, 100, 128, 8, 1), (1, 128, 128, 136, 1),
                                  (1, 128, 128, 8, 0), (1 << 21, 128, 128, 8, 1)])
def test_workspace_of_a_refused_shape_is_zero(lib, args):
    assert lib.twq_adapter_backward_workspace_bytes(*args) == 0


def test_launch_accounting(lib):
    assert twq.launches_per_call("twq_group_rows") == 1
    for ep in ("twq_adapter_linear", "twq_adapter_backward"):
        assert twq.launches_per_call(ep) == twq.launches_per_call(ep + "_i8") >= 1


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(ValueError):
        twq.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(TypeError):
        twq.group_rows([0, 1], 2)
    bf = torch.bfloat16
    with pytest.raises(ValueError):
        twq.Adapters(torch.zeros(1, 8, 128, dtype=bf), torch.zeros(1, 128, 8, dtype=bf), torch.zeros(1))


def test_buffers_come_from_the_stream_of_the_call(lib, monkeypatch):
    """With stream=s, what a call allocates is s's memory (a block freed on the caller's stream
    may have work queued there that s does not wait for) and is kept for the caller's stream,
    which reads it next. On the host: streams and tensors are stand-ins."""
    import contextlib
    from types import SimpleNamespace

    now, made = ["caller"], []

    class Buffer:
        def __init__(self, shape, device):
            self.shape, self.device, self.home, self.kept = shape, device, now[0], []
            made.append(self)

        def record_stream(self, stream):
            self.kept.append(stream)

        def data_ptr(self):
            return A

        def numel(self):
            return 1 << 20

    @contextlib.contextmanager
    def on(stream):
        now[0], back = stream, now[0]
        yield
        now[0] = back

    ok = lambda *args: 0
    monkeypatch.setattr(twq, "_lib", SimpleNamespace(
        twq_row_groups_sizes=lib.twq_row_groups_sizes, twq_group_rows=ok, twq_adapter_linear=ok,
        twq_adapter_backward=ok, twq_adapter_backward_workspace_bytes=lambda *args: 64))
    monkeypatch.setattr(twq, "_on", lambda device, stream: (0, None))
    monkeypatch.setattr(twq, "_mat", lambda *args: A)
    monkeypatch.setattr(twq, "_dev", lambda *args: A)
    monkeypatch.setattr(twq, "_strided_x", lambda *args: (A, 256))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: now[0])
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: Buffer(shape, device))
    monkeypatch.setattr(torch, "empty_like", lambda t: Buffer(t.shape, "gpu"))
    ad = SimpleNamespace(m=256, n=128, r=8, count=2, device="gpu", _ref=None, a=Buffer((2, 8, 256), "gpu"),
                         b=Buffer((2, 128, 8), "gpu"))
    ids = torch.zeros(5, dtype=torch.int32)
    for stream, home in ((None, "caller"), ("s", "s")):
        del made[:]
        groups = twq.group_rows(ids, 2, stream=stream)
        y, h = twq.adapter_linear(None, ad, SimpleNamespace(b=5, count=2, device="gpu", _ref=None),
                                  stream=stream)
        grads = twq.adapter_backward(None, None, None, ad,
                                     SimpleNamespace(b=5, count=2, device="gpu", _ref=None), stream=stream)
        assert [t.shape for t in (y, h, *grads)] == [(5, 128), (5, 8), (5, 256), (2, 8, 256), (2, 128, 8)]
        assert len(made) == 7 and groups._buf in made
        assert all(t.home == home for t in made)
        assert all(t.kept == ([] if stream is None else ["caller"]) for t in made)


def test_binding_imports_with_a_torch_without_cuda(monkeypatch):
    """Such a torch lacks the private call that tells the current stream; the host-side checks
    still run there."""
    import importlib.util
    import sys
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("rank_residual_w4a4_b200.twq_again", twq.__file__)
    module = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, module)  # dataclasses look their module up
    spec.loader.exec_module(module)
    with pytest.raises(ValueError):
        module.group_rows(torch.zeros(4, dtype=torch.int32), 2)


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_empty_batch_needs_no_order(lib, codes):
    """The order of an empty batch has 0 bytes, so it may be null, as twq_group_rows takes it."""
    arr = (ctypes.c_size_t * 3)()
    assert lib.twq_row_groups_sizes(0, 3, arr) == 0 and arr[0] == 0
    empty = groups(b=0, order=None)
    if codes:
        assert lib.twq_adapter_linear_i8(None, None, 0, adapters(), empty, None, None, None, None) == 0
    else:
        assert lib.twq_adapter_linear(None, 512, 0, adapters(), empty, None, None, None, None) == 0
    assert lib.twq_adapter_linear(A, 512, 0, adapters(), groups(b=0, offsets=None), None, A, A, None) == 1
    # the gradients of an empty batch are zeros that are written: refused for what it lacks alone
    need = lib.twq_adapter_backward_workspace_bytes(0, 512, 256, 16, 3)
    args = (None, None, None, None, 0) if codes else (None, None, 512, None, 0)
    f = lib.twq_adapter_backward_i8 if codes else lib.twq_adapter_backward
    assert f(*args, adapters(), empty, None, None, None, A, A, need, None) == 1       # da
    assert f(*args, adapters(), empty, None, None, A, A, A + 8, need, None) == 3      # workspace


@pytest.mark.parametrize("b,count", [(0, 4), (1, 1), (768, 1), (768, 4096), (769, 48), (769, 49),
                                     (1536, 95), (1536, 96), (1536, 4096), (1537, 97), (1537, 4096),
                                     (70001, 4096)])
def test_group_sizes_hold_both_lists_and_the_tiles_before(lib, b, count):
    """Room for the worst split in both tile lists, for a count of their tiles and for count + 1
    integers behind them. The 16-row list is there where some rank's forward pass takes it: up to
    768 rows, and up to 1536 where the adapters may have 16 rows or fewer each."""
    arr = (ctypes.c_size_t * 3)()
    assert lib.twq_row_groups_sizes(b, count, arr) == 0
    entries = 1
    for rows in (16, 128):
        if rows == 16 and not (b <= 768 or (b <= 1536 and b <= 16 * count)):
            continue
        keys = min(b, count + 1)  # all of them with rows, all but one with one row only
        entries += (keys - 1) + -(-(b - keys + 1) // rows) if b else 0
    assert arr[2] >= 16 * entries + 4 * (count + 1)


def test_stall_selftest_validation(lib):
    f = lib.twq_selftest_adapter_stall
    assert f(-1) == 1 and f(999) == 1 and f(1000000001) == 1
    assert f(1000) == 0 and f(1000000000) == 0 and f(0) == 0
