"""The adapter operators on the GPU against their definition in 64 bits (adapter_ref.py):
rows grouped by adapter, adapters beside the layer on BF16 X and on codes, and their
gradients; then the ways a program calls them (strided X, in place, another stream,
captured and replayed, beside the layer itself)."""
import pytest
import torch

import adapter_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def twq(device):
    from rank_residual_w4a4_b200 import _build, twq as binding
    _build.build()
    binding.load()
    return binding


def make_ids(b, count, kind, gen):
    if kind == "none":
        return torch.full((b,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((b,), count - 1, dtype=torch.int32)
    ids = torch.randint(-1, count, (b,), generator=gen, dtype=torch.int32)
    if kind == "runs":
        ids = ids.sort().values
    if kind == "wild":  # ids far outside the range mean no adapter
        ids[::3] = count
        ids[1::5] = 2 ** 31 - 1
        ids[2::7] = -2 ** 31
    return ids


@pytest.mark.parametrize("b,count,kind", [
    (0, 3, "mixed"), (1, 1, "one"), (1, 5, "none"), (31, 2, "mixed"), (33, 40, "wild"),
    (1000, 1, "one"), (1023, 7, "runs"), (4097, 1024, "mixed"), (5000, 4096, "mixed"),
    (16384, 64, "runs"), (65535, 33, "mixed"), (65536, 2, "one"), (70001, 4096, "wild"),
])
def test_group_rows(twq, device, b, count, kind):
    gen = torch.Generator().manual_seed(b + count)
    ids = make_ids(b, count, kind, gen)
    g = twq.group_rows(ids.to(device), count)
    key = torch.where((ids < 0) | (ids >= count), count, ids).long()
    order = torch.sort(key, stable=True).indices.int()
    hist = torch.bincount(key, minlength=count + 1)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), hist.cumsum(0)])[:count + 1].int()
    assert torch.equal(g.order.cpu(), order)
    assert torch.equal(g.offsets.cpu(), offsets)
    # the same buffers again, with other ids
    ids2 = ids.flip(0).contiguous()
    g2 = twq.group_rows(ids2.to(device), count, groups=g)
    assert g2 is g
    key2 = key.flip(0)
    assert torch.equal(g.order.cpu(), torch.sort(key2, stable=True).indices.int())


class Case:
    def __init__(self, twq, device, b, m, n, r, count, kind, codes, seed=0):
        gen = torch.Generator().manual_seed(seed + b + 7 * r)
        self.codes, self.b = codes, b

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16).to(device)

        self.ids = make_ids(b, count, kind, gen)
        x = normal(b, m)
        x[:, ::100] *= 30
        self.x, self.dy, self.h = x, normal(b, n, std=0.01), normal(b, r)
        self.base, self.dx_base = normal(b, n, std=3.0), normal(b, m, std=0.01)
        self.ad = twq.Adapters(normal(count, r, m, std=m ** -0.5), normal(count, n, r, std=0.05),
                               (torch.rand(count, generator=gen) * 4 - 2).to(device))
        self.groups = twq.group_rows(self.ids.to(device), count)
        if codes:
            self.xargs = twq.quantize_act_a8(x) if b else (
                torch.empty((0, m), dtype=torch.int8, device=device),
                torch.empty((0, m // 128), dtype=torch.float32, device=device))
            self.x64 = ref.x_of_codes(*self.xargs)
            self.linear, self.backward = twq.adapter_linear_i8, twq.adapter_backward_i8
        else:
            self.xargs, self.x64 = (x,), x.double()
            self.linear, self.backward = twq.adapter_linear, twq.adapter_backward

    def ref_linear(self, base):
        ad = self.ad
        return ref.linear(self.x64, ad.a, ad.b, ad.scale, self.ids.to(ad.device),
                          None if base is None else base.double(), self.codes)

    def ref_backward(self, dx_base):
        ad = self.ad
        return ref.backward(self.dy.double(), self.x64, self.h.double(), ad.a, ad.b, ad.scale,
                            self.ids.to(ad.device), None if dx_base is None else dx_base.double(),
                            self.codes)

    def check_linear(self, base, got):
        for g, w, e, name in zip(got, *self.ref_linear(base), ("y", "h")):
            ref.check(g, w, e, name)

    def check_backward(self, dx_base, got):
        for g, w, e, name in zip(got, *self.ref_backward(dx_base), ("dx", "da", "db")):
            ref.check(g, w, e, name)


# b, m, n, r, count, kind: one row to many, around the tile sizes, ranks that are no
# multiple of 16 or 32, no adapter at all, adapters without rows, uneven shapes
SHAPES = [
    (1, 128, 128, 8, 1, "one"), (1, 4096, 256, 16, 8, "one"), (2, 256, 128, 8, 3, "none"),
    (15, 512, 384, 24, 4, "mixed"), (16, 512, 512, 16, 1, "one"), (17, 640, 256, 40, 2, "one"),
    (64, 1024, 1152, 56, 64, "mixed"), (127, 256, 640, 128, 2, "runs"),
    (128, 384, 256, 64, 1, "one"), (129, 384, 256, 120, 1, "one"), (300, 1152, 896, 32, 5, "wild"),
    (333, 128, 128, 96, 3, "mixed"), (1000, 512, 768, 72, 17, "mixed"),
    (1500, 256, 1024, 16, 300, "mixed"), (2500, 768, 512, 128, 2, "runs"),
    (5000, 256, 256, 48, 1, "one"), (700, 4096, 128, 112, 1, "runs"),
    (1536, 512, 384, 16, 96, "mixed"), (1537, 512, 384, 16, 97, "runs"), (1500, 384, 512, 8, 93, "mixed"),
]


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_linear(twq, device, b, m, n, r, count, kind, codes):
    c = Case(twq, device, b, m, n, r, count, kind, codes)
    c.check_linear(c.base, c.linear(*c.xargs, c.ad, c.groups, base=c.base))
    c.check_linear(None, c.linear(*c.xargs, c.ad, c.groups))
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("b,m,n,r,count,kind", SHAPES)
def test_backward(twq, device, b, m, n, r, count, kind, codes):
    c = Case(twq, device, b, m, n, r, count, kind, codes)
    first = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    c.check_backward(c.dx_base, first)
    c.check_backward(None, c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups))
    again = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    assert all(torch.equal(p, q) for p, q in zip(first, again))  # equal calls, equal bits
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
def test_no_rows(twq, device, codes):
    c = Case(twq, device, 0, 256, 128, 16, 2, "mixed", codes)
    y, h = c.linear(*c.xargs, c.ad, c.groups, base=c.base)
    assert y.shape == (0, 128) and h.shape == (0, 16)
    dx, da, db = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups)
    assert dx.shape == (0, 256) and not da.any() and not db.any()


@pytest.mark.parametrize("b", [5, 40, 300, 2000])
def test_rows_without_adapter_and_bad_values_stay_apart(twq, device, b):
    """Rows without adapter are base bit for bit, whatever their X holds; an infinity or
    NaN in a row with an adapter reaches that row's y and no other."""
    c = Case(twq, device, b, 512, 256, 16, 3, "mixed", False)
    c.ids[0], c.ids[1], c.ids[b - 1] = -1, 1, 7
    c.groups = twq.group_rows(c.ids.to(device), 3)
    y0, h0 = twq.adapter_linear(c.x, c.ad, c.groups, base=c.base)
    bad = c.x.clone()
    bad[0], bad[b - 1] = float("nan"), float("inf")
    bad[1, 3] = float("nan")
    y, h = twq.adapter_linear(bad, c.ad, c.groups, base=c.base)
    out = (c.ids < 0) | (c.ids >= 3)
    assert torch.equal(y[out.to(device)], c.base[out.to(device)]) and not h[out.to(device)].any()
    assert y[1].isnan().all() and h[1].isnan().all()
    keep = torch.ones(b, dtype=torch.bool, device=device)
    keep[1] = False
    assert torch.equal(y[keep], y0[keep]) and torch.equal(h[keep], h0[keep])
    # gradients: a row without adapter takes no part
    dy = c.dy.clone()
    want = twq.adapter_backward(dy, c.x, c.h, c.ad, c.groups, dx_base=c.dx_base)
    bad = c.x.clone()
    bad[0] = float("nan")
    dy[0] = float("inf")
    hb = c.h.clone()
    hb[0] = float("nan")
    got = twq.adapter_backward(dy, bad, hb, c.ad, c.groups, dx_base=c.dx_base)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("b", [3, 200, 900])
def test_rows_are_independent_of_the_batch(twq, device, b):
    """A row's y does not depend on the order of the ids of the others."""
    c = Case(twq, device, b, 384, 256, 24, 4, "mixed", False)
    y, h = twq.adapter_linear(c.x, c.ad, c.groups, base=c.base)
    p = torch.randperm(b, generator=torch.Generator().manual_seed(1)).to(device)
    g = twq.group_rows(c.ids.to(device)[p].contiguous(), 4)
    yp, hp = twq.adapter_linear(c.x[p].contiguous(), c.ad, g, base=c.base[p].contiguous())
    assert torch.equal(yp, y[p]) and torch.equal(hp, h[p])


@pytest.mark.parametrize("b", [1, 9, 257])
def test_strided_x_and_in_place(twq, device, b):
    c = Case(twq, device, b, 256, 384, 16, 2, "mixed", False)
    wide = torch.full((b, 256 + 72), float("nan"), dtype=torch.bfloat16, device=device)
    wide[:, 64:320] = c.x
    xs = wide[:, 64:320]
    y, h = twq.adapter_linear(c.x, c.ad, c.groups, base=c.base)
    ys, hs = twq.adapter_linear(xs, c.ad, c.groups, base=c.base)
    assert torch.equal(y, ys) and torch.equal(h, hs)
    inplace = c.base.clone()
    yi, _ = twq.adapter_linear(xs, c.ad, c.groups, base=inplace, y=inplace)
    assert yi.data_ptr() == inplace.data_ptr() and torch.equal(y, inplace)
    want = twq.adapter_backward(c.dy, c.x, c.h, c.ad, c.groups, dx_base=c.dx_base)
    dx = c.dx_base.clone()
    got = twq.adapter_backward(c.dy, xs, c.h, c.ad, c.groups, dx_base=dx, dx=dx)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("b", [24, 700])
def test_stays_inside_its_buffers(twq, device, b):
    """Words around every output and the workspace keep their values."""
    c = Case(twq, device, b, 256, 384, 24, 3, "mixed", False)

    def guarded(*shape):
        n = 1
        for s in shape:
            n *= s
        buf = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=device)
        return buf, buf[256:256 + n].view(shape)

    nbytes = twq.adapter_backward_workspace_bytes(b, 256, 384, 24, 3)
    wsb = torch.full((nbytes + 512,), 9, dtype=torch.uint8, device=device)
    outs = [guarded(b, 384), guarded(b, 24), guarded(b, 256), guarded(3, 24, 256), guarded(3, 384, 24)]
    (_, y), (_, h), (_, dx), (_, da), (_, db) = outs
    twq.adapter_linear(c.x, c.ad, c.groups, base=c.base, y=y, h=h)
    twq.adapter_backward(c.dy, c.x, c.h, c.ad, c.groups, dx=dx, da=da, db=db,
                         workspace=wsb[256:256 + nbytes])
    for buf, _ in outs:
        assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())
    assert bool((wsb[:256] == 9).all()) and bool((wsb[-256:] == 9).all())


@pytest.mark.parametrize("b", [8, 600])
def test_other_stream_and_graph(twq, device, b):
    c = Case(twq, device, b, 512, 256, 16, 3, "mixed", False)
    want = twq.adapter_linear(c.x, c.ad, c.groups, base=c.base)
    wantb = twq.adapter_backward(c.dy, c.x, c.h, c.ad, c.groups, dx_base=c.dx_base)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = twq.adapter_linear(c.x, c.ad, c.groups, base=c.base, stream=s)
    gotb = twq.adapter_backward(c.dy, c.x, c.h, c.ad, c.groups, dx_base=c.dx_base, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(p, q) for p, q in zip(got + gotb, want + wantb))
    # captured once with the grouping inside, replayed for other ids and other values
    ids = c.ids.to(device)
    x, base, dy = c.x.clone(), c.base.clone(), c.dy.clone()
    g = twq.group_rows(ids, 3)
    ws = torch.empty(twq.adapter_backward_workspace_bytes(b, 512, 256, 16, 3), dtype=torch.uint8,
                     device=device)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twq.group_rows(ids, 3, groups=g)
        y, h = twq.adapter_linear(x, c.ad, g, base=base)
        grads = twq.adapter_backward(dy, x, h, c.ad, g, workspace=ws)
    for seed in (5, 6):
        d = Case(twq, device, b, 512, 256, 16, 3, "mixed", False, seed=seed)
        ids.copy_(d.ids), x.copy_(d.x), base.copy_(d.base), dy.copy_(d.dy)
        graph.replay()
        g2 = twq.group_rows(d.ids.to(device), 3)
        y2, h2 = twq.adapter_linear(d.x, c.ad, g2, base=d.base)
        grads2 = twq.adapter_backward(d.dy, d.x, h2, c.ad, g2)
        assert torch.equal(y, y2) and torch.equal(h, h2)
        assert all(torch.equal(p, q) for p, q in zip(grads, grads2))


def test_two_streams_at_once(twq, device):
    cases = [Case(twq, device, 900, 512, 512, 32, 3, "mixed", False, seed=s) for s in (1, 2)]
    want = [c.linear(*c.xargs, c.ad, c.groups, base=c.base)
            + c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [None, None]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i] = (c.linear(*c.xargs, c.ad, c.groups, base=c.base)
                          + c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(g, w))


@pytest.mark.parametrize("b", [12, 260])
def test_beside_the_layer(twq, device, b):
    """A W4A8 layer with adapters, forward and backward, as a program runs it: the layer's
    codes are quantized once and serve the layer, the adapters and, kept, the gradients."""
    c = Case(twq, device, b, 512, 256, 16, 3, "mixed", True)
    gen = torch.Generator().manual_seed(3)
    bf = torch.bfloat16
    w = twq.pack_weights((torch.randn(512, 256, generator=gen) * 0.02).to(bf).to(device),
                         (torch.randn(512, 32, generator=gen) * 0.05).to(bf).to(device),
                         (torch.randn(32, 256, generator=gen) * 0.05).to(bf).to(device))
    xq8, sx = twq.quantize_act_a8(c.x)
    layer = twq.fused_linear_a8(xq8, sx, w)
    base = layer.clone()
    y, h = twq.adapter_linear_i8(xq8, sx, c.ad, c.groups, base=layer, y=layer)
    c.check_linear(base, (y, h))
    c.h = h
    c.check_backward(c.dx_base, twq.adapter_backward_i8(c.dy, xq8, sx, h, c.ad, c.groups,
                                                        dx_base=c.dx_base))
    # the 4-bit codes one per byte go the same way
    q4, s4 = twq.quantize_act_i8(c.x)
    c.x64 = ref.x_of_codes(q4, s4)
    c.check_linear(None, twq.adapter_linear_i8(q4, s4, c.ad, c.groups))
    assert twq.device_status() == 0


@pytest.mark.parametrize("b", [20, 200])
def test_gradients_against_differences(twq, device, b):
    """y is linear in x, in A and in B, each for itself, so a difference of two forward
    passes over a step D is <dy, y(v + D) - y(v)> = <gradient, D> but for roundings:
    those of y (u |y| / sqrt(3) at most, independent) and h behind it (u |h| / sqrt(3)
    through B) in either pass, and of the gradient itself. Six standard deviations."""
    c = Case(twq, device, b, 256, 256, 16, 2, "one", False)
    ad, bf = c.ad, torch.bfloat16
    y0, h0 = twq.adapter_linear(c.x, ad, c.groups)
    dx, da, db = twq.adapter_backward(c.dy, c.x, h0, ad, c.groups)
    gen = torch.Generator().manual_seed(9)
    for grad, name in ((dx, "x"), (da, "a"), (db, "b")):
        at = {"x": c.x, "a": ad.a, "b": ad.b}
        v = at[name]
        moved = (v.float() + torch.randn(v.shape, generator=gen).to(device) * v.float().std()).to(bf)
        at[name] = moved
        ad1 = twq.Adapters(at["a"], at["b"], ad.scale)
        y1, h1 = twq.adapter_linear(at["x"], ad1, c.groups)
        step = moved.double() - v.double()
        left = (c.dy.double() * (y1.double() - y0.double())).sum().item()
        right = (grad.double() * step).sum().item()
        s = ad.scale.double()[-1].abs()
        through = (c.dy.double() @ at["b"][-1].double()) * s
        var = sum(((c.dy.double() * y.double()) ** 2).sum() + ((through * h.double()) ** 2).sum()
                  for y, h in ((y0, h0), (y1, h1))) + 2 * ((grad.double() * step) ** 2).sum()
        dev = ref.U / 3 ** 0.5 * var.sqrt().item()
        assert abs(left - right) <= 6 * dev, (name, left, right, dev)


@pytest.mark.parametrize("b,m,n,r,kind", [(1700, 512, 6400, 64, "runs"), (1300, 2048, 512, 16, "mixed"),
                                          (900, 512, 2048, 128, "runs")])
def test_many_calls_give_equal_bits(twq, device, b, m, n, r, kind):
    """Hundreds of calls in a row, whose warps meet at other times in each: no wait runs out
    and every call gives the first one's bits."""
    c = Case(twq, device, b, m, n, r, 4, kind, False)
    want = (c.linear(*c.xargs, c.ad, c.groups, base=c.base)
            + c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base))
    for _ in range(10):
        for _ in range(30):
            got = (c.linear(*c.xargs, c.ad, c.groups, base=c.base)
                   + c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base))
        assert twq.device_status() == 0
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("r", [8, 72])
@pytest.mark.parametrize("m,n", [(128, 131072), (131072, 128)])
def test_offsets_beyond_32_bits(twq, device, m, n, r, codes):
    """X, dY or Y of more than 2^31 elements: the rows at both ends and in the middle. The
    gradients of the weights are those of these rows, dY being 0 elsewhere."""
    b, count, bf = 17000, 2, torch.bfloat16
    gen = torch.Generator(device=device).manual_seed(r)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, dtype=bf, device=device) * std

    pick = torch.tensor([0, 1, b // 2, b - 2, b - 1], device=device)
    ids = torch.arange(b, dtype=torch.int32) % 3 - 1
    ids[b // 3:2 * b // 3] = 1  # tiles whose rows follow one another, too
    ids = ids.to(device)
    ad = twq.Adapters(normal(count, r, m, std=m ** -0.5), normal(count, n, r, std=0.05),
                      torch.tensor([0.5, -2.0], device=device))
    groups = twq.group_rows(ids, count)
    if codes:
        xargs = (torch.randint(-127, 128, (b, m), generator=gen, dtype=torch.int8, device=device),
                 torch.rand((b, m // 128), generator=gen, device=device) * 0.02)
        x64 = ref.x_of_codes(xargs[0][pick], xargs[1][pick])
        linear, backward = twq.adapter_linear_i8, twq.adapter_backward_i8
    else:
        xargs = (normal(b, m),)
        x64 = xargs[0][pick].double()
        linear, backward = twq.adapter_linear, twq.adapter_backward
    y = normal(b, n)
    base64 = y[pick].double()
    y, h = linear(*xargs, ad, groups, base=y, y=y)
    want = ref.linear(x64, ad.a, ad.b, ad.scale, ids[pick], base64, codes)
    for got, w, e, name in zip((y, h), *want, ("y", "h")):
        ref.check(got[pick], w, e, name)
    del y
    dy = torch.zeros((b, n), dtype=bf, device=device)
    dy[pick] = normal(5, n, std=0.01)
    dx, da, db = backward(dy, *xargs, h, ad, groups)
    want = ref.backward(dy[pick].double(), x64, h[pick].double(), ad.a, ad.b, ad.scale, ids[pick],
                        None, codes)
    for got, w, e, name in zip((dx[pick], da, db), *want, ("dx", "da", "db")):
        ref.check(got, w, e, name)
    dx[pick] = 0
    assert not bool(dx.any())  # rows without dY
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("b", [40, 1300])
def test_most_adapters(twq, device, b, codes):
    c = Case(twq, device, b, 256, 128, 16, 4096, "mixed", codes)
    c.check_linear(c.base, c.linear(*c.xargs, c.ad, c.groups, base=c.base))
    c.check_backward(None, c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups))
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("b,m,n,r,kind", [
    (40, 2048, 1024, 16, "mixed"), (3000, 6144, 256, 48, "runs"), (2500, 4096, 512, 128, "runs"),
    (2000, 1024, 2048, 24, "mixed"),
])
def test_equal_bits_from_cold_caches(twq, device, b, m, n, r, kind, codes):
    """What a copy brings late must not be read early, nor overwritten while it is read."""
    c = Case(twq, device, b, m, n, r, 6, kind, codes)
    want = c.linear(*c.xargs, c.ad, c.groups, base=c.base)
    wantb = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    c.check_linear(c.base, want)
    c.check_backward(c.dx_base, wantb)
    other = torch.empty(256 << 20, dtype=torch.uint8, device=device)  # twice the L2
    for i in range(24):
        other.fill_(i)
        got = c.linear(*c.xargs, c.ad, c.groups, base=c.base)
        if i % 2:
            other.fill_(i + 100)
        gotb = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
        assert all(torch.equal(p, q) for p, q in zip(got + gotb, want + wantb))
    assert twq.device_status() == 0


@pytest.mark.parametrize("b,m,n,r,count", [
    (2900, 256, 8192, 16, 7),   # forward pass: partial tiles of rows that follow one another
    (1500, 6400, 256, 48, 3),   # gradients: dx of 100 units of 64 columns
    (700, 5120, 4096, 128, 2),  # two stages of base only
])
def test_base_stages_are_refilled(twq, device, b, m, n, r, count):
    """A stage of base is combined in place and then filled again, by TMA where a tile's rows
    follow one another and by single copies where they do not; both kinds of tiles in turn,
    full and partial, base apart from the output and in its place."""
    c = Case(twq, device, b, m, n, r, count, "runs", False)
    ids = c.ids.clone()
    scattered = torch.randperm(b // 3, generator=torch.Generator().manual_seed(2))
    ids[:b // 3] = ids[:b // 3][scattered]
    c.ids = ids
    c.groups = twq.group_rows(ids.to(device), count)
    want = c.linear(*c.xargs, c.ad, c.groups, base=c.base)
    wantb = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    c.check_linear(c.base, want)
    c.check_backward(c.dx_base, wantb)
    for _ in range(20):
        y, dx = c.base.clone(), c.dx_base.clone()
        got = c.linear(*c.xargs, c.ad, c.groups, base=y, y=y)
        gotb = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=dx, dx=dx)
        assert all(torch.equal(p, q) for p, q in zip(got + gotb, want + wantb))
    assert twq.device_status() == 0


def test_call_on_another_stream_while_the_callers_is_busy(twq, device):
    """A block that the caller has freed while work on it is still queued: a call on another
    stream, whose inputs are ready, must not be given that block."""
    c = Case(twq, device, 64, 512, 1024, 16, 3, "mixed", False)
    want = (twq.adapter_linear(c.x, c.ad, c.groups, base=c.base)
            + twq.adapter_backward(c.dy, c.x, c.h, c.ad, c.groups))
    ids = c.ids.to(device)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [t.numel() * 2 for t in want]
    sizes += [twq.adapter_backward_workspace_bytes(64, 512, 1024, 16, 3), c.groups._buf.numel() * 4]
    blocks = [torch.empty(k, dtype=torch.uint8, device=device) for k in sizes]
    torch.cuda._sleep(200000000)  # some 0.1 s
    for t in blocks:
        t.fill_(255)
    del blocks, t
    g = twq.group_rows(ids, 3, stream=s)
    got = (twq.adapter_linear(c.x, c.ad, g, base=c.base, stream=s)
           + twq.adapter_backward(c.dy, c.x, c.h, c.ad, g, stream=s))
    torch.cuda.synchronize()
    assert torch.equal(g.order, c.groups.order) and torch.equal(g.offsets, c.groups.offsets)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


FIRST = [(1300, 1024, 256, r, 3, codes) for r in (16, 48, 80, 112, 128) for codes in (False, True)]


def first_calls(binding, device, how):
    """Digests of the outputs of FIRST's calls: one after another, at once on a thread each, or
    each captured into a graph without a call before."""
    import hashlib
    import threading

    def digest(tensors):
        torch.cuda.synchronize()
        return hashlib.sha256(b"".join(t.view(torch.int16).cpu().numpy().tobytes() for t in tensors)).hexdigest()

    cases = [Case(binding, device, b, m, n, r, count, "mixed", codes) for b, m, n, r, count, codes in FIRST]
    torch.cuda.synchronize()

    def call(c):
        return (*c.linear(*c.xargs, c.ad, c.groups, base=c.base),
                *c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base))

    out = [None] * len(cases)
    if how == "in turn":
        out = [call(c) for c in cases]
    elif how == "threads":
        gate = threading.Barrier(len(cases))

        def run(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait()
                out[i] = call(cases[i])
                torch.cuda.current_stream().synchronize()

        threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    else:
        for i, c in enumerate(cases):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out[i] = call(c)
            graph.replay()
            torch.cuda.synchronize()
    return [digest(o) for o in out]


@pytest.mark.parametrize("how", ["threads", "captured"])
def test_first_calls_of_a_process(twq, device, how):
    """What the library asks once (how many clusters fit) has the same answer, so the calls the
    same bits, whichever call comes first: from several threads at once, or under capture."""
    import os
    import subprocess
    import sys

    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import torch, test_gpu_adapters as t\n"
            "from rank_residual_w4a4_b200 import twq\n"
            "twq.load()\n"
            "print('\\n'.join(t.first_calls(twq, torch.device('cuda:0'), %r)))\n"
            % (os.path.dirname(os.path.abspath(__file__)),
               os.path.dirname(os.path.dirname(os.path.abspath(__file__))), how))
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
    assert run.stdout.split() == first_calls(twq, device, "in turn")


def test_calls_after_a_reset_of_the_device(twq, device):
    """twq_release_cache is all that a program has to call after a cudaDeviceReset. In a process
    of its own, whose context is the one that ends."""
    import os
    import subprocess
    import sys
    run = subprocess.run([sys.executable, os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                       "device_reset.py")],
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def check_infinities(got, want, bound, what):
    """As the definition: NaN where it has NaN, an infinity of its sign where it has one, and
    within the bound elsewhere."""
    g = got.double()
    assert torch.equal(g.isnan(), want.isnan()), "NaN of %s" % what
    inf = want.isinf()
    assert torch.equal(g[inf], want[inf]), "infinities of %s" % what
    fin = want.isfinite()
    assert bool(g[fin].isfinite().all()) and bool(bound[fin].isfinite().all()), what
    assert bool(((g[fin] - want[fin]).abs() <= bound[fin]).all()), what


def with_infinite_x(twq, device, b, r, codes):
    """A case with an infinity in the X of one row, positive A and B, so that no two infinities
    meet in a sum: (the case, the row, the columns of the infinity)."""
    c = Case(twq, device, b, 512, 256, r, 2, "one", codes)
    c.ad.a.abs_(), c.ad.b.abs_()
    i = b // 2
    if codes:
        xq8, sx = c.xargs
        xq8[i, 130], xq8[i, 128:256] = 1, xq8[i, 128:256].abs().clamp(min=1)
        sx[i, 1] = float("inf")
        c.x64 = ref.x_of_codes(xq8, sx)
        return c, i, slice(128, 256)
    c.x[i, 130] = float("inf")
    c.x64 = c.x.double()
    return c, i, slice(130, 131)


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 72, 120])
@pytest.mark.parametrize("b", [3, 1700])
def test_infinite_x_of_a_row_with_an_adapter(twq, device, b, r, codes):
    """h and y of the infinity's row are infinite, and no other row's."""
    c, i, _ = with_infinite_x(twq, device, b, r, codes)
    got = c.linear(*c.xargs, c.ad, c.groups, base=c.base)
    want = c.ref_linear(c.base)
    assert bool(want[0][0][i].isinf().all()) and bool(want[0][1][i].isinf().all())
    for g, w, e, name in zip(got, *want, ("y", "h")):
        check_infinities(g, w, e, name)
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 72, 120])
@pytest.mark.parametrize("b", [3, 1700])
def test_gradients_with_an_infinite_x(twq, device, b, r, codes):
    """The gradient of A is infinite, of the sign that dh has, in the infinity's columns, and
    nothing else is."""
    c, _, columns = with_infinite_x(twq, device, b, r, codes)
    got = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    want = c.ref_backward(c.dx_base)
    assert bool(want[0][1][-1][:, columns].isinf().all()) and int(want[0][1].isfinite().sum()) > 0
    for g, w, e, name in zip(got, *want, ("dx", "da", "db")):
        check_infinities(g, w, e, name)
    assert twq.device_status() == 0


@pytest.mark.parametrize("r", [8, 24, 80])
@pytest.mark.parametrize("b", [3, 1700])
def test_infinite_dy_of_a_row_with_an_adapter(twq, device, b, r):
    """An infinity in dY: dh of its row is infinite, so dx of that row (A is positive) and, where
    the row's X is not zero, all of dA; dB in the infinity's column."""
    c = Case(twq, device, b, 512, 256, r, 2, "one", False)
    c.ad.a.abs_(), c.ad.b.abs_()
    c.dy[b // 2, 200] = float("-inf")
    got = c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    want = c.ref_backward(c.dx_base)
    assert bool(want[0][0][b // 2].isinf().all())
    for g, w, e, name in zip(got, *want, ("dx", "da", "db")):
        check_infinities(g, w, e, name)
    assert twq.device_status() == 0


@pytest.mark.parametrize("b,count", [(0, 4), (1, 1), (768, 1), (768, 4096), (769, 48), (769, 49),
                                     (1536, 95), (1536, 96), (1536, 4096), (1537, 97), (1537, 4096),
                                     (20001, 4096)])
def test_grouping_stays_inside_its_buffers(twq, device, b, count):
    """As many tiles as a batch can have (every key has rows, all but one of them one row only):
    the words around order, offsets and tiles keep their values, and the forward pass of these
    tiles is right."""
    import ctypes

    keys = min(b, count + 1)
    ids = torch.zeros(b, dtype=torch.int32)
    ids[:keys] = torch.arange(keys, dtype=torch.int32) - 1 + (0 if keys > count else 1)
    ids = ids[torch.randperm(b, generator=torch.Generator().manual_seed(b))]
    sizes = (ctypes.c_size_t * 3)()
    assert twq.load().twq_row_groups_sizes(b, count, sizes) == 0
    bufs = [torch.full((s // 4 + 128,), 77, dtype=torch.int32, device=device) for s in sizes]
    g = twq.RowGroups(b, count, device)
    g._c = twq._RowGroups(b, count, *[t.data_ptr() + 256 for t in bufs])
    g._ref = ctypes.byref(g._c)
    twq.group_rows(ids.to(device), count, groups=g)
    order, offsets = (t[64:-64] for t in bufs[:2])
    key = torch.where(ids < 0, count, ids).long()
    assert torch.equal(order.cpu(), torch.sort(key, stable=True).indices.int())
    assert int(offsets[-1]) == int((ids >= 0).sum())
    for t in bufs:
        assert bool((t[:64] == 77).all()) and bool((t[-64:] == 77).all())
    if b:
        gen = torch.Generator(device=device).manual_seed(count)
        normal = lambda *shape: torch.randn(shape, generator=gen, device=device).to(torch.bfloat16)
        ad = twq.Adapters(normal(count, 8, 128) / 11, normal(count, 128, 8) / 20,
                          torch.ones(count, device=device))
        x, base = normal(b, 128), normal(b, 128)
        got = twq.adapter_linear(x, ad, g, base=base)
        want = ref.linear(x.double(), ad.a, ad.b, ad.scale, ids.to(device), base.double(), False)
        for p, w, e, name in zip(got, *want, ("y", "h")):
            ref.check(p, w, e, name)
        for t in bufs:
            assert bool((t[:64] == 77).all()) and bool((t[-64:] == 77).all())
    assert twq.device_status() == 0


@pytest.mark.parametrize("codes", [False, True], ids=["bf16", "codes"])
@pytest.mark.parametrize("kind", ["one", "mixed"])  # rows by TMA, rows one by one
@pytest.mark.parametrize("b,m,n,r", [(2000, 2048, 2560, 16), (1300, 4096, 4096, 64), (1200, 2560, 2048, 128),
                                     (130, 128, 128, 104)])
def test_waits_that_run_out(twq, device, b, m, n, r, kind, codes):
    """A loading warp of each kernel stops early: the waits on it run out after 0.2 ms, the copies
    under way land (a wait of their own, of up to 2 s each, that would be seen here), the kernels
    leave, the status tells, and the next calls are right."""
    import time

    c = Case(twq, device, b, m, n, r, 2, kind, codes)
    forward = lambda: c.linear(*c.xargs, c.ad, c.groups, base=c.base)
    backward = lambda: c.backward(c.dy, *c.xargs, c.h, c.ad, c.groups, dx_base=c.dx_base)
    want = forward() + backward()
    assert twq.device_status() == 0
    for call in (forward, backward):
        twq.selftest_adapter_stall(200000)
        try:
            t0 = time.perf_counter()
            call()
            code = twq.device_status()
            spent = time.perf_counter() - t0
        finally:
            twq.selftest_adapter_stall(0)
        assert 61 <= code <= 67 and spent < 1.0, (code, spent)
        assert twq.device_status() == 0
        assert all(torch.equal(p, q) for p, q in zip(forward() + backward(), want))
    assert twq.device_status() == 0
