"""The layer on BF16 activations, the choice of experts and their products on the GPU against
their definition in 64 bits (a16_ref.py); then the ways a program calls them (strided X, in place,
another stream, captured and replayed, one after another)."""
import pytest
import torch

import a16_ref as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def twq(device):
    from rank_residual_w4a4_b200 import _build, twq as binding
    _build.build()
    binding.load()
    return binding


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(BF)


def make_x(gen, b, m):
    x = normal(gen, b, m)
    x[:, ::100] *= 30
    return x


def make_layer(twq, gen, m, n, r, device):
    """A layer packed by the library from BF16 factors."""
    R = normal(gen, m, n, std=m ** -0.5).to(device)
    if not r:
        return twq.pack_weights(R, None, None)
    return twq.pack_weights(R, normal(gen, m, r, std=m ** -0.5).to(device),
                            normal(gen, r, n, std=0.4 * r ** -0.5).to(device))


def make_experts(twq, gen, count, m, f, r, rd, device):
    ex = twq.Experts.empty(count, m, f, r, device, r_down=rd)
    for e in range(count):
        def fac(a, n, rank):
            return (normal(gen, a, n, std=a ** -0.5).to(device),
                    normal(gen, a, rank, std=a ** -0.5).to(device) if rank else None,
                    normal(gen, rank, n, std=0.4 * rank ** -0.5).to(device) if rank else None)
        ex.pack(e, *fac(m, 2 * f, r), *fac(f, m, rd))
    return ex


# b, m, n, r: one token to 64, around the tiles of 8, 16 and 32 rows, one group and many, column
# tiles that end inside a tile of 32 ranks, odd numbers of groups
SHAPES = [
    (1, 128, 128, 0), (1, 128, 128, 16), (1, 4096, 256, 128), (2, 256, 384, 32), (3, 384, 128, 48),
    (7, 1152, 640, 256), (8, 512, 512, 0), (9, 640, 256, 80), (15, 2048, 128, 16), (16, 512, 1152, 144),
    (17, 256, 256, 0), (24, 896, 384, 208), (31, 1024, 128, 64), (32, 384, 896, 240), (33, 512, 512, 16),
    (63, 128, 1024, 32), (64, 2176, 256, 0), (64, 768, 512, 256), (5, 14336, 128, 112), (1, 128, 6400, 0),
    (12, 3200, 4736, 96), (64, 256, 9600, 16),
]


@pytest.mark.parametrize("b,m,n,r", SHAPES)
def test_linear(twq, device, b, m, n, r):
    gen = torch.Generator().manual_seed(b + m + 3 * n + 7 * r)
    w = make_layer(twq, gen, m, n, r, device)
    x = make_x(gen, b, m).to(device)
    h = torch.full((b, r), float("nan"), dtype=BF, device=device) if r else None
    y = twq.fused_linear_a16(x, w, h=h)
    (y64, h64), (ye, he) = ref.linear(x, w)
    ref.check(y, y64, ye, "y")
    if r:
        ref.check(h, h64, he, "h")
    assert torch.equal(y, twq.fused_linear_a16(x, w))  # equal calls, equal bits
    assert twq.device_status() == 0


def test_linear_rows_are_alone(twq, device):
    """A row's result does not depend on what other rows hold: infinities, NaN, zeros."""
    gen = torch.Generator().manual_seed(3)
    w = make_layer(twq, gen, 512, 384, 32, device)
    x = make_x(gen, 20, 512).to(device)
    clean = twq.fused_linear_a16(x, w)
    bad = x.clone()
    bad[3, 7], bad[11, 500], bad[19] = float("inf"), float("nan"), 0.0
    got = twq.fused_linear_a16(bad, w)
    rows = [i for i in range(20) if i not in (3, 11, 19)]
    assert torch.equal(got[rows], clean[rows])
    assert not bool(torch.isfinite(got[3]).any()) and bool(torch.isnan(got[11]).all())
    assert not bool(got[19].any())


def test_linear_zero_groups_and_extremes(twq, device):
    """Groups of zeros (scale 0) add nothing; the codes -7 and 7 and large X stay exact."""
    gen = torch.Generator().manual_seed(4)
    R = torch.zeros((384, 128), dtype=BF)
    R[128:256] = torch.where(torch.rand((128, 128), generator=gen) < 0.5, -1.75, 1.75)
    w = twq.pack_weights(R.to(device), None, None)
    x = torch.randint(-128, 128, (6, 384), generator=gen).to(BF)
    y = twq.fused_linear_a16(x.to(device), w)
    want = (x.double() @ R.double()).to(BF)  # sums of multiples of 1.75 that fp32 holds
    assert torch.equal(y.cpu(), want)


def test_linear_strided_x(twq, device):
    gen = torch.Generator().manual_seed(5)
    w = make_layer(twq, gen, 256, 256, 16, device)
    wide = make_x(gen, 12, 1024).to(device)
    x = wide[:, 512:768]
    assert torch.equal(twq.fused_linear_a16(x, w), twq.fused_linear_a16(x.contiguous(), w))
    with pytest.raises(twq.TwqError):
        twq.fused_linear_a16(wide[:, 4:260], w)       # not on a 16-byte boundary
    with pytest.raises(ValueError):
        twq.fused_linear_a16(wide[:, ::4], w)


def test_linear_matches_the_quantized_layer(twq, device):
    """On activations that the 8-bit quantizer holds exactly, the two layers agree within the
    rounding of y and h."""
    gen = torch.Generator().manual_seed(6)
    w = make_layer(twq, gen, 512, 512, 32, device)
    x = torch.randint(-127, 128, (4, 512), generator=gen).to(BF)
    x[:, ::128] = 127
    x = x.to(device)
    a8 = twq.fused_linear_a8(*twq.quantize_act_a8(x), w)
    (y64, _), (ye, _) = ref.linear(x, w)
    ref.check(a8, y64, ye, "quantized")
    ref.check(twq.fused_linear_a16(x, w), y64, ye, "bf16")


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("b,count,k", [(1, 1, 1), (1, 128, 8), (3, 5, 5), (9, 32, 4), (64, 33, 16), (17, 64, 1),
                                       (8, 200, 8), (100, 257, 6), (5, 600, 16), (1000, 1024, 8)])
def test_route(twq, device, b, count, k, dtype, renormalize):
    gen = torch.Generator().manual_seed(b + count + k)
    logits = (torch.randn((b, count), generator=gen) * 2).to(dtype)
    logits[::3, count // 2:] = -float("inf")      # masked experts; some rows have fewer than k left
    logits[1::4] = logits[1::4].round()           # ties
    ids, weights = twq.moe_route(logits.to(device), k, renormalize=renormalize)
    want_ids, want_w = ref.route(logits, k, renormalize)
    assert torch.equal(ids.cpu(), want_ids)
    # an exponential (2 ulps), sums of at most 1024 positive terms in fp32 and a division, in steps
    # of 2^-24; the exponent's own rounding counts |v - top| < 30 of them
    assert bool(((weights.cpu().double() - want_w).abs() <= (40 + 2 * 33) * 2.0 ** -24 * want_w).all())


def test_route_specials(twq, device):
    inf, nan = float("inf"), float("nan")
    rows = torch.tensor([
        [-inf, -inf, -inf, -inf, -inf], [0.0, -0.0, 0.0, -0.0, 0.0], [inf, 1.0, inf, -inf, 2.0],
        [1.0, nan, 3.0, 2.0, -inf], [-inf, -inf, -3e38, -inf, -inf], [3e38, -3e38, 3e38, 0.0, 1.0],
        [1e-42, -1e-42, 0.0, 2e-42, -inf]])
    for dtype in (torch.float32, BF):
        logits = rows.to(dtype)
        for renormalize in (True, False):
            ids, weights = twq.moe_route(logits.to(device), 3, renormalize=renormalize)
            want_ids, want_w = ref.route(logits, 3, renormalize)
            assert torch.equal(ids.cpu(), want_ids)
            assert torch.allclose(weights.cpu().double(), want_w, rtol=1e-6, atol=0, equal_nan=True)


def test_route_strided(twq, device):
    gen = torch.Generator().manual_seed(1)
    wide = torch.randn((6, 300), generator=gen).to(device)
    for view in (wide[:, 3:103], wide.to(BF)[:, 5:205]):
        a, b = twq.moe_route(view, 4), twq.moe_route(view.contiguous(), 4)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def make_ids(gen, b, k, count, kind):
    if kind == "none":
        return torch.full((b, k), -1, dtype=torch.int32)
    if kind == "one":                                  # every token on the last expert, in every slot
        return torch.full((b, k), count - 1, dtype=torch.int32)
    if kind == "any":                                  # the same expert twice in a token now and then
        return torch.randint(0, count, (b, k), generator=gen, dtype=torch.int32)
    ids = torch.rand((b, max(count, k)), generator=gen).argsort(dim=1)[:, :k].to(torch.int32)
    if kind == "wild":                                 # some elsewhere
        ids[::2, ::2] = count + 3
        ids[1::3] = -2 ** 31
        ids[2::5, -1] = 2 ** 31 - 1
    return ids.contiguous()


# b, m, f, r, r_down, count, k, kind
EXPERTS = [
    (1, 128, 128, 0, 0, 1, 1, "one"), (1, 256, 128, 16, 16, 4, 2, "mixed"), (1, 2048, 256, 0, 0, 16, 8, "mixed"),
    (2, 128, 384, 0, 48, 5, 3, "wild"), (4, 512, 256, 32, 0, 8, 2, "any"), (5, 256, 640, 64, 16, 3, 3, "mixed"),
    (8, 384, 256, 0, 0, 2, 1, "one"), (9, 640, 128, 16, 80, 16, 4, "mixed"), (13, 256, 256, 128, 128, 33, 8, "wild"),
    (16, 256, 512, 0, 16, 6, 2, "any"), (17, 128, 128, 16, 16, 4, 16, "any"), (24, 512, 128, 0, 0, 3, 2, "one"),
    (33, 256, 256, 48, 0, 40, 8, "mixed"), (64, 384, 384, 16, 16, 7, 4, "mixed"), (64, 128, 256, 0, 0, 64, 16, "wild"),
    (64, 256, 128, 32, 32, 2, 2, "one"), (3, 128, 2304, 0, 256, 2, 1, "any"), (6, 256, 128, 16, 16, 8, 2, "none"),
    (64, 128, 128, 0, 16, 1024, 16, "mixed"),
]


@pytest.mark.parametrize("b,m,f,r,rd,count,k,kind", EXPERTS)
def test_experts(twq, device, b, m, f, r, rd, count, k, kind):
    gen = torch.Generator().manual_seed(b + m + f + r + count)
    # many experts: a few packed ones, repeated
    few = make_experts(twq, gen, min(count, 7), m, f, r, rd, device)
    ex = few
    if count > 7:
        at = torch.arange(count, device=device) % 7
        def again(w):
            return twq.Weights(w.m, w.n, w.r, *(t[at].contiguous() for t in (w.rq, w.sr, w.l1q, w.sl1, w.l2t)))
        ex = twq.Experts(again(few.up), again(few.down))
    x, base = make_x(gen, b, m).to(device), normal(gen, b, m).to(device)
    ids = make_ids(gen, b, k, count, kind).to(device)
    weights = torch.rand((b, k), generator=gen).to(device)
    for bs in (base, None):
        y = twq.moe_experts(x, ids, weights, ex, base=bs)
        y64, ye = ref.experts(x, ids, weights, ex, bs)
        ref.check(y, y64, ye, "y")
        assert torch.equal(y, twq.moe_experts(x, ids, weights, ex, base=bs))
    if kind == "none":
        assert torch.equal(twq.moe_experts(x, ids, weights, ex, base=base), base)
    assert twq.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("b", [1, 6, 40])
def test_layer_is_route_and_experts(twq, device, b, dtype):
    gen = torch.Generator().manual_seed(b)
    ex = make_experts(twq, gen, 12, 256, 256, 32, 16, device)
    x, base = make_x(gen, b, 256).to(device), normal(gen, b, 256).to(device)
    logits = torch.randn((b, 12), generator=gen).to(dtype).to(device)
    logits[0, 1:] = -float("inf")                      # a token with one expert left
    y, ids, weights = twq.moe_layer(x, logits, 3, ex, base=base)
    ids2, weights2 = twq.moe_route(logits, 3)
    assert torch.equal(ids, ids2) and torch.equal(weights, weights2)
    assert torch.equal(y, twq.moe_experts(x, ids, weights, ex, base=base))
    y64, ye = ref.experts(x, ids, weights, ex, base)
    ref.check(y, y64, ye, "y")


def test_experts_tokens_are_alone(twq, device):
    gen = torch.Generator().manual_seed(8)
    ex = make_experts(twq, gen, 4, 256, 128, 16, 16, device)
    x, ids = make_x(gen, 10, 256).to(device), make_ids(gen, 10, 2, 4, "mixed").to(device)
    weights = torch.rand((10, 2), generator=gen).to(device)
    clean = twq.moe_experts(x, ids, weights, ex)
    bad = x.clone()
    bad[2, 5], bad[7, 200] = float("inf"), float("nan")
    got = twq.moe_experts(bad, ids, weights, ex)
    rows = [i for i in range(10) if i not in (2, 7)]
    assert torch.equal(got[rows], clean[rows])
    assert bool(torch.isnan(got[7]).all()) and not bool(torch.isfinite(got[2]).any())
    # an expert that has no row is never read
    ex.up.sr[3] = float("nan")
    some = torch.where(ids == 3, -1, ids)
    assert bool(torch.isfinite(twq.moe_experts(x, some, weights, ex)).all())


def test_in_place_base(twq, device):
    gen = torch.Generator().manual_seed(9)
    ex = make_experts(twq, gen, 4, 256, 128, 0, 0, device)
    x, base = make_x(gen, 5, 256).to(device), normal(gen, 5, 256).to(device)
    ids, weights = make_ids(gen, 5, 2, 4, "mixed").to(device), torch.rand((5, 2), generator=gen).to(device)
    want = twq.moe_experts(x, ids, weights, ex, base=base)
    y = base.clone()
    assert twq.moe_experts(x, ids, weights, ex, base=y, y=y) is y
    assert torch.equal(y, want)


def test_empty_batches(twq, device):
    gen = torch.Generator().manual_seed(10)
    w = make_layer(twq, gen, 256, 128, 16, device)
    ex = make_experts(twq, gen, 2, 256, 128, 0, 0, device)
    x = torch.empty((0, 256), dtype=BF, device=device)
    assert twq.fused_linear_a16(x, w).shape == (0, 128)
    y, ids, weights = twq.moe_layer(x, torch.empty((0, 2), device=device), 2, ex)
    assert y.shape == (0, 256) and ids.shape == (0, 2) and weights.shape == (0, 2)


def test_block_of_a_model(twq, device):
    """A decode step as a program runs it: projection, layer of experts on the residual stream, the
    next projection, each reading what the one before wrote, several steps in a row; then captured
    once and replayed on new inputs."""
    gen = torch.Generator().manual_seed(11)
    m, b = 512, 5
    proj, out = make_layer(twq, gen, m, m, 32, device), make_layer(twq, gen, m, 256, 0, device)
    ex = make_experts(twq, gen, 8, m, 256, 16, 16, device)
    router = normal(gen, m, 8, std=m ** -0.5).to(device)
    xs = [normal(gen, b, m).to(device) for _ in range(4)]

    def step(x):
        res = twq.fused_linear_a16(x, proj)
        y, ids, weights = twq.moe_layer(res, (res.float() @ router.float()), 2, ex, base=res)
        z = twq.fused_linear_a16(y, out)
        q = twq.fused_linear_x(y, proj)                # the quantized layer's kernel right after
        return res, y, ids, weights, z, q

    eager = [step(x) for x in xs]
    for x, (res, y, ids, weights, z, q) in zip(xs, eager):
        (r64, _), (re, _) = ref.linear(x, proj)
        ref.check(res, r64, re, "projection")
        y64, ye = ref.experts(res, ids, weights, ex, res)
        ref.check(y, y64, ye, "experts")
        (z64, _), (ze, _) = ref.linear(y, out)
        ref.check(z, z64, ze, "output")
        assert torch.equal(q, twq.fused_linear_x(y, proj))
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(static)
    for x, want in zip(xs, eager):
        static.copy_(x)
        graph.replay()
        for a, c in zip(held, want):
            assert torch.equal(a, c)
    assert twq.device_status() == 0


def test_two_streams(twq, device):
    """Calls that overlap, each with its own workspace."""
    gen = torch.Generator().manual_seed(12)
    ex = make_experts(twq, gen, 8, 512, 256, 16, 0, device)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for b in (3, 20):
        x, ids = make_x(gen, b, 512).to(device), make_ids(gen, b, 2, 8, "mixed").to(device)
        work.append((x, ids, torch.rand((b, 2), generator=gen).to(device)))
    want = [twq.moe_experts(*w[:3], ex) for w in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for s, w, o in zip(streams, work, got):
            o.append(twq.moe_experts(*w, ex, stream=s))
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(v, w) for v in o)


def test_experts_follow_their_weights(twq, device):
    """A field of up or down that is set anew is what the next call reads; one that does not fit is refused."""
    gen = torch.Generator().manual_seed(17)
    one, two = (make_experts(twq, gen, 3, 256, 128, 0, 0, device) for _ in range(2))
    x, ids = make_x(gen, 4, 256).to(device), make_ids(gen, 4, 2, 3, "mixed").to(device)
    w = torch.rand((4, 2), generator=gen).to(device)
    want = twq.moe_experts(x, ids, w, two)
    assert not torch.equal(twq.moe_experts(x, ids, w, one), want)
    one.up.rq, one.up.sr = two.up.rq.clone(), two.up.sr.clone()
    one.down = two.down
    assert torch.equal(twq.moe_experts(x, ids, w, one), want)
    one.up.rq = two.up.rq[:2].clone()
    with pytest.raises(ValueError):
        twq.moe_experts(x, ids, w, one)


def test_threads(twq, device):
    """Calls from several threads at once, each on a stream of its own."""
    import threading

    gen = torch.Generator().manual_seed(18)
    w, ex = make_layer(twq, gen, 1024, 512, 32, device), make_experts(twq, gen, 5, 512, 256, 16, 16, device)
    x, x2, logits = (t.to(device) for t in (make_x(gen, 7, 1024), make_x(gen, 7, 512), normal(gen, 7, 5)))
    calls = lambda: (twq.fused_linear_a16(x, w), twq.moe_layer(x2, logits, 2, ex)[0])
    want, wrong = calls(), []
    torch.cuda.synchronize()

    def run():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not all(torch.equal(a, c) for a, c in zip(calls(), want)):
                    wrong.append(1)

    threads = [threading.Thread(target=run) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and twq.device_status() == 0


def test_two_graphs_share_a_workspace(twq, device):
    """Two captured calls with one workspace and one output, replayed one after the other."""
    gen = torch.Generator().manual_seed(15)
    ex = make_experts(twq, gen, 8, 512, 256, 16, 16, device)
    ws = torch.empty(twq.moe_workspace_bytes(20, 3, ex), dtype=torch.uint8, device=device)
    y = torch.empty((20, 512), dtype=BF, device=device)
    graphs, want = [], []
    for b in (20, 2):
        x, logits = make_x(gen, b, 512).to(device), normal(gen, b, 8).to(device)
        want.append(twq.moe_layer(x, logits, 3, ex)[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = twq.moe_layer(x, logits, 3, ex, y=y[:b], workspace=ws)
        graphs.append((graph, b, held, x, logits))
    for _ in range(3):
        for (graph, b, *_), w in zip(graphs, want):
            y.fill_(7.0)
            graph.replay()
            assert torch.equal(y[:b], w) and (y[b:] == 7.0).all()  # rows behind the last: as they were


@pytest.mark.parametrize("call", ["linear", "experts"])
@pytest.mark.parametrize("b", [1, 12, 64])
def test_waits_that_run_out(twq, device, b, call):
    """The blocks' last steps get no activations: the waits on them run out after 0.2 ms, the
    copies under way land, the kernels leave, the status tells, and the next calls are right."""
    import time

    gen = torch.Generator().manual_seed(16)
    if call == "linear":
        x, w = make_x(gen, b, 8192).to(device), make_layer(twq, gen, 8192, 12800, 64, device)
        f = lambda: twq.fused_linear_a16(x, w)
    else:
        x, ex = make_x(gen, b, 2048).to(device), make_experts(twq, gen, 4, 2048, 1024, 16, 16, device)
        logits = normal(gen, b, 4).to(device)
        f = lambda: twq.moe_layer(x, logits, 2, ex)[0]
    want = f()
    assert twq.device_status() == 0
    twq.selftest_a16_stall(200000)
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


def test_experts_beyond_two_gigabytes(twq, device):
    """Codes of the last experts lie beyond 2^31 bytes."""
    count, m, f = 640, 2048, 2048
    ex = twq.Experts.empty(count, m, f, 0, device)
    assert ex.up.rq.numel() > 2 ** 31
    gen = torch.Generator().manual_seed(13)
    one = make_experts(twq, gen, 1, m, f, 0, 0, device)
    last = count - 1
    for a, c in ((ex.up, one.up), (ex.down, one.down)):
        a.rq[last], a.sr[last] = c.rq[0], c.sr[0]
    x = make_x(gen, 2, m).to(device)
    w = torch.ones((2, 1), device=device)
    got = twq.moe_experts(x, torch.full((2, 1), last, dtype=torch.int32, device=device), w, ex)
    # the order of the sums goes by the number of experts too, so not bit by bit
    y64, ye = ref.experts(x, torch.zeros((2, 1), dtype=torch.int32, device=device), w, one, None)
    ref.check(got, y64, ye, "y")


def test_refusals(twq, device):
    gen = torch.Generator().manual_seed(14)
    w = make_layer(twq, gen, 256, 128, 16, device)
    ex = make_experts(twq, gen, 2, 256, 128, 0, 0, device)
    x = make_x(gen, 65, 256).to(device)
    ids, weights = torch.zeros((4, 2), dtype=torch.int32, device=device), torch.ones((4, 2), device=device)
    for f in (lambda: twq.fused_linear_a16(x, w), lambda: twq.moe_route(x[:2].float(), 17),
              lambda: twq.moe_experts(x, ids.repeat(20, 1)[:65].contiguous(), weights.repeat(20, 1)[:65].contiguous(), ex),
              lambda: twq.moe_layer(x[:2], torch.ones((2, 2), device=device), 3, ex),
              lambda: twq.moe_experts(x[:4], ids, weights, ex, workspace=torch.empty(16, dtype=torch.uint8, device=device))):
        with pytest.raises(twq.TwqError):
            f()
    for f in (lambda: twq.fused_linear_a16(x[:4, :128], w), lambda: twq.fused_linear_a16(x[:4].cpu(), w),
              lambda: twq.moe_experts(x[:3], ids, weights, ex), lambda: twq.moe_experts(x[:4], ids, weights[:, :1], ex),
              lambda: twq.moe_layer(x[:2], torch.ones((2, 3), device=device), 1, ex),
              lambda: twq.Experts(ex.down, ex.up),
              lambda: twq.fused_linear_a16(x[:4], w, y=torch.empty((4, 129), dtype=BF, device=device))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: twq.fused_linear_a16(x[:4].float(), w), lambda: twq.moe_route(x[:4].half(), 1),
              lambda: twq.moe_experts(x[:4], ids.long(), weights, ex)):
        with pytest.raises(TypeError):
            f()
