"""The experts' products where their precision shows: cases on packed weights that are made without the
library, their definition in 64 bits (h rounded to BF16 as defined, nothing else), and a check of the
whole error against y's own rounding.

check_norm: with y = bf16(w + d) for the exact w, an element's error is at most that of bf16(w) plus
2 |d| (where the rounding goes the other way, w lies within |d| of the border). So the norm of the
error is at most r + 2 |d|, r the norm of bf16(w) - w, which is 0.0016 of y's to 0.0017. d in norm,
relative to y: the activations' two BF16 terms 2^-17 or less (they round twice: 2^-8 of 2^-8 half a
step each), fp32 sums of K / 16 products and the groups in order (K / 16 + K / 128) 2^-23, 2e-5 at the
longest here, much less as they go either way; h, by as much off, rounds the other way in one element of
some thousands, by a step of 2^-8 to 2^-7: 1e-4 of h, 4e-5 of y, twice. Together below 8e-5, and
2 |d| below a tenth of r."""
from types import SimpleNamespace

import torch

import a16_ref as ref

BF = torch.bfloat16

# b, m, f, r, r_down, count, k: for one, two and four tiles of the down product, with and without ranks
CASES = [
    (1, 256, 128, 16, 16, 4, 2), (1, 2048, 256, 0, 0, 16, 8), (4, 512, 256, 32, 0, 8, 2), (5, 256, 640, 64, 16, 3, 3),
    (8, 384, 256, 0, 0, 2, 1), (8, 384, 256, 0, 48, 2, 1), (7, 256, 384, 16, 32, 4, 2), (13, 256, 256, 128, 128, 33, 8),
    (24, 512, 128, 16, 16, 3, 2), (64, 384, 384, 16, 16, 7, 4), (64, 256, 128, 32, 32, 2, 2),
]
MUTANTS = ["one term", "y_e in bf16", "g and u in bf16", "one term, y_e in bf16", "silu off by 1e-3"]


def stacked(gen, count, m, n, r):
    """`count` layers of random codes and scales, as twq_weights holds them, on the CPU."""
    def codes(cols):
        c = torch.round(torch.randn((count, cols, m), generator=gen) * 2.3).clamp(-7, 7).to(torch.int32)
        return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8)

    def scales(cols):
        return (0.5 + torch.rand((count, m // 128, cols), generator=gen)) * (m ** -0.5 / 2.3)

    return SimpleNamespace(m=m, n=n, r=r, rq=codes(n), sr=scales(n), l1q=codes(r), sl1=scales(r),
                           l2t=(torch.randn((count, n, r), generator=gen) * (0.4 / max(r, 1) ** 0.5)).to(BF))


def make(case):
    b, m, f, r, rd, count, k = case
    gen = torch.Generator().manual_seed(sum(case))
    ex = SimpleNamespace(count=count, m=m, f=f, up=stacked(gen, count, m, 2 * f, r), down=stacked(gen, count, f, m, rd))
    x = torch.randn((b, m), generator=gen).to(BF)
    ids = torch.rand((b, count), generator=gen).argsort(dim=1)[:, :k].to(torch.int32).contiguous()
    return x, ids, 0.5 + torch.rand((b, k), generator=gen), ex


def make_low_rank(b):
    """Experts whose y_e is h2 itself, bit by bit: the down product's codes are 0, its L2 the identity."""
    x, ids, _, ex = make((b, 256, 256, 0, 256, 2, 1))
    ex.down.rq.zero_()
    ex.down.l2t.copy_(torch.eye(256, dtype=BF).expand(2, 256, 256))
    return x, ids, torch.ones((b, 1)), ex


def rounded(v):
    return v.to(torch.float32).to(BF).double()


def product(x, w, e):
    R, L1, L2 = ref.factors(w, e)
    return x @ R + (rounded(x @ L1) @ L2 if w.r else 0.0)


def experts(x, ids, weights, ex, how=None):
    """y before its rounding. how: None, the definition; "kernel", with a in two BF16 terms; else one of
    MUTANTS."""
    x, weights = x.double(), weights.double()
    y = torch.zeros_like(x)
    for e in range(ex.count):
        rows, slots = (ids == e).nonzero(as_tuple=True)
        if not rows.numel():
            continue
        gu = product(x[rows], ex.up, e)
        if how == "g and u in bf16":
            gu = rounded(gu)
        g, u = gu[:, :ex.f], gu[:, ex.f:]
        a = torch.sigmoid(g) * g * u
        if how == "silu off by 1e-3":
            a = a * (1 + 1e-3)
        if how is not None:
            high = rounded(a)
            a = high if how.startswith("one term") else high + rounded(a - high)
        ye = product(a, ex.down, e)
        if how is not None and how.endswith("y_e in bf16"):
            ye = rounded(ye)
        y.index_add_(0, rows, weights[rows, slots, None] * ye)
    return y


def ratio(got, want):
    """The norm of got's error, in norms of y's own rounding."""
    return ((got.double() - want).norm() / (rounded(want) - want).norm()).item()


def check_norm(got, want, what):
    over = ratio(got, want)
    assert over <= 1.1, "%s: error of %.3f times the output's own rounding" % (what, over)


def changed(got, want):
    """The share of elements that are not the definition's, rounded."""
    return (got.double() != rounded(want)).double().mean().item()
