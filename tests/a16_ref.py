"""The operators on packed weights with BF16 activations in 64 bits from their definition, with a
bound on each output's error.

u = 2^-8 is half a BF16 step; an fp32 sum of k terms is off by at most (k + 32) 2^-23 times the sum
of the terms' magnitudes (tensor cores may truncate an addition: a whole step of 2^-23 each). Codes
times BF16 are exact in fp32. Roundings: h once to BF16, the activations of an expert to two BF16
terms (u^2), y once; silu(g) u in fp32 is counted at 2^-20 of its value (an exponential, a division
and two products, some ulps each), and |silu'| < 1.1 carries g's error on."""
import torch

U = 2.0 ** -8
F = 2.0 ** -23


def dequant(q, s):
    """Codes (n, m/2 bytes) and scales (m/128, n) -> (m, n) float64."""
    n, half = q.shape
    v = torch.empty((n, 2 * half), dtype=torch.float64, device=q.device)
    v[:, 0::2], v[:, 1::2] = (q & 15).double(), (q >> 4).double()
    v = torch.where(v > 7, v - 16, v)
    return (v * s.double().t().repeat_interleave(128, dim=1)).t()


def factors(w, e=None):
    rq, sr, l1q, sl1, l2t = (t if e is None else t[e] for t in (w.rq, w.sr, w.l1q, w.sl1, w.l2t))
    return dequant(rq, sr), dequant(l1q, sl1) if w.r else None, l2t.double().t() if w.r else None


def product(x, x_err, w, e=None):
    """x D(R) + h L2 and its error, y not rounded; x has the error x_err. Also h and its error."""
    R, L1, L2 = factors(w, e)
    y, mag = x @ R, x.abs() @ R.abs()
    err = (w.m + 32) * F * mag + x_err @ R.abs()
    if not w.r:
        return y, err, None, None
    h = x @ L1
    e1 = (w.m + 32) * F * (x.abs() @ L1.abs()) + x_err @ L1.abs()
    he = e1 + U * (h.abs() + e1)
    err = err + he @ L2.abs() + (w.r + 34) * F * (h.abs() @ L2.abs() + mag)
    return y + h @ L2, err, h, he


def linear(x, w):
    """((y, h), (y_err, h_err)); h None with rank 0."""
    x = x.double()
    y, err, h, he = product(x, torch.zeros_like(x), w)
    return (y, h), (err + U * (y.abs() + err), he)


def experts(x, ids, weights, ex, base):
    """(y, y_err): every expert on its own tokens."""
    x, weights = x.double(), weights.double()
    y = torch.zeros_like(x) if base is None else base.double().clone()
    mag, err = y.abs(), torch.zeros_like(y)
    for e in range(ex.count):
        rows, slots = (ids == e).nonzero(as_tuple=True)
        if not rows.numel():
            continue
        gu, ge, _, _ = product(x[rows], torch.zeros_like(x[rows]), ex.up, e)
        g, u = gu[:, :ex.f], gu[:, ex.f:]
        eg, eu = ge[:, :ex.f], ge[:, ex.f:]
        silu = torch.sigmoid(g) * g
        a = silu * u
        ae = (1.1 * eg * (u.abs() + eu) + silu.abs() * eu) + (2.0 ** -20 + U * U) * (a.abs() + eu)
        ye, yerr, _, _ = product(a, ae, ex.down, e)
        p = weights[rows, slots, None]
        y.index_add_(0, rows, p * ye)
        mag.index_add_(0, rows, (p * ye).abs())
        err.index_add_(0, rows, p.abs() * yerr)
    err = err + (ids.shape[1] * 2 + 8) * F * mag
    return y, err + U * (y.abs() + err)


def route(logits, k, renormalize):
    """(ids, weights) from sorted Python rows: NaN first, then descending, ties by index."""
    ids, weights = [], []
    for row in logits.double().tolist():
        order = sorted(range(len(row)), key=lambda j: (row[j] == row[j], -row[j] if row[j] == row[j] else 0.0, j))
        chosen = [j for j in order[:k] if not row[j] == -float("inf")]
        v = torch.tensor(row, dtype=torch.float64)
        top = v[chosen[0]] if chosen else None
        e = torch.where(v == top, 1.0, torch.exp(v - top)) if chosen else v
        total = (e[chosen] if renormalize else e).sum() if chosen else 1.0
        ids.append(chosen + [-1] * (k - len(chosen)))
        weights.append([float(e[j] / total) for j in chosen] + [0.0] * (k - len(chosen)))
    return torch.tensor(ids, dtype=torch.int32), torch.tensor(weights, dtype=torch.float64)


def check(got, want, bound, what):
    """Elementwise bound, and the Frobenius norm: the roundings of y and of h are u/sqrt(3) each at
    most, together less than u; half as much again."""
    g = got.double()
    assert g.shape == want.shape, what
    assert bool(torch.isfinite(g).all()), "non-finite %s" % what
    over = ((g - want).abs() - bound).max().item() if g.numel() else 0.0
    assert over <= 0.0, "%s: bound exceeded by %.3g" % (what, over)
    nw = want.norm().item()
    if nw > 0:
        rel = (g - want).norm().item() / nw
        assert rel <= 1.5 * U, "%s: relative Frobenius error %.3g" % (what, rel)
