"""The adapter operators in 64 bits from their definition, with a bound on each output's
error: every rounding counted at half a step relative to the value it rounds.

u = 2^-8 is half a BF16 step; f32 sums of k terms are bounded by (k + 32) 2^-23 times the
sum of the terms' magnitudes (tensor cores may truncate an addition: a whole step of
2^-23 each). BF16 intermediates: h (by definition of the operator), dh (rounded once for dx;
for dA in two terms, the second one the rounding of what the first left, so u^2), and X when
it comes from codes (code * scale is rounded once to BF16 where a kernel uses it so)."""
import torch

U = 2.0 ** -8
F = 2.0 ** -23


def x_of_codes(xq8, sx):
    return xq8.double() * sx.double().repeat_interleave(128, dim=1)


def rows_of(ids, count):
    return [(k, (ids == k).nonzero().flatten()) for k in range(count) if bool((ids == k).any())]


def group(ids, count):
    key = [k if 0 <= k < count else count for k in ids.tolist()]
    order = sorted(range(len(key)), key=lambda i: (key[i], i))
    offsets = [sum(1 for k in key if k < g) for g in range(count + 1)]
    return order, offsets


def linear(x, a, b, scale, ids, base, codes):
    """(y, h) and their error bounds, all float64; x, base float64."""
    count, r, m = a.shape
    n = b.shape[1]
    y = torch.zeros((x.shape[0], n), dtype=torch.float64, device=x.device) if base is None else base.clone()
    y_err = torch.zeros_like(y)  # a row without adapter is base itself
    h = torch.zeros((x.shape[0], r), dtype=torch.float64, device=x.device)
    h_err = torch.zeros_like(h)
    for k, rows in rows_of(ids, count):
        ak, bk, s = a[k].double(), b[k].double(), scale[k].double()
        hk = x[rows] @ ak.T
        mag = x[rows].abs() @ ak.abs().T
        e_sum = (m + 32) * F * mag + (U * mag if codes else 0.0)
        he = e_sum + U * (hk.abs() + e_sum)
        h[rows], h_err[rows] = hk, he
        d = s * (hk @ bk.T)
        yk = y[rows] + d
        ye = s.abs() * (he @ bk.abs().T) + (r + 34) * F * (s.abs() * (hk.abs() @ bk.abs().T) + y[rows].abs())
        y[rows] = yk
        y_err[rows] = ye + U * (yk.abs() + ye)
    return (y, h), (y_err, h_err)


def backward(dy, x, h, a, b, scale, ids, dx_base, codes):
    """(dx, da, db) and their error bounds, all float64; dy, x, h, dx_base float64."""
    count, r, m = a.shape
    n = b.shape[1]
    dx = torch.zeros((dy.shape[0], m), dtype=torch.float64, device=dy.device) if dx_base is None else dx_base.clone()
    dx_err = torch.zeros_like(dx)
    da = torch.zeros(a.shape, dtype=torch.float64, device=a.device)
    db = torch.zeros(b.shape, dtype=torch.float64, device=a.device)
    da_err, db_err = torch.zeros_like(da), torch.zeros_like(db)
    for k, rows in rows_of(ids, count):
        ak, bk, s = a[k].double(), b[k].double(), scale[k].double()
        t = rows.numel()
        dyk, xk, hk = dy[rows], x[rows], h[rows]
        dh = s * (dyk @ bk)
        mag = s.abs() * (dyk.abs() @ bk.abs())
        e = (n + 34) * F * mag
        dhe, dhe2 = e + U * (dh.abs() + e), e + U * U * (dh.abs() + e)
        d = dx[rows] + dh @ ak
        de = dhe @ ak.abs() + (r + 34) * F * (dh.abs() @ ak.abs() + dx[rows].abs())
        dx[rows], dx_err[rows] = d, de + U * (d.abs() + de)
        da[k] = dh.T @ xk
        mag = dh.abs().T @ xk.abs()
        e = dhe2.T @ xk.abs() + (2 * t + 34) * F * mag + (U * 1.01 * mag if codes else 0.0)
        da_err[k] = e + U * (da[k].abs() + e)
        db[k] = s * (dyk.T @ hk)
        e = (t + 34) * F * s.abs() * (dyk.abs().T @ hk.abs())
        db_err[k] = e + U * (db[k].abs() + e)
    return (dx, da, db), (dx_err, da_err, db_err)


def check(got, want, bound, what):
    """Elementwise bound, and the Frobenius norm: independent roundings are u/sqrt(3)
    each at most, three of them (X or dh, h, the output) make u; half as much again."""
    g = got.double()
    assert g.shape == want.shape, what
    assert bool(torch.isfinite(g).all()), "non-finite %s" % what
    over = ((g - want).abs() - bound).max().item() if g.numel() else 0.0
    assert over <= 0.0, "%s: bound exceeded by %.3g" % (what, over)
    nw = want.norm().item()
    if nw > 0:
        rel = (g - want).norm().item() / nw
        assert rel <= 1.5 * U, "%s: relative Frobenius error %.3g" % (what, rel)
