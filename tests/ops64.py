"""Plain 64-bit forms of the stand-alone operators, with bounds on what fp32 arithmetic may add.

Every bound is a count of fp32 roundings: a rounding to nearest is off by at most U = 2^-24 of the
value, a sum of n terms in any tree of depth m by at most m * U times the sum of the terms' sizes (to
first order; each count below has a few steps to spare for the second), and the one rounding to
the result's type by finfo.eps / 2 of the result, or half the type's smallest step near zero.
"""
import math

import torch

U = 2.0 ** -24
F8 = torch.float64


def half_ulp(ref, dtype):
    """What rounding a value near ref once to dtype may change."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) * (1 + 2 * f.eps) + f.tiny * f.eps / 2


def assert_close(got, ref, tol, what=""):
    err = (got.to(F8) - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        worst = (err / tol.clamp_min(1e-300)).nan_to_num(math.inf).max().item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got "
                             f"{got[tuple(i)].item()}, exact {ref[tuple(i)].item()}, bound {tol[tuple(i)].item()}; "
                             f"worst {worst:.3g} x the bound")


def sort(idx, E):
    """offsets, perm, slot of a stable sort of idx [T, k] by expert (plain loops)."""
    flat = idx.flatten().tolist()
    by = [[] for _ in range(E)]
    for r, e in enumerate(flat):
        if 0 <= e < E:
            by[e].append(r)
    offsets, perm = [0], []
    for routes in by:
        perm += routes
        offsets.append(len(perm))
    slot = [-1] * len(flat)
    for row, r in enumerate(perm):
        slot[r] = row
    perm += [-1] * (len(flat) - len(perm))
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(perm, dtype=i32), torch.tensor(slot, dtype=i32).view(idx.shape))


def unsort(rows, slot, gate, dtype):
    """-> out, bound.  k products and k sums in fp32, one rounding."""
    T, k = slot.shape
    out = torch.zeros((T, rows.shape[1]), dtype=F8)
    size = torch.zeros_like(out)
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0)[:, 0]
        p = rows[slot[t, j].long()].to(F8) * (1 if gate is None else gate[t, j].to(F8)[:, None])
        out[t] += p
        size[t] += p.abs()
    return out, half_ulp(out, dtype) + (2 * k + 1) * U * size + 1e-44


def unsort_grad(dout, rows, slot, gate, dtype):
    """-> drows (nan where no route points), dgate, and their bounds."""
    T, k = slot.shape
    d = dout.shape[1]
    drows = torch.full((T * k, d), math.nan, dtype=F8)
    dgate = torch.zeros((T, k), dtype=F8)
    size = torch.zeros_like(dgate)
    for j in range(k):
        t = torch.nonzero(slot[:, j] >= 0)[:, 0]
        r = slot[t, j].long()
        g = dout[t].to(F8)
        drows[r] = g * (1 if gate is None else gate[t, j].to(F8)[:, None])
        if rows is not None:
            p = g * rows[r].to(F8)
            dgate[t, j] = p.sum(1)
            size[t, j] = p.abs().sum(1)
    # a thread of 32 or more adds its share of the row one by one, then 5 + 8 joins
    return drows, dgate, half_ulp(drows, dtype) + 2 * U * drows.abs(), (math.ceil(d / 32) + 16) * U * size + 1e-44


def norm(x, gain, bias, eps, layer, dtype):
    """-> y, stats, their bounds.  Chains: at most 64 terms a thread, 5 + 5 joins, the division: 80."""
    x = x.to(F8)
    d = x.shape[1]
    mean = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    dm = 80 * U * x.abs().mean(1, keepdim=True) if layer else torch.zeros_like(mean)
    c = x - mean
    var = (c * c).mean(1, keepdim=True)
    # the squares' chain, each difference's rounding, and the mean's error in each difference
    dvar = 84 * U * var + 2 * (dm + U * c.abs()).mul(c.abs()).mean(1, keepdim=True) + dm * dm
    r = (var + eps).rsqrt()
    rel = 0.5 * dvar / (var + eps) + 4 * U
    g = torch.ones(d, dtype=F8) if gain is None else gain.to(F8)
    b = torch.zeros(d, dtype=F8) if bias is None else bias.to(F8)
    y = c * r * g + b
    tol = half_ulp(y, dtype) + (c * r * g).abs() * (rel + 4 * U) + (g * r).abs() * dm + U * (y.abs() + b.abs()) + 1e-44
    return y, torch.cat([mean, r], 1), tol, torch.cat([dm + 1e-44, r * rel], 1)


def norm_grad(x, gain, stats, dy, layer, dtype):
    """-> dx, dgain, dbias, their bounds, at the statistics given."""
    x, dy, st = x.to(F8), dy.to(F8), stats.to(F8)
    T, d = x.shape
    mean = st[:, :1] if layer else torch.zeros_like(st[:, :1])
    r = st[:, 1:]
    xh = (x - mean) * r
    h = dy if gain is None else dy * gain.to(F8)
    m0 = h.mean(1, keepdim=True) if layer else torch.zeros_like(r)
    m1 = (h * xh).mean(1, keepdim=True)
    dx = r * (h - m0 - xh * m1)
    tol = half_ulp(dx, dtype) + r * (6 * U * (h.abs() + m0.abs() + (xh * m1).abs())
                                     + 84 * U * (h.abs().mean(1, keepdim=True) * (1 if layer else 0)
                                                 + xh.abs() * (h * xh).abs().mean(1, keepdim=True))) + 1e-44
    # a column: at least 64 blocks (or every row its own) share the rows, then 4 or 8 joins, then 64 + 8 more
    n = math.ceil(T / 64) + 100
    dgain, dbias = (dy * xh).sum(0), dy.sum(0)
    return (dx, dgain, dbias), (tol, n * U * (dy * xh).abs().sum(0) + 1e-44, n * U * dy.abs().sum(0) + 1e-44)


def w4(x, offsets, packs, group, dtype):
    """x [R, K], packs = [(q [E, K, N], s [E, groups, N])] (two: gated) -> y (nan in rows of no expert), bound.

    A group's sum may be taken as that of x (q + 8) and -8 times that of x, so its sizes are |x| (q + 16) s.  A multiply
    step adds 16 exact products and the running sum, each cut at the place of the largest: at most 17 * 2 U of those
    sizes a step; then G / 8 + 8 additions for the sum of x, one rounding a group, and at most 40 joins."""
    R, K = x.shape
    N = packs[0][0].shape[2]
    y = torch.full((R, N), math.nan, dtype=F8)
    tol = torch.zeros_like(y)
    count = 34 * group / 16 + group / 8 + 8 + 2 * math.ceil(K / group) + 40
    for e in range(len(offsets) - 1):
        r0, r1 = max(int(offsets[e]), 0), min(int(offsets[e + 1]), R)
        if r0 >= r1:
            continue
        xe = x[r0:r1].to(F8)
        v, dv = [], []
        for q, s in packs:
            se = s[e].to(F8).repeat_interleave(group, 0)[:K]
            v.append(xe @ (q[e].to(F8) * se))
            dv.append(count * U * (xe.abs() @ ((q[e].to(F8) + 16) * se.abs())))
        if len(packs) == 1:
            y[r0:r1], tol[r0:r1] = v[0], dv[0]
            continue
        a, da = v[0], dv[0]
        z = math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
        gelu = a / (1 + torch.exp(-2 * z))
        y[r0:r1] = gelu * v[1]
        # |gelu'| <= 1.13; z's few roundings come back 2 |z| times larger from the exponential
        tol[r0:r1] = (1.13 * da * (v[1].abs() + dv[1]) + gelu.abs() * dv[1]
                      + (8 * z.abs() + 8) * U * (gelu * v[1]).abs())
    return y, tol + half_ulp(y, dtype).nan_to_num(0.0) + 1e-44
