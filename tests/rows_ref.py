"""Plain 64-bit forms of the row operators (dispatch, combine, router gradient, norms around a
block) with, beside each result, a bound on what fp32 arithmetic may add to it.

The bounds. One fp32 operation is off by at most U = 2^-24 relative (rsqrtf, at most 2 ulp, by 4U).
A sum of n terms is off by at most n_chain * U * (sum of the terms' absolute values), where n_chain
is the longest chain of additions: a thread adds at most 8 values per chunk (16 with two chunks)
and two warp trees of 5 steps follow, so at most 26 for a sum over a row. Relative errors of factors
add up. A result stored in a type t is off by another finfo(t).eps / 2 relative, or half a
smallest subnormal. `mag` arrays are the results with every term replaced by its absolute value.
"""
import torch

U = 2.0 ** -24
ROW_SUM = 26                       # longest chain of additions of a sum over a row
R = ROW_SUM / 2 + 6                # 1/sqrt(mean + eps): half the sum's error, divide, add, rsqrtf


def stored(ref, dtype):
    """Bound of the rounding to dtype."""
    f = torch.finfo(dtype)
    return ref.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def check(got, ref, arith, what=""):
    """|got - ref| <= arith + the rounding of ref (and of its error) to got's type."""
    got, ref, arith = got.detach().cpu(), ref.detach().cpu().double(), torch.as_tensor(arith).cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    lim = arith + stored(ref.abs() + arith, got.dtype)
    off = (got.double() - ref).abs()
    bad = off > lim
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((off / lim.clamp(min=1e-300)).max()):.3g} of the bound")


def sort(idx, E):
    """counts, offsets, perm (kept pairs only), inv (-1: dropped) of int [T][k]."""
    e = idx.reshape(-1).tolist()
    lists = [[] for _ in range(E)]
    for p, x in enumerate(e):
        if 0 <= x < E:
            lists[x].append(p)
    perm = [p for ps in lists for p in ps]
    inv = [-1] * len(e)
    for n, p in enumerate(perm):
        inv[p] = n
    offsets = [0]
    for ps in lists:
        offsets.append(offsets[-1] + len(ps))
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)
    return as_int([len(ps) for ps in lists]), as_int(offsets), as_int(perm), as_int(inv).view(idx.shape)


def combine(yp, inv, wts):
    """(out, arithmetic bound): k products and k additions per value."""
    T, k = inv.shape
    y = yp.double()
    P = y.shape[0]
    ok = (inv >= 0) & (inv < P)
    rows = torch.where(ok[:, :, None], y[inv.clamp(0, P - 1).long()], 0.0)
    w = torch.ones(T, k, dtype=torch.float64) if wts is None else wts.double()
    out = (rows * w[:, :, None]).sum(1)
    mag = (rows.abs() * w.abs()[:, :, None]).sum(1)
    return out, (k + 1) * U * mag


def combine_backward(dout, yp, inv, wts):
    """(dyp with NaN in rows nothing points to, its bound, dwts, its bound)."""
    T, k = inv.shape
    d, y, w = dout.double(), yp.double(), wts.double()
    H = d.shape[1]
    dyp = torch.full_like(y, float("nan"))
    dw, mag = torch.zeros(T, k, dtype=torch.float64), torch.zeros(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            p = int(inv[t, j])
            if 0 <= p < y.shape[0]:
                dyp[p] = w[t, j] * d[t]
                dw[t, j] = d[t] @ y[p]
                mag[t, j] = d[t].abs() @ y[p].abs()
    # a thread adds 8 products per 2048-wide chunk of the row
    chain = 8 * -(-H // 2048) + 11
    return dyp, U * dyp.abs(), dw, chain * U * mag


def router_backward(idx, wts, dwts, E):
    T, k = idx.shape
    w, d = wts.double(), dwts.double()
    mean, mag_mean = (w * d).sum(1, keepdim=True), (w * d).abs().sum(1, keepdim=True)
    z, mag = w * (d - mean), w.abs() * (d.abs() + mag_mean)
    out, bound = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for j in range(k):
        for t in range(T):
            e = int(idx[t, j])
            if 0 <= e < E:
                out[t, e] += z[t, j]
                bound[t, e] += mag[t, j]
    # the mean: up to k/32 + 1 products per lane and a tree of 5; difference, product, up to k adds
    return out, (k / 32 + 8 + 2 + k) * U * bound


def rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def norm_pre(h, w, eps):
    h = h.double()
    x = h * rms(h, eps) * (1.0 if w is None else w.double())
    return x, (R + 2) * U * x.abs()


def norm_post(y, h, eps, alpha, norm_y, w, gate, w_next, next_, y_err=None):
    """(h_out, bound, x_next, bound). y_err: error already in y (the fused combine)."""
    y, h = y.double(), h.double()
    y_err = torch.zeros_like(y) if y_err is None else y_err
    one = torch.ones((), dtype=torch.float64)
    wd, g = one if w is None else w.double(), one if gate is None else gate.double()
    if norm_y:
        q = rms(y, eps)
        u = y * q * wd
        # y's own error, its effect on q, and the arithmetic
        u_err = wd.abs() * q * (y_err + y.abs() * q * q * (y.abs() * y_err).mean(1, keepdim=True)) \
            + (R + 2) * U * u.abs()
    else:
        u, u_err = y, y_err
    out = alpha * h + g * u
    err = g.abs() * u_err + 3 * U * ((alpha * h).abs() + (g * u).abs())
    if not next_:
        return out, err, None, None
    wn = one if w_next is None else w_next.double()
    r = rms(out, eps)
    x = out * r * wn
    x_err = wn.abs() * r * (err + out.abs() * r * r * (out.abs() * err).mean(1, keepdim=True)) + (R + 2) * U * x.abs()
    return out, err, x, x_err


def rms_backward(d, v, w, eps):
    """Towards v and (per row) w, with the magnitudes of their terms."""
    r = rms(v, eps)
    n = v * r
    dn = d if w is None else d * w
    m, mag_m = (dn * n).mean(1, keepdim=True), (dn * n).abs().mean(1, keepdim=True)
    return r * (dn - n * m), d * n, r * (dn.abs() + n.abs() * mag_m), n


# roundings in one rms_backward: r three times (in n twice and outside), the sum, six products
BACK = 3 * R + ROW_SUM + 6


def column_chain(T):
    """Longest chain of a sum over the tokens: a block's rows, its run of at most 19 blocks of 2368, the
    joining of the runs. The backward pass has at least min(T, 100) blocks."""
    return -(-T // min(T, 100)) + 19 + 32


def norm_pre_backward(dx, h, w, eps, dres):
    d, v = dx.double(), h.double()
    wd = None if w is None else w.double()
    dh, dw, mag, n = rms_backward(d, v, wd, eps)
    if dres is not None:
        dh, mag = dh + dres.double(), mag + dres.double().abs()
    T = h.shape[0]
    return dh, (BACK + 2) * U * mag, dw.sum(0), (R + 2 + column_chain(T)) * U * dw.abs().sum(0)


def norm_post_backward(dh_out, y, eps, alpha, norm_y, w, gate, h_out, w_next, dx_next):
    """dict of name -> (gradient, bound)."""
    d, y = dh_out.double(), y.double()
    T, H = y.shape
    mag = d.abs()
    out = {}
    if dx_next is not None:
        wn = None if w_next is None else w_next.double()
        dn, dwn, mag_n, _ = rms_backward(dx_next.double(), h_out.double(), wn, eps)
        d, mag = d + dn, mag + mag_n
        out["dw_next"] = dwn.sum(0), (R + 2 + column_chain(T)) * U * dwn.abs().sum(0)
    c = BACK + 2                                     # errors of d, in units of U * mag
    out["dh"] = alpha * d, (c + 1) * U * abs(alpha) * mag
    one = torch.ones((), dtype=torch.float64)
    wd, g = one if w is None else w.double(), one if gate is None else gate.double()
    if norm_y:
        n = y * rms(y, eps)
        u = n * wd
    else:
        n = u = y
    du, mag_du = g * d, g.abs() * mag
    cu = c + R + 3                                   # d u and du n: n's statistics and the products
    if gate is not None:
        dg, mag_g = d * u, mag * u.abs()
        if gate.dim() == 1:
            out["dgate"] = dg.sum(0), (cu + column_chain(T)) * U * mag_g.sum(0)
        elif gate.shape[1] == 1 and H > 1:
            out["dgate"] = dg.sum(1, keepdim=True), (cu + ROW_SUM) * U * mag_g.sum(1, keepdim=True)
        else:
            out["dgate"] = dg, cu * U * mag_g
    if norm_y:
        dy, dw, _, _ = rms_backward(du, y, wd, eps)
        q = rms(y, eps)
        mag_y = q * (wd.abs() * mag_du + n.abs() * (wd.abs() * mag_du * n.abs()).mean(1, keepdim=True))
        out["dy"] = dy, (cu + BACK + 2) * U * mag_y
        out["dw"] = dw.sum(0), (cu + column_chain(T)) * U * (mag_du * n.abs()).sum(0)
    else:
        out["dy"] = du, (c + 1) * U * mag_du
    return out
