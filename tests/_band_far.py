"""A plain 64-bit form of the band attention from given scores, with bounds per row: for scores so
far from zero that a sum of exponentials cannot be kept in its logarithm (one log sum in 32 bits loses
the sum where the scores are of 10^6 or of the type's lowest value)."""
import torch

from _band import E32, HALF, TINY


def far_reference(q, k, v, g, s, es, scale, dtype, buckets=None):
    """Dict of values and bounds of out, gq, gk, gv and, with `buckets` (a bucket of every pair
    [Lq, Lk], and their number), gb.  q, k, v, g [N, L, H, D]; s [N, Hq, Lq, Lk]: the scores with their bias,
    -infinity where a key is not seen, as exact as the kernels have them but for errors of at most `es` each.

    A probability e^(s - m) / l is then off by 2 es (numerator and sum), e^x by (4 + |x|) e with |x| below 100
    where it counts, its sum and its products' sums of at most n terms by n e, and by half a step of the
    type for its product, as in _band.py; so are the rest of the roundings."""
    N, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1:3]
    G, u, tiny = Hq // Hk, HALF[dtype], TINY[dtype]
    half = u if dtype != "f32" else 0.0
    q, k, v, g = (t.double() for t in (q, k, v, g))
    kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    m = s.amax(-1, keepdim=True)
    x = (s - torch.where(m > -torch.inf, m, torch.zeros_like(m))).exp()
    p = x / x.sum(-1, keepdim=True).clamp_min(1e-300)
    see = (s > -torch.inf).double()
    n = E32 * (max(Lq * G, Lk) + 8)
    rp32 = 2 * es + (Lk + 116) * E32
    rp = rp32 + half
    low = 2.0 ** -25 if dtype == "f16" else 0.0  # fp16's last step, of probabilities relative to the row's largest
    out = torch.einsum("nhij,njhd->nihd", p, vv)
    pv = torch.einsum("nhij,njhd->nihd", rp * p + low * p.amax(-1, keepdim=True) * see, vv.abs())
    r = {"out": out, "out_tol": pv + 1.01 * u * out.abs() + tiny}
    head = lambda t: t.unflatten(2, (Hk, G)).sum(3)  # noqa: E731
    dp = torch.einsum("nihd,njhd->nhij", g, vv)
    dpa = torch.einsum("nihd,njhd->nhij", g.abs(), vv.abs())
    delta = (p * dp).sum(-1, keepdim=True)
    dd32 = (rp32 * (p * dp.abs()).sum(-1, keepdim=True) + (D + 2 + Lk) * E32 * (p * dpa).sum(-1, keepdim=True))
    dd = dd32 + (g.abs() * (r["out_tol"] + u * out.abs())).sum(-1).transpose(1, 2)[..., None]  # from a rounded out
    ds = p * (dp - delta)

    def eds(dd):
        return p * (dd + (D + 2) * E32 * dpa) + rp32 * p * (dp.abs() + delta.abs())
    e = eds(dd) + half * ds.abs() + n * ds.abs() + tiny
    r["gq"], r["gk"] = torch.einsum("nhij,njhd->nihd", ds, kk) * scale, head(torch.einsum("nhij,nihd->njhd", ds, q)) * scale
    r["gv"] = head(torch.einsum("nhij,nihd->njhd", p, g))
    r["gq_tol"] = torch.einsum("nhij,njhd->nihd", e, kk.abs()) * abs(scale) + 1.01 * u * r["gq"].abs() + tiny
    r["gk_tol"] = head(torch.einsum("nhij,nihd->njhd", e, q.abs())) * abs(scale) + 1.01 * u * r["gk"].abs() + tiny
    r["gv_tol"] = head(torch.einsum("nhij,nihd->njhd", (rp + n) * p + tiny * see, g.abs())) + 1.01 * u * r["gv"].abs() + tiny
    if buckets is not None:
        which, nb = buckets
        one = torch.zeros(Lq * Lk, nb, dtype=torch.float64)
        one[torch.arange(Lq * Lk), which.reshape(-1)] = 1.0
        gb = ds.sum(0).reshape(Hq, -1) @ one
        # delta is right to 32 bits here: what its rounding left is taken off where it adds up
        eb = (eds(dd32) + 4096 * E32 * ds.abs()).sum(0).reshape(Hq, -1) @ one
        r["gb"], r["gb_tol"] = gb.t(), (eb + 1.01 * u * gb.abs()).t() + tiny
    return r
