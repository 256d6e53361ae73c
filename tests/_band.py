"""Plain 64-bit forms of the band attention and of the query/key norm with
rotation, and elementwise bounds on what the kernels may differ from them by.

The bounds follow the roundings: u = 2^-8 (bf16), 2^-11 (fp16), 2^-24 (fp32) is
half a step of a value, e = 2^-24 that of the fp32 arithmetic.

Band forward: a score is a sum of D products and a bias in fp32, so it is off by
at most ds = (D + 4) e (scale |q|.|k| + |b|); with |s - m| up to a few hundred,
e^(s - m) adds (4 + |s - m|) e of itself.  The probabilities that meet the values
are rounded to the type once (16-bit types), relative to a running maximum that
may lag (no effect: a rounding is relative, but for fp16's steps of 2^-24 below 2^-14:
half of one off each probability relative to the row's largest, low = 2^-25 e^(max - lse)
sum |V| on out).  Sums of Lk terms in fp32: Lk e in
the worst case.  So each p is off by at most rp p with
    rp = u + 2 max_row(ds) + (Lk + 16 + spread) e,
out by rp (P |V|) + u |out| and lse by rp (without u) plus e |lse|.

Backward from the kernel's own rounded out: delta = g.out is off by
    dd = sum |g| (rp P|V| + u |out|) + D e sum |g||out|,
g.v by (D + 1) e |g|.|v|, so ds = p (g.v - delta) by
    eds = p (dd + D e |g||v|) + rp |ds|        (rp: p's own error, and ds rounded to
the type once more for its products), and the products and their final rounding
give, with n terms each,  gq: scale (eds |k|) + u |gq|, and likewise gk, gv, gb.
"""
import math

import torch

HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E32 = 2.0 ** -24
TINY = {"f32": 1e-37, "f16": 2.0 ** -24, "bf16": 1e-37}  # what the smallest steps of the type are off by


def seen_and_rel(N, Lq, Lk, left, right, sinks, q_start, q_len, k_len):
    i, j = torch.arange(Lq)[None, :, None], torch.arange(Lk)[None, None, :]
    start = torch.tensor(q_start if q_start is not None else [Lk - Lq] * N)[:, None, None]
    ql = torch.tensor(q_len if q_len is not None else [Lq] * N)[:, None, None].clamp(0, Lq)
    kl = torch.tensor(k_len if k_len is not None else [Lk] * N)[:, None, None].clamp(0, Lk)
    rel = j - (start + i)
    seen = (j < kl) & (i < ql)
    if left >= 0:
        seen = seen & ((-rel <= left) | (j < sinks))
    if right >= 0:
        seen = seen & (rel <= right)
    return seen.expand(N, Lq, Lk), rel.expand(N, Lq, Lk)


def reference(q, k, v, g=None, *, left=-1, right=-1, sinks=0, scale=None, bias=None, buckets=None, q_start=None,
              q_len=None, k_len=None, dtype="f32"):
    """Dict of 64-bit values and bounds: out, lse and, with g, gq, gk, gv, gb; tensors on the CPU."""
    N, Lq, Hq, D = q.shape
    Lk, Hk = k.shape[1:3]
    G = Hq // Hk
    scale = D ** -0.5 if scale is None else scale
    u = HALF[dtype]
    seen, rel = seen_and_rel(N, Lq, Lk, left, right, sinks, q_start, q_len, k_len)
    live_k, live_q = seen.any(1), seen.any(2)  # what nobody sees may hold anything
    q, k, v = q.double(), k.double(), v.double()
    q = torch.where(live_q[:, :, None, None], q, torch.zeros(()).double())
    k, v = (torch.where(live_k[:, :, None, None], t, torch.zeros(()).double()) for t in (k, v))
    kk, vv = k.repeat_interleave(G, 2), v.repeat_interleave(G, 2)
    s = torch.einsum("nihd,njhd->nhij", q, kk) * scale
    ds_ = torch.einsum("nihd,njhd->nhij", q.abs(), kk.abs()) * abs(scale)
    which = None
    if bias is not None:
        M, nb = buckets.numel() // 2, bias.shape[0]
        which = buckets.long()[rel.clamp(-M, M) + M]  # [N, Lq, Lk]
        ok = (which >= 0) & (which < nb)
        b = torch.where(ok[..., None], bias.double()[which.clamp(0, nb - 1)], torch.zeros(()).double())
        s = s + b.permute(0, 3, 1, 2)
        ds_ = ds_ + torch.where(torch.isfinite(b), b.abs(), torch.zeros(()).double()).permute(0, 3, 1, 2)
    see = seen[:, None].expand(N, Hq, Lq, Lk)
    s = torch.where(see, s, torch.full_like(s, -math.inf))
    lse = torch.logsumexp(s, -1) if Lk else torch.full((N, Hq, Lq), -math.inf, dtype=torch.float64)
    some = lse > -math.inf
    p = torch.where(some[..., None] & see, (s - torch.where(some, lse, torch.zeros(()).double())[..., None]).exp(), torch.zeros(()).double())
    fin = torch.where(see & (s > -math.inf), s, torch.zeros(()).double())
    spread = (fin.amax(-1) - fin.amin(-1)).amax() if s.numel() else torch.zeros(())
    ds_ = torch.where(p > 0, ds_, torch.zeros(()).double())
    err_s = ((D + 4) * E32 * ds_).amax(-1, keepdim=True) if Lk else torch.zeros(N, Hq, Lq, 1, dtype=torch.float64)
    rp32 = 2 * err_s + (Lk + 16 + float(spread)) * E32
    rp = rp32 + (u if dtype != "f32" else 0.0)
    tiny = TINY[dtype]
    pv = torch.einsum("nhij,njhd->nhid", p, vv.abs())
    out = torch.einsum("nhij,njhd->nihd", p, vv)
    r = {"out": out, "lse": lse}
    low = 0.0
    if dtype == "f16" and Lk:
        top = torch.where(some, s.amax(-1) - torch.where(some, lse, torch.zeros(()).double()), torch.zeros(()).double()).exp()
        low = 2.0 ** -25 * (top[..., None] * torch.einsum("nhij,njhd->nhid", see.double(), vv.abs())).transpose(1, 2)
    e_out = (rp * pv).transpose(1, 2) + low + u * out.abs() * 1.01 + tiny
    r["out_tol"] = e_out
    r["lse_tol"] = rp32[..., 0] * 1.01 + 4 * E32 * torch.where(some, lse.abs(), torch.zeros(()).double())
    if g is None:
        return r
    g = torch.where(live_q[:, :, None, None], g.double(), torch.zeros(()).double())
    ga = g.abs()
    dp = torch.einsum("nihd,njhd->nhij", g, vv)
    dpa = torch.einsum("nihd,njhd->nhij", ga, vv.abs())
    delta = (g * out).sum(-1).transpose(1, 2)[..., None]
    dd = ((ga * (e_out + u * out.abs())).sum(-1) + (D + 2) * E32 * (ga * out.abs()).sum(-1)).transpose(1, 2)[..., None]
    dsm = p * (dp - delta)
    eds32 = p * (dd + (D + 2) * E32 * dpa) + rp32 * p * (dp.abs() + delta.abs())
    eds = eds32 + (u if dtype != "f32" else 0.0) * dsm.abs() + tiny  # the rounding for the products
    n = E32 * (max(Lq * G, Lk) + 8)
    head = lambda t: t.unflatten(2, (Hk, G)).sum(3)  # noqa: E731
    gq = torch.einsum("nhij,njhd->nihd", dsm, kk) * scale
    gk = head(torch.einsum("nhij,nihd->njhd", dsm, q)) * scale
    gv = head(torch.einsum("nhij,nihd->njhd", p, g))
    r.update(gq=gq, gk=gk, gv=gv)
    r["gq_tol"] = torch.einsum("nhij,njhd->nihd", eds + n * dsm.abs(), kk.abs()) * abs(scale) + 1.01 * u * gq.abs() + tiny
    r["gk_tol"] = head(torch.einsum("nhij,nihd->njhd", eds + n * dsm.abs(), q.abs())) * abs(scale) + 1.01 * u * gk.abs() + tiny
    r["gv_tol"] = head(torch.einsum("nhij,nihd->njhd", (rp + n) * p + tiny, ga)) + 1.01 * u * gv.abs() + tiny
    if bias is not None:
        gb, eb = torch.zeros(nb, Hq).double(), torch.zeros(nb, Hq).double()
        idx = torch.where(ok, which, torch.full_like(which, nb)).reshape(-1)
        terms = N * Lq * Lk
        for h in range(Hq):
            d, e = dsm[:, h].reshape(-1), (eds32[:, h] + min(terms, 4096) * E32 * dsm[:, h].abs()).reshape(-1)
            gb[:, h] = torch.bincount(idx, weights=d, minlength=nb + 1)[:nb]
            eb[:, h] = torch.bincount(idx, weights=e, minlength=nb + 1)[:nb]
        r["gb"], r["gb_tol"] = gb, eb + 1.01 * u * gb.abs() + tiny
    return r


def check(name, got, ref, tol):
    """Every element within its bound; infinities equal."""
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{name}: infinities differ"
    d = torch.where(inf, torch.zeros(()).double(), (got - ref).abs())
    assert not torch.isnan(d).any(), f"{name}: NaN"
    bad = d > torch.where(inf, torch.ones(()).double(), tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside their bounds, worst "
                           f"{float((d / tol.clamp_min(1e-300))[bad].max()):.2f} times, first at {bad.nonzero()[0].tolist()}")


def rotate(y, cos, sin, R, interleaved):
    if not R:
        return y
    rot = y[..., :R]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :R // 2], rot[..., R // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([rot, y[..., R:]], -1)


def qknorm_reference(x, w, pos, inv_freq, interleaved, eps, dtype, g=None):
    """(out, its bound[, gx, bound, gw, bound]) of one side in 64 bits.  A norm is a sum of D squares, an
    rsqrt and products in fp32: (D / 2 + 8) e of itself; cos and sin of an fp32 angle below pi are off by
    4 e absolutely; then one rounding to the type."""
    D = x.shape[-1]
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    cos = sin = None
    if R:
        p = pos.double() if pos.dim() == 3 else pos.double()[..., None]
        axes = p.shape[-1]
        angle = (p.repeat_interleave(R // 2 // axes, -1) * inv_freq.double())[:, :, None]
        cos, sin = angle.cos(), angle.sin()
    u, tiny = HALF[dtype], TINY[dtype]
    x = x.double()
    w = torch.ones(D).double() if w is None else w.double()
    s = ((x * x).mean(-1, keepdim=True) + eps).rsqrt()
    y = x * s * w
    rel = (D / 2 + 8) * E32

    def amax(t):  # |a| + |b| of each pair, on both members
        t = t.abs()
        one = torch.ones(()).double()
        return rotate(t, one, -one, R, interleaved).abs().maximum(rotate(t, one, one, R, interleaved).abs()) if R else t
    out = rotate(y, cos, sin, R, interleaved)
    tol = (rel + 8 * E32) * amax(y) + 1.01 * u * out.abs() + tiny
    if g is None:
        return out, tol
    g = g.double()
    gy = rotate(g, cos, None if sin is None else -sin, R, interleaved)
    egy = 8 * E32 * amax(g)
    a, hat = gy * w, x * s
    mean = (a * hat).mean(-1, keepdim=True)
    gx = s * (a - hat * mean)
    em = ((egy * w.abs() + (rel + (D + 4) * E32) * a.abs()) * hat.abs()).mean(-1, keepdim=True)
    egx = s * (egy * w.abs() + rel * a.abs() + hat.abs() * (em + 3 * rel * mean.abs())) + 1.01 * u * gx.abs() + tiny
    gw = (gy * hat).sum((0, 1, 2))
    n = x[..., 0].numel()
    egw = ((egy + (rel + min(n, 2048) * E32) * gy.abs()) * hat.abs()).sum((0, 1, 2)) + 1.01 * u * gw.abs() + tiny
    return out, tol, gx, egx, gw, egw
