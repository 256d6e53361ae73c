"""The attention-layer operators that stand beside the deformable attention, as measured calls.

Two operators and the bias that one of them takes:

* ``qknorm``: an RMS norm of every query and key head and the position rotation, in one pass
  (the queries and keys are strided views of one packed projection);
* ``band``: dense attention over a band of keys (a sliding window) whose first tokens stay
  visible (sinks), with shared key heads, ragged batches and caches;
* ``band`` with ``nb > 0``: the same with a learned relative position bias by buckets, whose
  gradient the training direction returns.

``dir`` is "fwd" (the forward alone) or "train" (the forward, then the backward from a given
upstream gradient).  ``run`` computes the plain form in elementary torch operations, or, where
``own`` is true, calls the framework; ``exact`` gives the same values in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def _qk(name, dir, dtype, N, L, Hq, Hk, D, R, axes=1, interleaved=False, far=0):
    return dict(name=name, op="qknorm", dir=dir, dtype=dtype, N=N, L=L, Hq=Hq, Hk=Hk, D=D, R=R, axes=axes,
                interleaved=interleaved, far=far)


def _band(name, dir, dtype, N, Lq, Lk, Hq, Hk, D, left=-1, right=-1, sinks=0, nb=0, M=0, ragged=False):
    return dict(name=name, op="band", dir=dir, dtype=dtype, N=N, Lq=Lq, Lk=Lk, Hq=Hq, Hk=Hk, D=D, left=left,
                right=right, sinks=sinks, nb=nb, M=M, ragged=ragged)


def listed():
    return [
        # one new token of 16 sequences far into their caches: a call whose latency counts
        _qk("qknorm one token bf16", "fwd", "bf16", 16, 1, 32, 8, 128, 128, far=100000),
        # the queries and keys of a 64 x 64 map of 256 channels in 8 heads, rotated by (x, y)
        _qk("qknorm map f16", "fwd", "f16", 8, 4096, 8, 8, 32, 32, axes=2),
        # a training step with shared key heads and half of each head rotated
        _qk("qknorm train bf16", "train", "bf16", 4, 4096, 16, 4, 128, 64),
        # full precision, odd sizes, adjacent pairs rotated
        _qk("qknorm train odd f32", "train", "f32", 3, 1531, 5, 1, 80, 40, interleaved=True, far=5000),
        # self-attention among the 300 queries of a detection decoder
        _band("band queries bf16", "fwd", "bf16", 8, 300, 300, 8, 8, 32),
        # a 64 x 64 map in raster order: four rows of pixels either way, four register tokens, a learned bias
        _band("band map bias f16", "fwd", "f16", 8, 4096, 4096, 8, 8, 32, left=256, right=256, sinks=4, nb=32, M=128),
        # a long causal sequence with a sliding window and sinks
        _band("band long bf16", "fwd", "bf16", 1, 8192, 8192, 16, 4, 128, left=2047, right=0, sinks=4),
        # its training step
        _band("band train bf16", "train", "bf16", 2, 4096, 4096, 16, 4, 128, left=1023, right=0, sinks=4),
        # a ragged batch of 28 x 28 maps and a class token, every key visible, with the bias and its gradient
        _band("band train bias f16", "train", "f16", 16, 785, 785, 8, 8, 64, nb=32, M=128, ragged=True),
        # one token over long caches of differing lengths: bound by reading the cache
        _band("band decode bf16", "fwd", "bf16", 16, 1, 16384, 32, 8, 128, right=0, ragged=True),
        # one token over a short window of a cache, with the bias: a call whose latency counts
        _band("band decode window bias f16", "fwd", "f16", 4, 1, 4096, 8, 8, 64, left=1023, right=0, sinks=4, nb=32,
              M=512, ragged=True),
        # full precision, odd sizes, an uneven window
        _band("band train odd bias f32", "train", "f32", 2, 333, 333, 4, 2, 40, left=100, right=20, sinks=1, nb=16,
              M=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
    dir = rng.choice(["fwd", "train"])
    D = 8 * rng.randint(2, 16)
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 1, 2, 4, 5])
    if rng.random() < 0.35:
        L = _log(rng, 1, 8192)
        N = _log(rng, 1, max(1, min(64, 4 * 4096 * 20 * 128 // (L * (Hq + Hk) * D))))
        axes = rng.choice([1, 2])
        R = rng.choice([0, D // (2 * axes) * (2 * axes), max(1, D // (4 * axes)) * 2 * axes])
        return {k: v for k, v in _qk("", dir, dtype, N, L, Hq, Hk, D, R, axes, rng.random() < 0.5,
                                     rng.choice([0, 1000, 100000])).items() if k != "name"}
    kind = rng.choice(["self", "self", "cross", "decode"])
    most = 200 * 10**9 // 14 // (8 if dtype == "f32" else 1)  # every pair seen: the largest listed case's products
    if kind == "decode":
        dir, Lq, Lk = "fwd", rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 16, 16384)
        N = _log(rng, 1, max(1, min(32, 16 * 16384 * 8 * 128 // (Lk * Hk * D))))
    else:
        # a training step over a single key has gradients of zero, which only rounding fills
        Lk = min(_log(rng, 1 if dir == "fwd" else 2, 4096), math.isqrt(most // (Hq * D)))
        Lq = Lk if kind == "self" else min(_log(rng, 1, 2048), most // (Hq * D * Lk))
        N = _log(rng, 1, max(1, min(64, most // (Hq * Lq * Lk * D))))
    if kind == "cross":
        left = right = -1
        sinks = 0
    else:
        right = 0 if kind == "decode" else rng.choice([0, 0, -1, _log(rng, 1, Lk)])
        left = rng.choice([-1, _log(rng, 1, Lk)])
        sinks = rng.choice([0, 1, 4]) if left >= 0 else 0
    nb = rng.choice([0, 0, 8, 16, 32])
    M = rng.choice([16, 64, 128, 512]) if nb else 0
    return {k: v for k, v in _band("", dir, dtype, N, Lq, Lk, Hq, Hk, D, left, right, min(sinks, Lk), nb, M,
                                   rng.random() < 0.4).items() if k != "name"}


def _lengths(c):
    """Valid keys of each sequence of a ragged batch (a rule on its index)."""
    return [max(1, c["Lk"] - (n * 37 * max(1, c["Lk"] // 64)) % (c["Lk"] // 2 + 1)) for n in range(c["N"])]


def _starts(c):
    """Position of each sequence's first query: 0, or for a few tokens over a cache its last places."""
    if c["ragged"] and c["Lq"] == c["Lk"]:
        return [0] * c["N"]
    lens = _lengths(c) if c["ragged"] else [c["Lk"]] * c["N"]
    return [n - c["Lq"] for n in lens]


def _queries(c):
    return _lengths(c) if c["ragged"] and c["Lq"] == c["Lk"] else [c["Lq"]] * c["N"]


def _bucket_table(nb, M, both):
    """Bucket of every relative position j - p in -M..M: near distances one by one, far ones by their
    logarithm up to M; the keys behind a query have buckets of their own where it sees both sides."""
    half = nb // 2 if both else nb
    exact = max(1, half // 2)

    def of(d):
        if d < exact:
            return d
        return min(half - 1, exact + int(math.log(d / exact) / math.log(max(M, exact + 1) / exact) * (half - exact)))

    return [(half if both and r > 0 else 0) + (of(abs(r)) if both or r <= 0 else 0) for r in range(-M, M + 1)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, scale=1.0, shift=0.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale + shift).to(dt)

    N, Hq, Hk, D = c["N"], c["Hq"], c["Hk"], c["D"]
    s = {"case": c}
    if c["op"] == "qknorm":
        L, R = c["L"], c["R"]
        packed = normal(N, L, (Hq + 2 * Hk) * D, scale=1.5)
        s["q"] = packed[..., :Hq * D].unflatten(-1, (Hq, D))
        s["k"] = packed[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        s["wq"], s["wk"] = normal(D, scale=0.2, shift=1.0), normal(D, scale=0.2, shift=1.0)
        s["pos"] = s["inv_freq"] = None
        if R:
            base = torch.randint(0, c["far"] + 1, (N, 1), generator=g, device="cuda").float()
            t = torch.arange(L, device="cuda").float()
            if c["axes"] == 2:
                w = max(1, math.isqrt(L))
                s["pos"] = torch.stack([base + t % w, base + torch.floor(t / w)], -1)
            else:
                s["pos"] = (base + t)[..., None].contiguous()
            n = R // 2 // c["axes"]
            f = 10000.0 ** (-torch.arange(n, dtype=torch.float64, device="cuda") / n)
            s["inv_freq"] = f.float().repeat(c["axes"])
        if c["dir"] == "train":
            s["gq"], s["gk"] = normal(N, L, Hq, D), normal(N, L, Hk, D)
        return s
    Lq, Lk = c["Lq"], c["Lk"]
    s["q"], s["k"], s["v"] = normal(N, Lq, Hq, D), normal(N, Lk, Hk, D), normal(N, Lk, Hk, D)
    s["bias"] = s["buckets"] = s["q_start"] = s["q_len"] = s["k_len"] = None
    if c["nb"]:
        s["bias"] = normal(c["nb"], Hq)
        s["buckets"] = torch.tensor(_bucket_table(c["nb"], c["M"], c["right"] != 0), dtype=torch.int32, device="cuda")
    if c["ragged"]:
        s["k_len"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        s["q_len"] = torch.tensor(_queries(c), dtype=torch.int32, device="cuda")
        s["q_start"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
    if c["dir"] == "train":
        s["g"] = normal(N, Lq, Hq, D)
    return s


# --- the framework's calls ---

def _own_qknorm(s):
    import deformable_convolution_sampling_b200 as dcn
    c = s["case"]
    a = (s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["inv_freq"])
    p = dcn.qknorm_params_for(*a, interleaved=c["interleaved"], eps=EPS)
    out = dcn.qknorm_forward(p, *a)
    return out + dcn.qknorm_backward(p, *a, s["gq"], s["gk"]) if c["dir"] == "train" else out


def _own_band(s):
    import deformable_convolution_sampling_b200 as dcn
    c = s["case"]
    more = dict(bias=s["bias"], buckets=s["buckets"], q_start=s["q_start"], q_len=s["q_len"], k_len=s["k_len"])
    p = dcn.band_params_for(s["q"], s["k"], s["v"], left=c["left"], right=c["right"], sinks=c["sinks"], **more)
    out, lse = dcn.band_forward(p, s["q"], s["k"], s["v"], **more)
    if c["dir"] == "fwd":
        return out, lse
    return (out, lse) + dcn.band_backward(p, s["q"], s["k"], s["v"], out, lse, s["g"], **more)


# --- the plain forms ---

def _turn(y, cos, sin, R, interleaved):
    """Rotates the pairs of the first R entries: (i, i + R/2), or (2i, 2i + 1)."""
    if not R:
        return y
    rot, rest = y[..., :R], y[..., R:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :R // 2], rot[..., R // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    rot = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([rot, rest], -1)


def _angles(s):
    c = s["case"]
    if not c["R"]:
        return None, None
    n = c["R"] // 2 // c["axes"]
    angle = s["pos"].double().repeat_interleave(n, -1) * s["inv_freq"].double()  # [N, L, R/2], exact enough far out
    return angle.cos()[:, :, None].float(), angle.sin()[:, :, None].float()


def _plain_qknorm(s):
    c = s["case"]
    cos, sin = _angles(s)
    outs, grads, wgrads = [], [], []
    for x, w, up in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        xf, wf = x.float(), w.float()
        r = (xf.square().mean(-1, keepdim=True) + EPS).rsqrt()
        hat = xf * r
        outs.append(_turn(hat * wf, cos, sin, c["R"], c["interleaved"]).to(x.dtype))
        if up is not None:
            gy = _turn(up.float(), cos, None if sin is None else -sin, c["R"], c["interleaved"])
            wgrads.append((gy * hat).sum((0, 1, 2), dtype=torch.float64).to(x.dtype))
            gh = gy * wf
            grads.append((r * (gh - hat * (gh * hat).mean(-1, keepdim=True))).to(x.dtype))
    return tuple(outs + grads + wgrads)


def _seen(s):
    """[N, Lq, Lk] visible pairs and [N, Lq, Lk] relative positions key - query."""
    c, dev = s["case"], s["q"].device
    i, j = torch.arange(c["Lq"], device=dev), torch.arange(c["Lk"], device=dev)
    start = s["q_start"] if s["q_start"] is not None else torch.full((1,), c["Lk"] - c["Lq"], device=dev)
    rel = j[None, None, :] - (start[:, None, None] + i[None, :, None])
    seen = torch.ones_like(rel, dtype=torch.bool)
    if c["left"] >= 0:
        seen = seen & ((rel >= -c["left"]) | (j < c["sinks"]))
    if c["right"] >= 0:
        seen = seen & (rel <= c["right"])
    if s["k_len"] is not None:
        seen = seen & (j[None, None, :] < s["k_len"][:, None, None]) & (i[None, :, None] < s["q_len"][:, None, None])
    return seen, rel


def _plain_band(s):
    c = s["case"]
    N, Lq, Lk, Hq, Hk, D, G = c["N"], c["Lq"], c["Lk"], c["Hq"], c["Hk"], c["D"], c["Hq"] // c["Hk"]
    scale, dt = 1.0 / math.sqrt(D), s["q"].dtype

    def rows(t):  # [N, L, Hk * G, D] -> [N, Hk, G * L, D]
        return t.float().unflatten(2, (Hk, G)).permute(0, 2, 3, 1, 4).reshape(N, Hk, G * Lq, D)

    def back(t):  # [N, Hk, G * L, D] -> [N, L, Hq, D]
        return t.unflatten(2, (G, Lq)).permute(0, 3, 1, 2, 4).reshape(N, Lq, Hq, D)

    q, k, v = rows(s["q"]), s["k"].float().transpose(1, 2), s["v"].float().transpose(1, 2)
    seen, rel = _seen(s)
    x = (q @ k.transpose(2, 3) * scale).unflatten(2, (G, Lq))
    if c["nb"]:
        b = s["buckets"].long()[rel.clamp(-c["M"], c["M"]) + c["M"]]  # [N or 1, Lq, Lk]
        x += s["bias"].float()[b].permute(0, 3, 1, 2).unflatten(1, (Hk, G))
    hidden = ~seen[:, None, None]
    x = x.masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].reshape(N, Hq, Lq)
    prob = x.div_(torch.where(total == 0, torch.ones_like(total), total)).flatten(2, 3)
    out = back(prob @ v).to(dt)
    if c["dir"] == "fwd":
        return out, lse
    g = rows(s["g"])
    gv = (prob.transpose(2, 3) @ g).transpose(1, 2).to(dt)
    ds = g @ v.transpose(2, 3)
    ds = ds.sub_((ds * prob).sum(-1, keepdim=True)).mul_(prob)
    gq = back(ds @ k * scale).to(dt)
    gk = (ds.transpose(2, 3) @ q * scale).transpose(1, 2).to(dt)
    if not c["nb"]:
        return out, lse, gq, gk.contiguous(), gv.contiguous(), None
    per = ds.view(N, Hq, Lq, Lk)
    per = per.sum(0, keepdim=True, dtype=torch.float64) if b.shape[0] == 1 else per.double()
    per = per.permute(1, 0, 2, 3).reshape(Hq, -1)
    gb = torch.zeros(Hq, c["nb"], dtype=torch.float64, device=q.device).index_add_(1, b.reshape(-1), per)
    return out, lse, gq, gk.contiguous(), gv.contiguous(), gb.t().to(dt).contiguous()


def run(state):
    if state["case"]["op"] == "qknorm":
        return _own_qknorm(state) if own else _plain_qknorm(state)
    return _own_band(state) if own else _plain_band(state)


# --- what a pass cannot do without ---

def _pairs(c):
    """Visible (query, key) pairs of one head, over the batch."""
    n = 0
    for start, nq, nk in zip(_starts(c), _queries(c), _lengths(c) if c["ragged"] else [c["Lk"]] * c["N"]):
        p = torch.arange(start, start + nq)
        hi = (p + c["right"] + 1).clamp(0, nk) if c["right"] >= 0 else torch.full_like(p, nk)
        lo = (p - c["left"]).clamp(min=0) if c["left"] >= 0 else torch.zeros_like(p)
        n += int((hi - torch.minimum(lo, hi)).sum())
        if c["left"] >= 0:  # sinks before the window
            n += int(torch.minimum(torch.minimum(lo, hi), torch.full_like(p, c["sinks"])).sum())
    return n


def _keys(c):
    """Keys that some query sees, over the batch."""
    n = 0
    for start, nq, nk in zip(_starts(c), _queries(c), _lengths(c) if c["ragged"] else [c["Lk"]] * c["N"]):
        hi = min(nk, start + nq + c["right"]) if c["right"] >= 0 else nk
        lo = max(0, start - c["left"]) if c["left"] >= 0 else 0
        n += max(0, hi - lo) + (min(c["sinks"], lo, max(hi, 0)) if c["left"] >= 0 else 0)
    return n


def work(case):
    c = case
    b = 4 if c["dtype"] == "f32" else 2
    train = c["dir"] == "train"
    if c["op"] == "qknorm":
        n = c["N"] * c["L"] * (c["Hq"] + c["Hk"]) * c["D"]
        # inputs and outputs; the training direction reads the upstream gradient and writes the inputs' too
        return {"bytes": n * b * (4 if train else 2) + (c["N"] * c["L"] * c["axes"] * 4 if c["R"] else 0),
                "flops": n * (20 if train else 7)}
    nq, nk = sum(_queries(c)) * c["Hq"] * c["D"], _keys(c) * c["Hk"] * c["D"]
    return {"bytes": b * ((4 * nq + 4 * nk) if train else (2 * nq + 2 * nk)),
            "flops": (14 if train else 4) * c["D"] * c["Hq"] * _pairs(c)}


# --- the definition in 64 bits ---

def _exact_qknorm(s):
    c = s["case"]
    R, axes = c["R"], c["axes"]
    N, L, D = c["N"], c["L"], c["D"]
    turn = torch.eye(D, dtype=torch.float64, device=s["q"].device).expand(N, L, D, D).clone() if R else None
    outs, grads, wgrads = [], [], []
    if R:  # the rotation as a matrix of each token
        i = torch.arange(R // 2, device=s["q"].device)
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        angle = s["pos"].double()[:, :, i // (R // 2 // axes)] * s["inv_freq"].double()
        turn[:, :, first, first], turn[:, :, second, second] = angle.cos(), angle.cos()
        turn[:, :, first, second], turn[:, :, second, first] = -angle.sin(), angle.sin()
    for x, w, up in ((s["q"], s["wq"], s.get("gq")), (s["k"], s["wk"], s.get("gk"))):
        x, w = x.double(), w.double()
        size = ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt()
        y = x / size * w
        outs.append((turn @ y.transpose(2, 3)).transpose(2, 3) if R else y)
        if up is not None:
            gy = (turn.transpose(2, 3) @ up.double().transpose(2, 3)).transpose(2, 3) if R else up.double()
            wgrads.append((gy * x / size).sum((0, 1, 2)))
            a = gy * w
            grads.append(a / size - x * (a * x).sum(-1, keepdim=True) / (D * size ** 3))
    return tuple(outs + grads + wgrads)


def _exact_band(s):
    c = s["case"]
    N, Lq, Lk, Hq, D, G = c["N"], c["Lq"], c["Lk"], c["Hq"], c["D"], c["Hq"] // c["Hk"]
    dev = s["q"].device
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=dev)  # noqa: E731
    out, lse = new(N, Lq, Hq, D), torch.full((N, Hq, Lq), -math.inf, dtype=torch.float64, device=dev)
    gq, gk, gv, gb = new(N, Lq, Hq, D), new(N, Lk, c["Hk"], D), new(N, Lk, c["Hk"], D), new(max(1, c["nb"]), Hq)
    starts = _starts(c)
    nqs, nks = _queries(c), _lengths(c) if c["ragged"] else [Lk] * N
    for n in range(N):
        nq, nk = nqs[n], nks[n]
        at = starts[n] + torch.arange(nq, device=dev)[:, None]
        key = torch.arange(nk, device=dev)[None]
        seen = torch.ones(nq, nk, dtype=torch.bool, device=dev)
        if c["left"] >= 0:
            seen &= (at - key <= c["left"]) | (key < c["sinks"])
        if c["right"] >= 0:
            seen &= key - at <= c["right"]
        some = seen.any(-1)
        if c["nb"]:
            which = s["buckets"].long()[(key - at).clamp(-c["M"], c["M"]) + c["M"]]
        for h in range(Hq):
            q, k, v = s["q"][n, :nq, h].double(), s["k"][n, :nk, h // G].double(), s["v"][n, :nk, h // G].double()
            x = q @ k.t() / math.sqrt(D)
            if c["nb"]:
                x = x + s["bias"][:, h].double()[which]
            x = torch.where(seen, x, torch.full_like(x, -math.inf))
            l = torch.logsumexp(x, -1)
            lse[n, h, :nq] = l
            p = torch.where(some[:, None], (x - torch.where(some, l, torch.zeros_like(l))[:, None]).exp(), torch.zeros_like(x))
            o = p @ v
            out[n, :nq, h] = o
            if c["dir"] == "train":
                g = s["g"][n, :nq, h].double()
                t = p * (g @ v.t() - (g * o).sum(-1, keepdim=True))
                gq[n, :nq, h] = t @ k / math.sqrt(D)
                gk[n, :nk, h // G] += t.t() @ q / math.sqrt(D)
                gv[n, :nk, h // G] += p.t() @ g
                if c["nb"]:
                    gb[:, h] += torch.bincount(which.reshape(-1), weights=t.reshape(-1), minlength=c["nb"])
    if c["dir"] == "fwd":
        return out, lse
    return out, lse, gq, gk, gv, gb if c["nb"] else None


def exact(case, seed):
    c = case
    if c["op"] == "qknorm":
        if c["N"] * c["L"] * c["D"] ** 2 * 8 > 24e9:
            return None
        return _exact_qknorm(prepare(case, seed))
    if c["N"] * c["Hq"] > 1024:
        return None
    return _exact_band(prepare(case, seed))
