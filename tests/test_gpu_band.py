"""The dense attention over a band of keys (sinks, relative bias, caches) and the query/key
norm with rotation against 64-bit plain forms, elementwise, within the bounds of tests/_band.py."""
import math

import pytest
import torch

from _band import DTYPES, check, qknorm_reference, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def dcn():
    import deformable_convolution_sampling_b200 as d
    return d


def make(c, seed=0):
    """CPU tensors of a case, q, k and v as views of one packed projection where `packed`."""
    g = torch.Generator().manual_seed(seed + 17)
    dt = DTYPES[c["dtype"]]
    N, Lq, Lk, Hq, Hk, D = (c[x] for x in ("N", "Lq", "Lk", "Hq", "Hk", "D"))
    rand = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    if c.get("packed"):
        w = rand(N, Lk, (Hq + 2 * Hk) * D + 16)
        t = dict(q=w[..., :Hq * D].unflatten(-1, (Hq, D)), k=w[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)),
                 v=w[..., (Hq + Hk) * D:(Hq + 2 * Hk) * D].unflatten(-1, (Hk, D)))
    else:
        cache = c.get("cache", Lk)  # keys and values may be the first Lk tokens of longer caches
        t = dict(q=rand(N, Lq, Hq, D), k=rand(N, cache, Hk, D)[:, :Lk], v=rand(N, cache, Hk, D)[:, :Lk])
    t["g"] = rand(N, Lq, Hq, D)
    t["bias"] = t["buckets"] = None
    if c.get("nb"):
        t["bias"] = rand(c["nb"], Hq)
        t["buckets"] = torch.randint(0, c["nb"], (2 * c["M"] + 1,), generator=g, dtype=torch.int32)
    vec = lambda x: None if c.get(x) is None else torch.tensor(c[x], dtype=torch.int32)  # noqa: E731
    t.update(q_start=vec("q_start"), q_len=vec("q_len"), k_len=vec("k_len"))
    if c.get("poison"):  # what lies behind a sequence's lengths must not matter
        for n in range(N):
            if c.get("k_len") is not None:
                t["k"][n, max(0, c["k_len"][n]):] = math.nan
                t["v"][n, max(0, c["k_len"][n]):] = math.inf
            if c.get("q_len") is not None:
                t["q"][n, max(0, c["q_len"][n]):] = math.nan
                t["g"][n, max(0, c["q_len"][n]):] = math.nan
    return t


def run(dcn, c, t, backward=True):
    cu = {k: (None if v is None else v.cuda() if v.is_contiguous() else
              torch.empty_strided(v.shape, v.stride(), dtype=v.dtype, device="cuda").copy_(v)) for k, v in t.items()}
    more = {k: cu[k] for k in ("bias", "buckets", "q_start", "q_len", "k_len")}
    p = dcn.band_params_for(cu["q"], cu["k"], cu["v"], left=c.get("left", -1), right=c.get("right", -1),
                            sinks=c.get("sinks", 0), scale=c.get("scale"), **more)
    out, lse = dcn.band_forward(p, cu["q"], cu["k"], cu["v"], **more)
    grads = dcn.band_backward(p, cu["q"], cu["k"], cu["v"], out, lse, cu["g"], **more) if backward else ()
    assert dcn.dcn4_band_status() == 0
    return (out, lse) + tuple(grads)


def compare(dcn, c, t=None, backward=True):
    t = make(c) if t is None else t
    got = run(dcn, c, t, backward)
    r = reference(t["q"], t["k"], t["v"], t["g"] if backward else None, left=c.get("left", -1), right=c.get("right", -1),
                  sinks=c.get("sinks", 0), scale=c.get("scale"), bias=t["bias"], buckets=t["buckets"],
                  q_start=c.get("q_start"), q_len=c.get("q_len"), k_len=c.get("k_len"), dtype=c["dtype"])
    names = ["out", "lse"] + (["gq", "gk", "gv"] + (["gb"] if c.get("nb") else []) if backward else [])
    for name, x in zip(names, got):
        check(name, x, r[name], r[name + "_tol"])
    return got


def case(dtype, N, Lq, Lk, Hq, Hk, D, **more):
    return dict(dtype=dtype, N=N, Lq=Lq, Lk=Lk, Hq=Hq, Hk=Hk, D=D, **more)


CASES = [
    case("f32", 2, 5, 5, 2, 1, 4),
    case("f32", 2, 70, 70, 4, 2, 40, left=10, right=7, sinks=3, nb=8, M=16),
    case("f32", 1, 130, 200, 3, 3, 128, right=0),
    case("f16", 1, 1, 1, 1, 1, 8),
    case("bf16", 1, 1, 1, 4, 1, 128, nb=1, M=1),
    case("bf16", 2, 300, 300, 2, 2, 32),
    case("f16", 2, 129, 129, 2, 2, 24, right=0, packed=True),
    case("f16", 1, 257, 385, 3, 1, 80, left=100, right=20, sinks=5, nb=16, M=33),
    case("bf16", 2, 200, 200, 5, 1, 128, left=64, right=0, sinks=4, packed=True),
    case("bf16", 1, 513, 513, 2, 1, 64, left=127, right=0, sinks=1),
    case("bf16", 1, 640, 640, 1, 1, 128, left=130, right=130, sinks=2, nb=32, M=128),
    case("f16", 3, 150, 170, 4, 2, 56, q_start=[20, 0, -5], q_len=[150, 3, 140], k_len=[170, 131, 64], poison=True,
         nb=4, M=200),
    case("f16", 2, 100, 90, 2, 2, 16, q_start=[1 << 28, -(1 << 28)], left=5, right=9),     # most or all see nothing
    case("bf16", 3, 140, 260, 2, 1, 96, q_start=[120, 0, 50], q_len=[140, 0, 150], k_len=[260, 100, 0], poison=True,
         left=40, right=0, sinks=2),
    case("f16", 1, 7, 1000, 8, 2, 64, right=0, left=300, sinks=4, nb=12, M=64),
    case("bf16", 2, 3, 700, 6, 2, 48, cache=900, k_len=[700, 333], q_start=[697, 330], right=0, poison=True),
    case("f16", 1, 140, 140, 2, 1, 64, left=0, right=0),
    case("f16", 1, 140, 140, 2, 1, 64, left=0, right=5, sinks=140),
    case("bf16", 2, 64, 320, 2, 1, 112, scale=0.0),
    case("f16", 2, 50, 128, 4, 4, 40, scale=-0.3, nb=3, M=1024),
    case("bf16", 1, 160, 160, 24, 1, 64, right=0, nb=8, M=20),                              # many heads share a key head
    case("f16", 1, 9, 150, 256, 2, 16, right=0),                                            # a head group of 128
    case("f16", 70, 3, 20, 2, 2, 8, left=2, right=2),
    case("bf16", 1, 700, 700, 2, 1, 64, left=5, right=0, sinks=600),                        # most keys are sinks
    case("f16", 1, 1000, 1000, 2, 1, 32, left=40, right=0, sinks=3, nb=8, M=16),            # the sinks' tile is split
    case("f32", 1, 300, 300, 2, 1, 24, left=9, right=0, sinks=130, nb=4, M=40),
    case("bf16", 2, 30, 900, 6, 2, 72, nb=9, M=1000, left=800, right=100),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if not isinstance(v, list))[:70])
def test_band_matches_the_definition(dcn, c):
    compare(dcn, c)


DECODE = [
    case("bf16", 3, 1, 5000, 8, 2, 128, right=0, k_len=[5000, 1, 2777], q_start=[4999, 0, 2776], poison=True),
    case("f16", 2, 1, 4096, 8, 8, 64, left=1023, right=0, sinks=4, nb=32, M=512, k_len=[4096, 700],
         q_start=[4095, 699], poison=True),
    case("bf16", 1, 2, 9000, 16, 1, 64, right=0, cache=10000),
    case("f16", 2, 1, 3001, 5, 1, 72, right=0, nb=8, M=16),
    case("f32", 2, 1, 3000, 6, 2, 64, right=0, left=2000, sinks=1, nb=8, M=16),
    case("f16", 5, 4, 2000, 4, 1, 128, right=0, k_len=[2000, 64, 0, 65, 1999], q_start=[1996, 60, 0, 61, 1995]),
    case("bf16", 1, 1, 17, 64, 1, 128),
    case("f16", 1, 7, 6000, 20, 4, 96, right=0, left=4000, sinks=4),
    case("bf16", 2, 2, 4100, 40, 2, 64, right=0),
    case("bf16", 2, 1, 300, 17, 1, 64),                                                     # one row more than sixteen
    case("f16", 3, 2, 129, 8, 1, 40, left=70, right=3, sinks=2, nb=5, M=30, k_len=[129, 80, 129],
         q_start=[100, 10, 128], q_len=[2, 2, 1], poison=True),
    case("f16", 2, 1, 70, 2, 2, 8, nb=2, M=3),
    case("bf16", 2, 2, 500, 8, 1, 120, left=90, right=-1, q_start=[1 << 20, -70]),          # one sees nothing
]


@pytest.mark.parametrize("c", DECODE, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if not isinstance(v, list))[:70])
def test_few_tokens_over_a_cache(dcn, c):
    compare(dcn, c, backward=False)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_lowest_and_infinite_biases(dcn, dtype):
    """Buckets whose bias is the type's lowest value or -infinity: rows that see only such keys are uniform
    over the lowest ones, and empty (out 0, lse -infinity, gradients 0) over the infinite ones."""
    c = case(dtype, 1, 150, 150, 2, 1, 64, nb=4, M=100, left=60, right=60)
    t = make(c)
    low = torch.finfo(DTYPES[dtype]).min
    t["bias"] = torch.tensor([[low, -math.inf], [low, -math.inf], [low, -math.inf], [0.5, 0.25]]).to(DTYPES[dtype])
    t["buckets"] = torch.zeros(201, dtype=torch.int32)
    t["buckets"][130:140] = 3
    got = compare(dcn, c, t, backward=dtype != "f32")
    assert torch.isinf(got[1][0, 1]).any() and not torch.isinf(got[1][0, 0]).any()
    t["bias"][3] = t["bias"][0]
    got = compare(dcn, c, t)
    assert (got[0][0, :, 1] == 0).all() and (got[2][0, :, 1] == 0).all()


def test_bucket_entries_outside_the_table_mean_no_bias(dcn):
    c = case("f16", 1, 80, 80, 2, 2, 32, nb=4, M=10)
    t = make(c)
    t["buckets"][3], t["buckets"][12] = -1, 4
    compare(dcn, c, t)


def test_no_keys(dcn):
    c = case("bf16", 2, 9, 0, 2, 1, 32)
    out, lse, gq, gk, gv, _ = run(dcn, c, make(c))
    assert (out == 0).all() and (lse == -math.inf).all() and (gq == 0).all() and gk.numel() == 0 and gv.numel() == 0


@pytest.mark.parametrize("c", [CASES[7], CASES[10], CASES[11], DECODE[0]], ids=str)
def test_results_do_not_change_from_call_to_call(dcn, c):
    t = make(c)
    a, b = run(dcn, c, t), run(dcn, c, t)
    for x, y in zip(a, b):
        assert (x is None and y is None) or torch.equal(x, y)


def test_offsets_beyond_32_bits(dcn):
    """One token over a cache whose second image lies 2^32 elements behind the first."""
    far = 1 << 32
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * 2 * far:
        pytest.skip("needs 26 GB free")
    buf = torch.empty(far + 300 * 128, dtype=torch.float16, device="cuda")
    view = buf.as_strided((2, 300, 2, 64), (far, 128, 64, 1))
    c = case("f16", 2, 1, 300, 4, 2, 64, right=0)
    t = make(c)
    view.copy_(t["k"])
    q, v = t["q"].cuda(), t["v"].cuda()
    p = dcn.band_params_for(q, view, v, right=0)
    out, lse = dcn.band_forward(p, q, view, v)
    r = reference(t["q"], t["k"], t["v"], right=0, dtype="f16")
    check("out", out, r["out"], r["out_tol"])
    check("lse", lse, r["lse"], r["lse_tol"])


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_gradients_against_differences(dcn, dtype):
    """Directional derivatives of sum(g out) by central differences of the 64-bit form."""
    c = case(dtype, 1, 40, 40, 4, 2, 16, left=9, right=3, sinks=2, nb=6, M=12)
    t = make(c)
    grads = run(dcn, c, t)[2:]
    tol = reference(t["q"], t["k"], t["v"], t["g"], left=9, right=3, sinks=2, bias=t["bias"], buckets=t["buckets"], dtype=dtype)
    gen = torch.Generator().manual_seed(3)
    for name, key, got in (("q", "gq", grads[0]), ("k", "gk", grads[1]), ("v", "gv", grads[2]), ("bias", "gb", grads[3])):
        d = torch.randn(t[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-5

        def value(sign):
            m = {k: t[k].double() for k in ("q", "k", "v", "bias")}
            m[name] = m[name] + sign * h * d
            r = reference(m["q"], m["k"], m["v"], left=9, right=3, sinks=2, bias=m["bias"], buckets=t["buckets"])
            return float((t["g"].double() * r["out"]).sum())
        diff = (value(1) - value(-1)) / (2 * h)
        # the kernel's bound in this direction, and h^2 of the difference (third derivatives below 1e4 here)
        bound = float((tol[key + "_tol"] * d.abs()).sum()) + 1e4 * h * h
        assert abs(diff - float((got.double().cpu() * d).sum())) <= bound, (name, diff)


def test_autograd_layer_with_graph_replay(dcn):
    """The two operators as a layer uses them: packed projection, norms with rotation, banded attention with a
    bias; its gradients against the chain of the 64-bit forms, then captured in a CUDA graph and replayed on
    other inputs, forward and backward, bit for bit the eager call's."""
    N, L, Hq, Hk, D = 2, 150, 4, 2, 64
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    x, g = rand(N, L, (Hq + 2 * Hk) * D), rand(N, L, Hq, D)
    wq, wk, bias = rand(D), rand(D), rand(8, Hq)
    buckets = dcn.rel_buckets(8, 20)
    pos = torch.stack([torch.arange(L) % 12, torch.arange(L) // 12], -1).float().expand(N, L, 2).contiguous().cuda()
    inv = (100.0 ** (-torch.arange(8).double() / 8)).float().repeat(2).cuda()

    def layer(x, wq, wk, bias):
        q, k = x[..., :Hq * D].unflatten(-1, (Hq, D)), x[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
        v = x[..., (Hq + Hk) * D:].unflatten(-1, (Hk, D))
        q, k = dcn.qk_norm_rotate(q, k, wq, wk, pos, inv)
        return q, k, v, dcn.band_attention(q, k, v, left=40, right=40, sinks=2, bias=bias, buckets=buckets)

    def step(x, wq, wk, bias, g):
        leaves = [t.detach().requires_grad_(True) for t in (x, wq, wk, bias)]
        out = layer(*leaves)[-1]
        return (out.detach(),) + torch.autograd.grad(out, leaves, g)

    eager = step(x, wq, wk, bias, g)
    # the chain: the kernel's rounded q and k feed the definition
    q, k, v, _ = (t.detach() for t in layer(x, wq, wk, bias))
    r = reference(q.cpu(), k.cpu(), v.cpu(), g.cpu(), left=40, right=40, sinks=2, bias=bias.cpu(), buckets=buckets.cpu(), dtype="bf16")
    check("out", eager[0], r["out"], r["out_tol"])
    check("bias", eager[4], r["gb"], r["gb_tol"])
    check("v", eager[1][..., (Hq + Hk) * D:].unflatten(-1, (Hk, D)), r["gv"], r["gv_tol"])
    for name, lo, hi, H, w, i in (("q", 0, Hq, Hq, wq, 2), ("k", Hq, Hq + Hk, Hk, wk, 3)):
        up, xs = r["g" + name], x[..., lo * D:hi * D].unflatten(-1, (H, D)).cpu()
        ref = qknorm_reference(xs, w.cpu(), pos.cpu(), inv.cpu(), False, 1e-6, "bf16", up)
        # the upstream gradient itself is within its bound: the norm's backward is linear in it, and a
        # rotation and a projection move no more than sqrt(2) * 2 of it times weight and scale
        xd = xs.double()
        s = (xd.square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        spill = r[f"g{name}_tol"].amax(-1, keepdim=True) * 2 * w.double().cpu().abs().amax() * s * (1 + (xd * s).abs())
        check("g" + name, eager[1][..., lo * D:hi * D].unflatten(-1, (H, D)), ref[2], ref[3] + spill)
        spill_w = (r[f"g{name}_tol"].amax(-1, keepdim=True) * 1.5 * (xd * s).abs()).sum((0, 1, 2))
        check("gw" + name, eager[i], ref[4], ref[5] + spill_w)

    live = layer(*[t.detach().requires_grad_(True) for t in (x, wq, wk, bias)])  # an eager graph of other leaves lives on
    static = [t.clone() for t in (x, wq, wk, bias, g)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step(*static)
    for new in ((x, wq, wk, bias, g), (x.flip(1).contiguous(), wk, wq, -bias, g * 0.5)):
        for s, t in zip(static, new):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(replayed, step(*new)):
            assert torch.equal(a, b)
    assert live[-1].requires_grad


def test_two_streams_at_once(dcn):
    c = CASES[8]
    a, b = make(c, 1), make(c, 2)
    want = run(dcn, c, a), run(dcn, c, b)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for s, t in ((s1, a), (s2, b)):
        with torch.cuda.stream(s):
            cu = {k: t[k].cuda() for k in ("q", "k", "v", "g")}
            p = dcn.band_params_for(cu["q"], cu["k"], cu["v"], left=64, right=0, sinks=4)
            out, lse = dcn.band_forward(p, cu["q"], cu["k"], cu["v"])
            got.append((out, lse) + dcn.band_backward(p, cu["q"], cu["k"], cu["v"], out, lse, cu["g"]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x, y in zip(w[:5], g[:5]):
            assert torch.equal(x, y)


QK = [
    dict(dtype="f32", N=2, L=3, Hq=2, Hk=1, D=4, R=4),
    dict(dtype="f32", N=2, L=50, Hq=5, Hk=1, D=80, R=40, interleaved=True, far=5000),
    dict(dtype="f32", N=1, L=33, Hq=2, Hk=2, D=256, R=256, far=100000),
    dict(dtype="f16", N=1, L=1, Hq=1, Hk=1, D=8, R=8, axes=2),
    dict(dtype="bf16", N=3, L=1, Hq=32, Hk=8, D=128, R=128, far=100000),
    dict(dtype="f16", N=2, L=700, Hq=8, Hk=8, D=32, R=32, axes=2),
    dict(dtype="bf16", N=2, L=257, Hq=16, Hk=4, D=128, R=64, packed=True),
    dict(dtype="f16", N=2, L=63, Hq=3, Hk=1, D=104, R=52, axes=2, interleaved=True, packed=True),
    dict(dtype="bf16", N=1, L=19, Hq=4, Hk=0, D=256, R=6),
    dict(dtype="f16", N=1, L=19, Hq=0, Hk=3, D=48, R=0),
    dict(dtype="bf16", N=2, L=40, Hq=2, Hk=2, D=64, R=64, plain=True),
]


@pytest.mark.parametrize("c", QK, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_qknorm_matches_the_definition(dcn, c):
    g = torch.Generator().manual_seed(23)
    dt, axes = DTYPES[c["dtype"]], c.get("axes", 1)
    N, L, Hq, Hk, D, R = (c[x] for x in ("N", "L", "Hq", "Hk", "D", "R"))
    rand = lambda *s: torch.randn(*s, generator=g).to(dt)  # noqa: E731
    w = rand(N, L, (Hq + Hk) * D + (8 if c.get("packed") else 0)).cuda()
    q, k = w[..., :Hq * D].unflatten(-1, (Hq, D)), w[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D))
    if N * L and L > 2:
        w[0, 1] = 0  # a head of zeros: eps carries it
        w[0, 2] = 100 * w[0, 2]
    wq, wk = (None, None) if c.get("plain") else (rand(D).cuda(), rand(D).cuda())
    pos = inv = None
    if R:
        pos = (torch.randint(-c.get("far", 30), c.get("far", 30) + 1, (N, L, axes), generator=g).float()).cuda()
        pos[0, 0] += 0.25
        inv = (10000.0 ** (-torch.arange(R // 2).double() / (R // 2))).float().cuda()
    inter = c.get("interleaved", False)
    p = dcn.qknorm_params_for(q, k, wq, wk, pos, inv, interleaved=inter)
    outs = dcn.qknorm_forward(p, q, k, wq, wk, pos, inv)
    ups = rand(N, L, Hq, D).cuda(), rand(N, L, Hk, D).cuda()
    gq, gk, gwq, gwk = dcn.qknorm_backward(p, q, k, wq, wk, pos, inv, *ups)
    again = dcn.qknorm_backward(p, q, k, wq, wk, pos, inv, *ups)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    for x, wt, out, up, gx, gw in ((q, wq, outs[0], ups[0], gq, gwq), (k, wk, outs[1], ups[1], gk, gwk)):
        if not x.numel():
            continue
        r = qknorm_reference(x.cpu(), cpu(wt), cpu(pos), cpu(inv), inter, 1e-6, c["dtype"], up.cpu())
        check("out", out, r[0], r[1])
        check("gx", gx, r[2], r[3])
        if wt is not None:
            check("gw", gw, r[4], r[5])
        else:
            assert gw is None
    for a, b in zip((gq, gk, gwq, gwk), again):
        assert a is None or torch.equal(a, b)


def test_qknorm_gradients_against_differences(dcn):
    g = torch.Generator().manual_seed(29)
    f32 = dict(generator=g, dtype=torch.float32)
    x = torch.randn(2, 9, 3, 16, **f32)
    w, up = torch.randn(16, **f32), torch.randn(2, 9, 3, 16, **f32)
    pos, inv = torch.randint(0, 50, (2, 9, 1), generator=g).float(), torch.rand(6, **f32)
    leaves = [x.cuda().requires_grad_(True), w.cuda().requires_grad_(True)]
    out, _ = dcn.qk_norm_rotate(leaves[0], leaves[0].detach()[:, :, :1], leaves[1], None, pos.cuda(), inv.cuda())
    gx, gw = torch.autograd.grad(out, leaves, up.cuda())
    ref = qknorm_reference(x, w, pos, inv, False, 1e-6, "f32", up)
    for base, got, tol in ((0, gx, ref[3]), (1, gw, ref[5])):
        d = torch.randn(got.shape, generator=g, dtype=torch.float64)
        h = 1e-5
        val = []
        for sgn in (1, -1):
            a = [x.double(), w.double()]
            a[base] = a[base] + sgn * h * d
            val.append(float((qknorm_reference(a[0], a[1], pos, inv, False, 1e-6, "f32")[0] * up.double()).sum()))
        bound = float((tol * d.abs()).sum()) + 1e4 * h * h
        assert abs((val[0] - val[1]) / (2 * h) - float((got.double().cpu() * d).sum())) <= bound
