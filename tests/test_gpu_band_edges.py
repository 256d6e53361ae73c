"""The band attention and the query/key norm where they can go wrong beyond the sizes of
tests/test_gpu_band.py: scores far from zero, non-finite inputs, large head groups, units of
several tokens, gradients that are not wanted.  References are plain 64-bit forms; each bound is
derived where it is used."""
import pytest
import torch

from _band import E32, check
from _band_far import far_reference
from test_gpu_band import DTYPES, case, compare, dcn, make, run  # noqa: F401  (dcn is a fixture)
from test_gpu_band import test_qknorm_matches_the_definition as qknorm_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


# One active key tile a half in grad_q's second pass over the keys: nothing but the kernel's own barriers
# orders the exchange of a row's sum before it and the one behind it.
ONE_TILE = [
    case("f16", 2, 200, 60, 4, 4, 64),                       # 60 keys
    case("bf16", 1, 512, 512, 8, 2, 128, right=0),           # the first CTAs of a causal band with shared heads
    case("f16", 1, 300, 300, 4, 1, 32, right=0, nb=8, M=16),
]


# Rings of two and three slots with many tiles behind them: grad_q's halves may be as far apart as the ring.
RINGS = [
    case("bf16", 1, 700, 700, 4, 2, 128, nb=8, M=16),
    case("f16", 2, 300, 900, 4, 4, 72, left=500, right=0),
]


@pytest.mark.parametrize("c", ONE_TILE + RINGS, ids=str)
def test_order_within_grad_q(dcn, c):  # noqa: F811
    """Equal to the definition and the same from call to call."""
    t = make(c, 3)
    first = compare(dcn, c, t)
    for _ in range(20):
        for x, y in zip(first, run(dcn, c, t)):
            assert x is y is None or torch.equal(x, y)


def far_compare(dcn, c, t, s, es, names, loose=1.0):  # noqa: F811
    """run(c, t) against far_reference; the bounds must be below the values, or they would say nothing."""
    M = c.get("M", 0)
    buckets = None
    if c.get("nb"):
        rel = torch.arange(c["Lk"])[None] - (c["Lk"] - c["Lq"] + torch.arange(c["Lq"])[:, None])
        buckets = t["buckets"].long()[rel.clamp(-M, M) + M], c["nb"]
    scale = c["D"] ** -0.5 if c.get("scale") is None else c["scale"]
    r = far_reference(t["q"], t["k"], t["v"], t["g"], s, es, scale, c["dtype"], buckets)
    got = dict(zip(("out", "lse", "gq", "gk", "gv", "gb"), run(dcn, c, t)))
    for name in names:
        part = r[name + "_tol"].median() / r[name].abs().mean()
        assert part < loose, f"{name}: a bound of {float(part):.2f} of the values says nothing"
        check(name, got[name], r[name], r[name + "_tol"])
    return got, r


def rel_of(c):
    return torch.arange(c["Lk"])[None] - (c["Lk"] - c["Lq"] + torch.arange(c["Lq"])[:, None])


# Scores of about 2^20 that differ by a few: products, scores and biases are exact in 32 bits (whole numbers and
# quarters), so that only what is done with them is at stake.
COMMON = [dict(Lq=150, Lk=150, Hq=2, Hk=1, D=64), dict(Lq=64, Lk=900, Hq=2, Hk=2, D=128), dict(Lq=40, Lk=60, Hq=4, Hk=2, D=32),
          dict(Lq=300, Lk=300, Hq=2, Hk=1, D=64, nb=4, M=16), dict(Lq=130, Lk=130, Hq=24, Hk=1, D=40, nb=4, M=16)]


def common_part(dtype, i, c=None, sign=1):
    """A case (of COMMON), its tensors and its scores."""
    c = case(dtype, 1, scale=0.25 * sign, right=0, **(c or COMMON[i]))
    t = make(c, i)
    gen = torch.Generator().manual_seed(i)
    for x in ("q", "k"):
        t[x] = torch.randint(-1, 2, t[x].shape, generator=gen).to(t[x].dtype)
        t[x][..., 0] = 2048.0 if x == "q" else 2048.0 * sign
    b = 0.0
    if c.get("nb"):
        t["bias"] = torch.randint(-8, 9, t["bias"].shape, generator=gen).to(t["bias"].dtype) / 4
        b = t["bias"].double()[t["buckets"].long()[rel_of(c).clamp(-c["M"], c["M"]) + c["M"]]].permute(2, 0, 1)
    kk = t["k"].double().repeat_interleave(c["Hq"] // c["Hk"], 2)
    s = torch.einsum("nihd,njhd->nhij", t["q"].double(), kk) * c["scale"] + b
    return c, t, torch.where(rel_of(c) <= 0, s, torch.full_like(s, -torch.inf))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(COMMON)))
def test_scores_with_a_large_common_part(dcn, dtype, i):  # noqa: F811
    """Differences of scores are below 100, and formed to 32 bits."""
    c, t, s = common_part(dtype, i)
    far_compare(dcn, c, t, s, 100 * E32, ["out"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i,sign", [(i, 1) for i in range(len(COMMON))] + [(0, -1), (3, -1)])
def test_gradients_of_scores_with_a_large_common_part(dcn, dtype, i, sign):  # noqa: F811
    """One log sum in 32 bits is off by 0.06 at 2^20.  (The first entries of q and k, 2048, have their gradients
    from sums that cancel: bounds above the values, as they are 2048 times the rest's.)"""
    c, t, s = common_part(dtype, i, sign=sign)
    got, r = far_compare(dcn, c, t, s, 100 * E32, ["gv"] + (["gb"] if c.get("nb") else []))
    for name in ("gq", "gk"):
        tol, ref = r[name + "_tol"], r[name]
        assert tol[..., 1:].median() < ref[..., 1:].abs().mean()
        check(name, got[name], ref, tol)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("c", [dict(Lq=1, Lk=3000, Hq=4, Hk=2, D=64), dict(Lq=2, Lk=200, Hq=4, Hk=1, D=128), dict(Lq=40, Lk=5000, Hq=2, Hk=2, D=64)], ids=str)
def test_few_rows_with_scores_of_a_large_common_part(dcn, dtype, c):  # noqa: F811
    c, t, s = common_part(dtype, 9, c)
    far_compare(dcn, c, t, s, 100 * E32, ["out"])


# Many rows with and without split keys, both halves on the same rows, few rows with and without split keys, fp32.
NAN = [case("bf16", 1, 300, 300, 2, 1, 64), case("f16", 1, 40, 2000, 2, 2, 128), case("f16", 1, 60, 60, 2, 1, 32),
       case("bf16", 2, 1, 3000, 4, 2, 64), case("f16", 1, 2, 100, 4, 2, 128), case("f16", 600, 1, 70, 2, 2, 64), case("f32", 1, 70, 100, 2, 2, 32),
       case("bf16", 1, 200, 200, 2, 1, 64, nb=4, M=8)]


@pytest.mark.parametrize("c", NAN, ids=str)
def test_nan_reaches_the_rows_that_see_it(dcn, c):  # noqa: F811
    """A NaN in a query reaches its rows, one in a key that everybody sees everything, of its heads."""
    t = make(c)
    t["q"][0, 0, 0, 3] = torch.nan
    out, lse, gq = run(dcn, c, t)[:3]
    for x in (out[0, 0, 0], lse[0, 0, 0], gq[0, 0, 0]):
        assert x.isnan().all()
    assert c["Lq"] == 1 or not lse[0, 0, 1:].isnan().any()
    assert not out[:, :, 1].isnan().any() and not lse[:, 1].isnan().any()
    t = make(c)
    t["k"][0, c["Lk"] // 2, 0, 1] = torch.nan
    out, lse, gq = run(dcn, c, t)[:3]
    for x in (out[0, :, 0], lse[0, 0], gq[0, :, 0]):
        assert x.isnan().all()
    assert c["Hk"] == 1 or not lse[:, -1].isnan().any()
    t = make(c)
    t["v"][0, c["Lk"] - 1, 0, 2] = torch.inf
    out, lse = run(dcn, c, t)[:2]
    assert not out[0, :, 0, 2].isfinite().any() and lse.isfinite().all()


def test_a_value_that_no_query_sees_may_not_be_finite_behind_k_len(dcn):  # noqa: F811
    """Infinities ahead of a token are kept out by k_len."""
    c = case("bf16", 2, 1, 200, 4, 2, 64, right=0, k_len=[150, 77], q_start=[149, 76], poison=True)
    compare(dcn, c, backward=False)


# Rows that see only keys with the type's lowest bias: uniform over them.  Few keys and many (grad_q goes over the
# keys once or twice), heads of up to 64 and up to 128, a head group of 24.
LOWEST = [dict(Lq=150, Lk=150, Hq=2, Hk=1, D=64, left=60, right=60), dict(Lq=900, Lk=900, Hq=2, Hk=2, D=32),
          dict(Lq=70, Lk=700, Hq=2, Hk=1, D=128), dict(Lq=130, Lk=130, Hq=24, Hk=1, D=40)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("i", range(len(LOWEST)))
def test_rows_of_lowest_biases(dcn, dtype, i):  # noqa: F811
    c = case(dtype, 1, nb=4, M=100, **LOWEST[i])
    t = make(c, i)
    low = torch.finfo(DTYPES[dtype]).min
    t["bias"] = torch.full((4, c["Hq"]), low, dtype=DTYPES[dtype])
    t["bias"][3] = 0.5
    t["buckets"] = torch.zeros(201, dtype=torch.int32)
    t["buckets"][130:140] = 3
    rel = rel_of(c)
    seen = (-rel <= c.get("left", 10**9)) & (rel <= c.get("right", 10**9))
    normal = seen & (rel >= 30) & (rel < 40)
    D = c["D"]
    kk = t["k"].double().repeat_interleave(c["Hq"] // c["Hk"], 2)
    x = torch.einsum("nihd,njhd->nhij", t["q"].double(), kk) * D ** -0.5
    # beside a key of another bucket the lowest ones vanish; on their own, fp16's keep their scores (2^-9 of
    # rounding each at 65504, and the products'), the other types' scores all are the lowest value itself
    flat = torch.zeros_like(x) if dtype != "f16" else x
    s = torch.where(normal, x, torch.where(normal.any(-1, keepdim=True), torch.full_like(x, -torch.inf), flat))
    s = torch.where(seen, s, torch.full_like(x, -torch.inf))
    es = (D + 4) * E32 * 60 + (2.0 ** -9 if dtype == "f16" else 0.0)  # sum |q k| / sqrt(D) is below 60 here
    assert float(torch.einsum("nihd,njhd->nhij", t["q"].double().abs(), kk.abs()).amax()) * D ** -0.5 < 60
    got, r = far_compare(dcn, c, t, s, es, ["out", "gq", "gk", "gv"])
    # 0 but for rounding: all keys that count in a row are of one bucket
    check("gb", got["gb"], r["gb"], r["gb_tol"])
    last = got["out"][0, -1, 0].double().cpu()  # sees no key of bucket 3
    if dtype != "f16":
        mean = t["v"][0, seen[-1], 0].double().mean(0)
        # |out| is below 1, and a probability off by half a step, of |v| below 5
        assert float(mean.abs().max()) < 1 and ((last - mean).abs() <= 4 * torch.finfo(DTYPES[dtype]).eps).all()


# Groups whose heads' bias tables fit shared memory together, and groups whose do not.
GROUPS = [dict(Hq=2, Hk=1, M=32), dict(Hq=16, Hk=1, M=128), dict(Hq=16, Hk=2, M=512), dict(Hq=4, Hk=1, M=1024), dict(Hq=128, Hk=1, M=64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("i", range(len(GROUPS)))
def test_bias_gradient_does_not_take_up_the_rounding_of_out(dcn, dtype, i):  # noqa: F811
    """Values of 1 and the next number above it, a quarter of them the latter, and uniform probabilities: out
    rounds down by a quarter of a step in every row, and delta from it would be off by the same amount in all of
    them: a sum of over a hundred times what the bias gradient may be off by."""
    # (few keys for fp16, whose steps are near those of fp32 sums over many)
    c = case(dtype, 1, 600, 150 if dtype == "f16" else 600, D=64, nb=4, **GROUPS[i])
    t = make(c, i)
    t["q"].zero_()
    t["bias"].zero_()
    t["v"][:] = 1.0
    t["v"][:, ::4] = 1 + torch.finfo(DTYPES[dtype]).eps
    t["g"][:] = 1.0
    s = torch.zeros(1, c["Hq"], c["Lq"], c["Lk"], dtype=torch.float64)
    which = t["buckets"].long()[rel_of(c).clamp(-c["M"], c["M"]) + c["M"]]
    r = far_reference(t["q"], t["k"], t["v"], t["g"], s, 0.0, 64 ** -0.5, dtype, (which, c["nb"]))
    share = torch.bincount(which.reshape(-1), minlength=c["nb"]) / c["Lk"]  # rows' probabilities in each bucket
    off = 64 * torch.finfo(DTYPES[dtype]).eps / 4 * share[:, None]  # what a rounded out would add, about
    assert (r["gb_tol"] < off / 2).all()
    check("gb", run(dcn, c, t)[5], r["gb"], r["gb_tol"])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("c", [dict(Lq=300, Lk=300, Hq=16, Hk=1, D=64, M=128, right=0), dict(Lq=200, Lk=333, Hq=16, Hk=2, D=80, M=512, left=100, right=50, sinks=3),
                               dict(Lq=700, Lk=130, Hq=6, Hk=1, D=128, M=1024, q_len=[700, 333], k_len=[130, 97], poison=True),
                               dict(Lq=9, Lk=70, Hq=128, Hk=1, D=16, M=100), dict(Lq=65, Lk=40, Hq=25, Hk=1, D=32, M=100)], ids=str)
def test_large_groups_with_a_bias(dcn, dtype, c):  # noqa: F811
    c = case(dtype, 2, nb=12, **c)
    a, b = compare(dcn, c), run(dcn, c, make(c))
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_more_heads_than_a_grid_has_rows(dcn):  # noqa: F811
    compare(dcn, case("f16", 1, 2, 3, 70000, 70000, 8, nb=2, M=1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_the_angle_beyond_32_bits(dcn, interleaved):  # noqa: F811
    """A head (2, 0, 0, 0) has a norm of 1 and comes out as 2 cos f and 2 sin f, f near +-pi.  sincosf is good to
    2 steps (2^-22 of a value at most) and a sum behind it to half of one: 2.5 * 2^-23.  An angle held in 32 bits
    alone is off by up to 2^-23, which is 2^-23 / sin f of the sine: up to ten times as much here."""
    pos = torch.arange(100000, dtype=torch.float64)
    f = torch.remainder(pos + torch.pi, 2 * torch.pi) - torch.pi
    pos = pos[(f.abs() > 2.9) & (f.abs() < 3.1)].float().cuda()[None]
    L = pos.shape[1]
    x = torch.zeros(1, L, 2, 4, dtype=torch.float32, device="cuda")
    x[..., 0] = 2.0
    inv = torch.tensor([1.0, 0.5], dtype=torch.float32, device="cuda")
    a = (x, x[:, :, :1].contiguous(), None, None, pos, inv)
    p = dcn.qknorm_params_for(*a, interleaved=interleaved, eps=1e-30)
    out, _ = dcn.qknorm_forward(p, *a)
    angle = pos[0].double()
    for got, ref in ((out[0, :, :, 0], 2 * angle.cos()), (out[0, :, :, 1 if interleaved else 2], 2 * angle.sin())):
        assert ((got.double() - ref[:, None]).abs() <= 2.5 * 2.0 ** -23 * ref.abs()[:, None]).all()


def test_weight_gradients_are_rounded_once(dcn):  # noqa: F811
    """Heads of +-1 have a norm of 1, so that a weight's gradient is a sum of 888 given numbers.  With two heads a token
    that is a head for each of the backward's 1776 warps: no lane adds two of them, and the rest is 64 bits, so that
    the result is off by half a step of 2^-23 at most."""
    gen = torch.Generator().manual_seed(11)
    N, L, D = 3, 296, 256
    x = torch.randint(0, 2, (N, L, 1, D), generator=gen).float() * 2 - 1
    gq, gk = (torch.randn(x.shape, generator=gen, dtype=torch.float32) for _ in range(2))
    one = torch.ones(D, dtype=torch.float32).cuda()
    a = (x.cuda(), x.cuda(), one, one, None, None)
    p = dcn.qknorm_params_for(*a, eps=1e-30)
    got = dcn.qknorm_backward(p, *a, gq.cuda(), gk.cuda())[2:]
    for gw, g in zip(got, (gq, gk)):
        ref = (x.double() * g.double()).sum((0, 1, 2))
        assert ((gw.cpu().double() - ref).abs() <= 2.0 ** -24 * 1.0001 * ref.abs()).all()


def test_norm_of_zeros_with_a_tiny_eps(dcn):  # noqa: F811
    """1 / eps beyond the type's largest number: the gradient at zero is g w / sqrt(eps), a number."""
    x, g = (torch.full((1, 5, 2, 16), v, dtype=torch.float32).cuda() for v in (0.0, 1.0))
    p = dcn.qknorm_params_for(x, x, eps=1e-40)
    gx = dcn.qknorm_backward(p, x, x, None, None, None, None, g, g)[0]
    assert ((gx * 1e-20 - 1).abs() < 1e-4).all()  # eps is a subnormal: 1e-40 to 17 bits


@pytest.mark.parametrize("c", [case("f16", 1, 300, 300, 4, 2, 64, nb=8, M=16), case("f32", 1, 100, 100, 4, 2, 64, nb=8, M=16),
                               case("bf16", 1, 200, 200, 16, 1, 64, nb=8, M=128)], ids=str)
def test_a_frozen_bias_changes_nothing_else(dcn, c):  # noqa: F811
    t = make(c)
    cu = {k: None if v is None else v.cuda() for k, v in t.items()}
    a = (cu["q"], cu["k"], cu["v"])
    more = dict(bias=cu["bias"], buckets=cu["buckets"])
    p = dcn.band_params_for(*a, **more)
    out, lse = dcn.band_forward(p, *a, **more)
    full = dcn.band_backward(p, *a, out, lse, cu["g"], **more)
    part = dcn.band_backward(p, *a, out, lse, cu["g"], **more, want_bias=False)
    assert part[3] is None and full[3] is not None
    for x, y in zip(full[:3], part):
        assert torch.equal(x, y)
    q, k, v = (x.clone().requires_grad_(True) for x in a)
    grads = torch.autograd.grad(dcn.band_attention(q, k, v, **more), (q, k, v), cu["g"])
    for x, y in zip(full, grads):
        assert torch.equal(x, y)


def test_frozen_norm_weights_change_nothing_else(dcn):  # noqa: F811
    gen = torch.Generator().manual_seed(3)
    q, k, w = (torch.randn(*s, generator=gen).half().cuda() for s in ((2, 9, 4, 32), (2, 9, 2, 32), (32,)))
    p = dcn.qknorm_params_for(q, k, w, w)
    full = dcn.qknorm_backward(p, q, k, w, w, None, None, q, k)
    for wants in ((False, False), (True, False), (False, True)):
        part = dcn.qknorm_backward(p, q, k, w, w, None, None, q, k, *wants)
        for x, y, want in zip(full, part, (True, True) + wants):
            assert torch.equal(x, y) if want else y is None
    a, b = q.clone().requires_grad_(True), k.clone().requires_grad_(True)
    grads = torch.autograd.grad(dcn.qk_norm_rotate(a, b, w, w), (a, b), (q, k))
    assert torch.equal(grads[0], full[0]) and torch.equal(grads[1], full[1])


def test_gradients_from_outside_may_start_anywhere(dcn):  # noqa: F811
    """A contiguous upstream gradient that starts at an odd element, as a part of a longer buffer does."""
    gen = torch.Generator().manual_seed(5)
    q, k, v, w = (torch.randn(*s, generator=gen).half().cuda() for s in ((2, 9, 4, 32), (2, 9, 2, 32), (2, 9, 2, 32), (32,)))
    g = torch.randn(2, 9, 4, 32, generator=gen).half().cuda()
    odd = torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:].view(g.shape).copy_(g)
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v, w)]
    out = dcn.band_attention(*dcn.qk_norm_rotate(leaves[0], leaves[1], leaves[3], None), leaves[2])
    want = torch.autograd.grad(out, leaves, g, retain_graph=True)
    for x, y in zip(want, torch.autograd.grad(out, leaves, odd)):
        assert torch.equal(x, y)
    qn, _ = dcn.qk_norm_rotate(leaves[0], leaves[1], leaves[3], None)
    want = torch.autograd.grad(qn, leaves[0], g, retain_graph=True)
    assert torch.equal(want[0], torch.autograd.grad(qn, leaves[0], odd)[0])


MANY = [dict(dtype="bf16", N=3, L=1501, Hq=4, Hk=2, D=64, R=64, packed=True, far=3000),
        dict(dtype="f16", N=3, L=5003, Hq=2, Hk=1, D=32, R=16, axes=2),
        dict(dtype="f32", N=2, L=3001, Hq=5, Hk=1, D=80, R=40, interleaved=True, far=5000),
        dict(dtype="f16", N=3, L=2222, Hq=3, Hk=1, D=104, R=52, axes=2, packed=True),
        dict(dtype="bf16", N=7, L=700, Hq=3, Hk=0, D=128, R=0), dict(dtype="f32", N=2, L=4000, Hq=0, Hk=2, D=16, R=16),
        dict(dtype="f16", N=4999, L=3, Hq=1, Hk=1, D=8, R=8)]


@pytest.mark.parametrize("c", MANY, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_norms_of_several_tokens_a_warp(dcn, c):  # noqa: F811
    """Units of several tokens, warps with several units, units over the end of an image."""
    qknorm_case(dcn, c)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_far_rows_of_a_ragged_batch(dcn, dtype):  # noqa: F811
    """Rows of lowest biases with lengths, starts and sinks: each image's as its own call's on what it has.  (Both
    hold the same tiles; where fewer keys are split otherwise, sums of 32 bits differ by their order.)"""
    c = case(dtype, 3, 200, 330, 4, 2, 64, left=90, right=20, sinks=3, nb=4, M=100, q_start=[0, 130, 40], q_len=[200, 77, 130],
             k_len=[150, 330, 61], poison=True)
    t = make(c, 2)
    t["bias"][:3] = torch.finfo(DTYPES[dtype]).min
    t["buckets"] = torch.where(torch.arange(201) < 60, torch.full((201,), 3), torch.arange(201) % 3).int()
    got = run(dcn, c, t)
    gb = 0
    for n in range(3):
        a, b = c["q_len"][n], c["k_len"][n]
        one = case(dtype, 1, a, b, 4, 2, 64, left=90, right=20, sinks=3, nb=4, M=100)
        s = dict(t, q=t["q"][n:n + 1, :a].contiguous(), g=t["g"][n:n + 1, :a].contiguous(), k=t["k"][n:n + 1, :b].contiguous(),
                 v=t["v"][n:n + 1, :b].contiguous(), q_start=t["q_start"][n:n + 1], q_len=None, k_len=None)
        alone = run(dcn, one, s)
        for x, y, m in zip(got, alone, (a, a, a, b, b)):
            x = x[n, :, :m] if x.dim() == 3 else x[n, :m]
            assert torch.allclose(x.float(), y[0].float(), rtol=4 * torch.finfo(DTYPES[dtype]).eps, atol=2e-5 if dtype == "f32" else 2e-2)
            assert x.isfinite().all()
        gb = gb + alone[5].float()
    assert torch.allclose(got[5].float(), gb, rtol=8 * torch.finfo(DTYPES[dtype]).eps, atol=1e-3 if dtype == "f32" else 0.1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_captured_step_meets_far_rows_at_its_replay(dcn, dtype):  # noqa: F811
    c = case(dtype, 1, 150, 700, 4, 2, 64, nb=4, M=50)
    t = make(c, 4)
    cu = {k: None if v is None else v.cuda() for k, v in t.items()}
    low = torch.full_like(cu["bias"], torch.finfo(DTYPES[dtype]).min)

    def step(bias):
        leaves = [x.detach().requires_grad_(True) for x in (cu["q"], cu["k"], cu["v"], bias)]
        out = dcn.band_attention(*leaves[:3], bias=leaves[3], buckets=cu["buckets"])
        return (out.detach(),) + torch.autograd.grad(out, leaves, cu["g"])
    static = cu["bias"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step(static)
    for bias in (cu["bias"], low, cu["bias"]):
        static.copy_(bias)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(replayed, step(bias)):
            assert torch.equal(x, y) and x.isfinite().all()


@pytest.mark.parametrize("c", [case("bf16", 1, 100, 150, 2, 1, 64, scale=0.0, right=0), case("bf16", 1, 2, 150, 2, 1, 64, scale=0.0),
                               case("f32", 1, 30, 50, 2, 1, 64, scale=0.0, left=9)], ids=str)
def test_a_scale_of_zero_hides_large_products(dcn, c):  # noqa: F811
    """Products of 10^29 times 0 are 0: uniform rows."""
    t = make(c)
    t["q"], t["k"] = t["q"] * 1e14, t["k"] * 1e14
    compare(dcn, c, t)
