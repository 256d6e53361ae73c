"""Host side of the band attention and the query/key norm: struct mirrors, refusals, workspaces, the
bucket table (CPU only: nothing is launched)."""
import ctypes
import math
import re

import pytest

from test_abi_host import HEADER, dcn, run_without_gpu  # noqa: F401  (dcn is a fixture)

CTYPES = {"int": ctypes.c_int, "float": ctypes.c_float, "long long": ctypes.c_longlong}


@pytest.mark.parametrize("name", ["dcn4_band_params", "dcn4_qknorm_params"])
def test_struct_mirrors_match_the_header(dcn, name):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, text, flags=re.S).group(1)
    want = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        ctype, names = re.match(r"(long long|int|float)\s+(.*)", decl, flags=re.S).groups()
        want += [(n.strip(), CTYPES[ctype]) for n in names.split(",")]
    assert list(getattr(dcn, name)._fields_) == want


BAND = dict(N=2, Lq=40, Lk=50, Hq=4, Hk=2, D=32, left=5, right=5, sinks=1, nb=4, M=8, dtype="f16")


@pytest.mark.parametrize("field,value,status", [
    ("dtype", 7, -8), ("N", -1, -2), ("Lq", -1, -2), ("Lk", -3, -2), ("Hq", 0, -2), ("Hq", 3, -2), ("Hk", 0, -2),
    ("D", 0, -2), ("D", 4, -5), ("D", 136, -5), ("left", -2, -2), ("right", -2, -2), ("sinks", -1, -2),
    ("scale", math.nan, -2), ("scale", math.inf, -2), ("nb", -1, -2), ("M", 0, -2), ("nb", 1025, -5), ("M", 1025, -5),
    ("Hq", 512, -5), ("Lk", 1 << 28, -5), ("N", 1 << 24, -5), ("q_row", 64, -2), ("k_row", 68, -5), ("v_batch", -8, -2),
    ("k_batch", 1 << 39, -2), ("q_batch", 12, -5),
])
def test_band_refusals(dcn, field, value, status):
    p = dcn.make_band_params(**BAND)
    assert dcn.dcn4_band_check_params(p) == 0
    setattr(p, field, value)
    assert dcn.dcn4_band_check_params(p) == status
    assert dcn.dcn4_band_forward(p, *[None] * 10, None, 0) == status
    assert dcn.dcn4_band_backward(p, *[None] * 15, None, 0) == status
    assert dcn.dcn4_band_forward_workspace_size(p) == 0 and dcn.dcn4_band_backward_workspace_size(p) == 0


@pytest.mark.parametrize("field,value,status", [
    ("dtype", -1, -8), ("N", -1, -2), ("L", -1, -2), ("Hq", -1, -2), ("D", 0, -2), ("D", 20, -5), ("D", 264, -5),
    ("R", 34, -2), ("R", 3, -2), ("R", -2, -2), ("axes", 3, -2), ("axes", 0, -2), ("interleaved", 2, -2), ("eps", 0.0, -2),
    ("eps", math.nan, -2), ("Hq", 70000, -5), ("L", 1 << 30, -5), ("q_row", 32, -2), ("k_batch", 4, -5), ("q_batch", -8, -2),
])
def test_qknorm_refusals(dcn, field, value, status):
    p = dcn.make_qknorm_params(N=2, L=40, Hq=4, Hk=2, D=32, R=16)
    assert dcn.dcn4_qknorm_check_params(p) == 0
    setattr(p, field, value)
    assert dcn.dcn4_qknorm_check_params(p) == status
    assert dcn.dcn4_qknorm_forward(p, *[None] * 8) == status
    assert dcn.dcn4_qknorm_backward(p, *[None] * 13, 0) == status
    assert dcn.dcn4_qknorm_backward_workspace_size(p) == 0


def test_pointer_and_workspace_refusals():
    """NULL, misaligned and missing-workspace refusals (made-up addresses: checked in a child
    process that sees no GPU)."""
    run_without_gpu("""
p = dcn.make_band_params(N=2, Lq=40, Lk=50, Hq=4, Hk=2, D=32, nb=4, M=8, dtype="f16")
a = [16 * (i + 1) for i in range(16)]
f = lambda i=None, v=None, ws=4096, n=1 << 30: dcn.dcn4_band_forward(p, *[v if j == i else x for j, x in enumerate(a[:10])], ws, n)
b = lambda i=None, v=None, ws=4096, n=1 << 30: dcn.dcn4_band_backward(p, *[v if j == i else x for j, x in enumerate(a[:15])], ws, n)
for i in (0, 1, 2, 3, 4, 8, 9):
    assert f(i, None) == -1 and f(i, 24) == -4, i
for i in (5, 6, 7):
    assert f(i, 18) == -4, i
for i in (0, 1, 2, 3, 4, 8, 9, 10, 11, 12, 13):
    assert b(i, None) == -1 and b(i, 24) == -4, i
assert b(14, 24) == -4
assert b(ws=None) == -6 and b(n=16) == -6 and b(ws=4104) == -4
plain = dcn.make_band_params(N=2, Lq=40, Lk=50, Hq=4, Hk=2, D=32)
assert dcn.dcn4_band_forward(plain, *a[:10], None, 0) == -1            # a bias that nothing asked for
assert dcn.dcn4_band_backward(plain, *a[:3], None, None, *a[5:15], 4096, 1 << 30) == -1
long = dcn.make_band_params(N=1, Lq=1, Lk=100000, Hq=4, Hk=2, D=32)
assert dcn.dcn4_band_forward_workspace_size(long) > 0
assert dcn.dcn4_band_forward(long, *a[:3], None, None, *a[5:10], None, 0) == -6
none = dcn.make_band_params(N=0, Lq=40, Lk=50, Hq=4, Hk=2, D=32)
assert dcn.dcn4_band_forward(none, *[None] * 10, None, 0) == 0 and dcn.dcn4_band_backward(none, *[None] * 15, None, 0) == 0
q = dcn.make_qknorm_params(N=2, L=4, Hq=4, Hk=2, D=32, R=16)
g = lambda i=None, v=None: dcn.dcn4_qknorm_forward(q, *[v if j == i else x for j, x in enumerate(a[:8])])
for i in (0, 1, 4, 5, 6, 7):
    assert g(i, None) == -1 and g(i, 24) == -4, i
for i in (2, 3):
    assert g(i, 24) == -4, i
h = lambda i=None, v=None, ws=4096, n=1 << 30: dcn.dcn4_qknorm_backward(q, *[v if j == i else x for j, x in enumerate(a[:12])], ws, n)
for i in (0, 1, 4, 5, 6, 7, 8, 9):
    assert h(i, None) == -1 and h(i, 24) == -4, i
assert h(10, 24) == -4 and h(ws=None) == -6 and h(n=16) == -6
""")


def test_bucket_table(dcn):
    """Near distances one by one, then by their logarithm, the last bucket from M on; both sides apart."""
    t = (ctypes.c_int * 257)()
    assert dcn.dcn4_rel_buckets(32, 128, True, t) == 0
    v = list(t)
    assert v[128] == 0 and v[128 - 7] == 7 and v[128 + 7] == 16 + 7
    assert v[0] == 15 and v[256] == 31 and max(v) == 31
    assert v[:129] == sorted(v[:129], reverse=True) and v[129:] == sorted(v[129:])
    # distance 32 of exact 8, M 128: 8 + floor(8 log(4) / log(16)) = 12, on the border itself
    assert v[128 - 32] == 12 and v[128 - 31] == 11
    assert dcn.dcn4_rel_buckets(32, 128, False, t) == 0
    v = list(t)
    assert v[129:] == [0] * 128 and v[128 - 15] == 15 and v[0] == 31
    one = (ctypes.c_int * 3)()
    assert dcn.dcn4_rel_buckets(1, 1, False, one) == 0 and list(one) == [0, 0, 0]
    for nb, M, both in ((0, 8, 0), (4, 0, 0), (5, 8, 1), (2000, 8, 0), (4, 5000, 0)):
        assert dcn.dcn4_rel_buckets(nb, M, both, (ctypes.c_int * 10001)()) < 0
    assert dcn.dcn4_rel_buckets(4, 8, 1, None) == -1


def test_tensor_helpers_refuse_on_the_host(dcn):
    """The tensor helpers' own checks; CPU tensors are refused first."""
    import torch
    q = torch.zeros(2, 4, 2, 8).half()
    with pytest.raises(ValueError, match="CUDA"):
        dcn.band_attention(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.qk_norm_rotate(q, q)
    with pytest.raises(ValueError):
        dcn._heads_strides("q", q[0], q.dtype, q.device)
    p = dcn.make_band_params(N=2, Lq=4, Lk=4, Hq=2, D=8)
    for t in (q[:, :3], q.float(), torch.zeros(2, 4, 4, 8).half()):
        with pytest.raises(ValueError, match="not the tensor"):
            dcn.band_forward(p, t, q, q)
    b = dcn.make_band_params(N=2, Lq=4, Lk=4, Hq=2, D=8, nb=3, M=2)
    five = torch.zeros(5, dtype=torch.int32)
    for bias, buckets, vec in ((torch.zeros(4, 2).half(), five, None), (torch.zeros(3, 2).half(), five[:3].clone(), None),
                               (torch.zeros(3, 2).half(), five, five[:1].clone()), (torch.zeros(3, 2).half(), five, torch.zeros(2))):
        with pytest.raises(ValueError, match="must be a contiguous"):
            dcn.band_forward(b, q, q, q, bias, buckets, k_len=vec)
    r = dcn.make_qknorm_params(N=2, L=4, Hq=2, Hk=2, D=8, R=4)
    f32 = torch.float32
    ok = (torch.zeros(8).half(), None, torch.zeros(2, 4, dtype=f32), torch.zeros(2, dtype=f32))
    for i, t in ((0, torch.zeros(7).half()), (0, torch.zeros(8)), (2, torch.zeros(2, 3)), (3, torch.zeros(3)), (3, torch.zeros(2).double())):
        with pytest.raises(ValueError, match="made for"):
            dcn.qknorm_forward(r, q, q, *(t if j == i else x for j, x in enumerate(ok)))
    s = dcn.make_band_params(N=2, Lq=4, Lk=4, Hq=2, D=8, k_row=32, k_batch=128)
    with pytest.raises(ValueError, match="not the tensor"):
        dcn.band_forward(s, q, q, q)
