"""Host side of the band attention and the query/key norm, beyond tests/test_band_host.py: tensors that
parameters are not for, workspaces of calls that want less (CPU only: nothing is launched)."""
import pytest

from test_abi_host import dcn, run_without_gpu  # noqa: F401  (dcn is a fixture)


def _views(shape):
    """Tensors of `shape` that dense parameters are not for: expanded, with transposed heads, every second
    entry of longer rows, tokens of a longer row, on another device (as q: not on a GPU)."""
    import torch
    N, L, H, D = shape
    z = lambda *s: torch.zeros(*s).half()  # noqa: E731
    return {"expanded images": z(1, L, H, D).expand(shape), "expanded tokens": z(N, 1, H, D).expand(shape),
            "transposed heads": z(N, L, D, H).transpose(2, 3), "head by head": z(N, H, L, D).transpose(1, 2),
            "every second entry": z(N, L, H, 2 * D)[..., ::2], "longer rows": z(N, L, H + 1, D)[:, :, :H],
            "longer images": z(N, L + 1, H, D)[:, :L], "another device": torch.zeros(shape, dtype=torch.float16, device="meta")}


@pytest.mark.parametrize("name", list(_views((2, 4, 2, 8))))
@pytest.mark.parametrize("explicit", [False, True])
def test_tensors_that_the_parameters_are_not_for(dcn, name, explicit):
    """Shapes and types alone do not make a tensor the parameters' own (host checks: nothing is launched)."""
    import torch
    shape = (2, 4, 2, 8)
    dense, other = torch.zeros(shape).half(), _views(shape)[name]
    st = dict(q_batch=64, q_row=16, k_batch=64, k_row=16) if explicit else {}
    b = dcn.make_band_params(N=2, Lq=4, Lk=4, Hq=2, D=8, **st, **(dict(v_batch=64, v_row=16) if explicit else {}))
    r = dcn.make_qknorm_params(N=2, L=4, Hq=2, Hk=2, D=8, **st)
    for i in range(3):
        args = [other if i == j else dense for j in range(3)]
        with pytest.raises(ValueError, match="not the tensor"):
            dcn.band_forward(b, *args)
        with pytest.raises(ValueError, match="not the tensor"):
            dcn.band_backward(b, *args, dense, torch.zeros(2, 2, 4), dense)
    for args in ((other, dense), (dense, other)):
        with pytest.raises(ValueError, match="not the tensor"):
            dcn.qknorm_forward(r, *args)
        with pytest.raises(ValueError, match="not the tensor"):
            dcn.qknorm_backward(r, *args, None, None, None, None, dense, dense)


def test_parameters_of_dense_tensors_take_no_cpu_tensors(dcn):
    import torch
    t = torch.zeros(2, 4, 2, 8).half()
    with pytest.raises(ValueError, match="CUDA"):
        dcn.band_forward(dcn.make_band_params(N=2, Lq=4, Lk=4, Hq=2, D=8), t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        dcn.qknorm_forward(dcn.make_qknorm_params(N=2, L=4, Hq=2, Hk=2, D=8), t, t)


def test_workspaces_hold_what_is_used(dcn):  # noqa: F811
    """A long window with sinks: only the sinks' tile of keys is split, and only its parts are held."""
    p = dcn.make_band_params(N=1, Lq=131072, Lk=131072, Hq=8, D=128, left=4095, right=0, sinks=4, dtype="bf16")
    rows = 8 * 131072
    parts = 2 * 128 * 128 * 4 * (4 * 148)  # fp32 gradients of 128 keys, of four items an SM at most
    assert dcn.dcn4_band_backward_workspace_size(p) < rows * 16 + parts


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_a_frozen_bias_needs_no_memory_for_its_gradient(dcn, dtype):  # noqa: F811
    """The size that the call itself asks for (made-up addresses, no GPU in sight)."""
    p = dcn.make_band_params(N=4, Lq=1024, Lk=1024, Hq=16, D=64, nb=32, M=512, dtype=dtype)
    rows = 4 * 16 * 1024
    whole, frozen = dcn.dcn4_band_backward_workspace_size(p), dcn.dcn4_band_backward_frozen_workspace_size(p)
    assert frozen <= rows * 16 + 4096 and whole > 5 * frozen
    plain = dcn.make_band_params(N=4, Lq=1024, Lk=1024, Hq=16, D=64, dtype=dtype)
    assert dcn.dcn4_band_backward_workspace_size(plain) == dcn.dcn4_band_backward_frozen_workspace_size(plain) == frozen
    p.D = 3
    assert dcn.dcn4_band_backward_frozen_workspace_size(p) == 0
    run_without_gpu(f"""
p = dcn.make_band_params(N=4, Lq=1024, Lk=1024, Hq=16, D=64, nb=32, M=512, dtype="{dtype}")
a = [16 * (i + 1) for i in range(14)]
frozen = dcn.dcn4_band_backward_frozen_workspace_size(p)
assert dcn.dcn4_band_backward(p, *a, 4096, 4096, frozen) == -6           # a gradient wanted
assert dcn.dcn4_band_backward(p, *a, None, 4096, frozen - 1) == -6
assert dcn.dcn4_band_backward(p, *a, None, 4096, frozen) not in (0, -6)  # as far as the launch, which has no GPU
""")
