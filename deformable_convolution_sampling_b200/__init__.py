"""Python binding of libdcn4, the sm_100a DCNv4 core spatial aggregation.

The C ABI (include/dcn4.h) is exposed under the same names -- ``dcn4_forward``,
``dcn4_backward``, ``dcn4_output_dims`` ... -- taking a :class:`dcn4_params`
and raw device pointers.  They only marshal arguments: every step of the
operator runs in the library's CUDA kernels.  There is no CPU fallback; if the
library is not built, importing this package fails.

``forward`` / ``backward`` are conveniences over the same calls for torch
tensors (torch provides device memory and streams only).
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdcn4.so")

DCN4_F32, DCN4_F16, DCN4_BF16 = 0, 1, 2
STATUS = {
    0: "DCN4_OK", -1: "DCN4_ERR_NULL", -2: "DCN4_ERR_BAD_SHAPE", -3: "DCN4_ERR_BAD_P",
    -4: "DCN4_ERR_MISALIGNED", -5: "DCN4_ERR_UNSUPPORTED", -6: "DCN4_ERR_WORKSPACE",
    -7: "DCN4_ERR_LAUNCH", -8: "DCN4_ERR_DTYPE",
}
DTYPE_NAMES = {"f32": DCN4_F32, "f16": DCN4_F16, "bf16": DCN4_BF16}


class Dcn4Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status


class dcn4_params(ctypes.Structure):
    """Mirror of the C struct dcn4_params."""

    _fields_ = [
        ("N", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
        ("G", ctypes.c_int), ("Cg", ctypes.c_int),
        ("kh", ctypes.c_int), ("kw", ctypes.c_int),
        ("sh", ctypes.c_int), ("sw", ctypes.c_int),
        ("ph", ctypes.c_int), ("pw", ctypes.c_int),
        ("dh", ctypes.c_int), ("dw", ctypes.c_int),
        ("offset_scale", ctypes.c_float),
        ("remove_center", ctypes.c_int),
        ("P", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("softmax", ctypes.c_int),
    ]


class dcn4_attn_params(ctypes.Structure):
    """Mirror of dcn4_attn_params in include/dcn4.h (field order matters)."""

    _fields_ = [
        ("N", ctypes.c_int), ("H", ctypes.c_int), ("W", ctypes.c_int),
        ("G", ctypes.c_int), ("Cg", ctypes.c_int),
        ("Nq", ctypes.c_int), ("K", ctypes.c_int),
        ("offset_scale", ctypes.c_float),
        ("P", ctypes.c_int),
        ("dtype", ctypes.c_int),
    ]


class dcn4_band_params(ctypes.Structure):
    """Mirror of dcn4_band_params in include/dcn4.h (field order matters)."""

    _fields_ = [
        ("N", ctypes.c_int), ("Lq", ctypes.c_int), ("Lk", ctypes.c_int),
        ("Hq", ctypes.c_int), ("Hk", ctypes.c_int), ("D", ctypes.c_int),
        ("left", ctypes.c_int), ("right", ctypes.c_int), ("sinks", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("nb", ctypes.c_int), ("M", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("q_batch", ctypes.c_longlong), ("q_row", ctypes.c_longlong),
        ("k_batch", ctypes.c_longlong), ("k_row", ctypes.c_longlong),
        ("v_batch", ctypes.c_longlong), ("v_row", ctypes.c_longlong),
    ]


class dcn4_qknorm_params(ctypes.Structure):
    """Mirror of dcn4_qknorm_params in include/dcn4.h (field order matters)."""

    _fields_ = [
        ("N", ctypes.c_int), ("L", ctypes.c_int),
        ("Hq", ctypes.c_int), ("Hk", ctypes.c_int), ("D", ctypes.c_int),
        ("R", ctypes.c_int), ("axes", ctypes.c_int), ("interleaved", ctypes.c_int),
        ("eps", ctypes.c_float),
        ("dtype", ctypes.c_int),
        ("q_batch", ctypes.c_longlong), ("q_row", ctypes.c_longlong),
        ("k_batch", ctypes.c_longlong), ("k_row", ctypes.c_longlong),
    ]


def make_band_params(*, N, Lq, Lk, Hq, D, Hk=None, left=-1, right=-1, sinks=0, scale=None, nb=0, M=0, dtype="f16",
                     q_batch=0, q_row=0, k_batch=0, k_row=0, v_batch=0, v_row=0) -> dcn4_band_params:
    """dcn4_band_params of a dense attention over a band of keys; Hk defaults to Hq, scale
    to 1/sqrt(D), and strides of 0 mean dense tensors."""
    if isinstance(dtype, str):
        dtype = DTYPE_NAMES[dtype]
    return dcn4_band_params(N, Lq, Lk, Hq, Hq if Hk is None else Hk, D, left, right, sinks,
                            D ** -0.5 if scale is None else float(scale), nb, M, dtype,
                            q_batch, q_row, k_batch, k_row, v_batch, v_row)


def make_qknorm_params(*, N, L, Hq, Hk, D, R=0, axes=1, interleaved=0, eps=1e-6, dtype="f16",
                       q_batch=0, q_row=0, k_batch=0, k_row=0) -> dcn4_qknorm_params:
    """dcn4_qknorm_params of a query/key norm with rotation; strides of 0 mean dense tensors."""
    if isinstance(dtype, str):
        dtype = DTYPE_NAMES[dtype]
    return dcn4_qknorm_params(N, L, Hq, Hk, D, R, axes, 1 if interleaved else 0, float(eps), dtype,
                              q_batch, q_row, k_batch, k_row)


def make_attn_params(*, N, H, W, G, Cg, Nq, K, offset_scale=1.0, P=None, dtype="f16") -> dcn4_attn_params:
    """dcn4_attn_params for a single-scale deformable attention call; P defaults to G*3K rounded up to 8."""
    if isinstance(dtype, str):
        dtype = DTYPE_NAMES[dtype]
    if P is None:
        P = -(-G * 3 * K // 8) * 8
    return dcn4_attn_params(N, H, W, G, Cg, Nq, K, float(offset_scale), P, dtype)


def make_params(*, N, H, W, G, Cg, kh=3, kw=3, sh=1, sw=1, ph=1, pw=1, dh=1, dw=1,
                offset_scale=1.0, remove_center=0, P=None, dtype="f32", softmax=0) -> dcn4_params:
    """Build a dcn4_params; P defaults to the smallest valid padded row.  softmax=1
    normalises the K masks of each (pixel, group) with a softmax (the DCNv3 form)."""
    if isinstance(dtype, str):
        dtype = DTYPE_NAMES[dtype]
    if P is None:
        P = dcn4_padded_offset_dim(G, kh * kw - (1 if remove_center else 0))
    return dcn4_params(N, H, W, G, Cg, kh, kw, sh, sw, ph, pw, dh, dw, float(offset_scale),
                       1 if remove_center else 0, P, dtype, 1 if softmax else 0)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built; run `python deformable_convolution_sampling_b200/build.py` "
            "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(dcn4_params)
    AP = ctypes.POINTER(dcn4_attn_params)
    BP = ctypes.POINTER(dcn4_band_params)
    QP = ctypes.POINTER(dcn4_qknorm_params)
    vp, ip = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)
    sig = {
        "dcn4_version": ([], ctypes.c_int),
        "dcn4_num_points": ([P], ctypes.c_int),
        "dcn4_padded_offset_dim": ([ctypes.c_int, ctypes.c_int], ctypes.c_int),
        "dcn4_output_dims": ([P, ip, ip], ctypes.c_int),
        "dcn4_check_params": ([P], ctypes.c_int),
        "dcn4_forward": ([P, vp, vp, vp, vp], ctypes.c_int),
        "dcn4_forward_linear": ([P, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "dcn4_backward_workspace_size": ([P], ctypes.c_size_t),
        "dcn4_backward": ([P, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "dcn4_last_error": ([], ctypes.c_char_p),
        "dcn4_backward_offset_mask": ([P, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_backward_value": ([P, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_backward_noalloc": ([P, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "dcn4_backward_noalloc_capacity": ([], ctypes.c_size_t),
        "dcn4_noalloc_last_error": ([], ctypes.c_char_p),
        "dcn4_backward_diagnostics": ([P, vp, ctypes.c_size_t, ip, vp], ctypes.c_int),
        "dcn4_backward_linear_workspace_size": ([P, ctypes.c_int], ctypes.c_size_t),
        "dcn4_backward_linear": ([P, ctypes.c_int] + [vp] * 11 + [ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_forward_proj": ([P, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "dcn4_forward_tc_status": ([ctypes.c_int], ctypes.c_int),
        "dcn4_backward_proj_workspace_size": ([P, ctypes.c_int], ctypes.c_size_t),
        "dcn4_backward_proj": ([P, ctypes.c_int] + [vp] * 10 + [ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_attn_check_params": ([AP], ctypes.c_int),
        "dcn4_attn_forward": ([AP, vp, vp, vp, vp, vp], ctypes.c_int),
        "dcn4_attn_backward_workspace_size": ([AP], ctypes.c_size_t),
        "dcn4_attn_backward": ([AP, vp, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_band_check_params": ([BP], ctypes.c_int),
        "dcn4_rel_buckets": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, ip], ctypes.c_int),
        "dcn4_band_forward_workspace_size": ([BP], ctypes.c_size_t),
        "dcn4_band_forward": ([BP] + [vp] * 11 + [ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_band_backward_workspace_size": ([BP], ctypes.c_size_t),
        "dcn4_band_backward_frozen_workspace_size": ([BP], ctypes.c_size_t),
        "dcn4_band_backward": ([BP] + [vp] * 16 + [ctypes.c_size_t, vp], ctypes.c_int),
        "dcn4_band_status": ([ctypes.c_int], ctypes.c_int),
        "dcn4_qknorm_check_params": ([QP], ctypes.c_int),
        "dcn4_qknorm_forward": ([QP] + [vp] * 9, ctypes.c_int),
        "dcn4_qknorm_backward_workspace_size": ([QP], ctypes.c_size_t),
        "dcn4_qknorm_backward": ([QP] + [vp] * 13 + [ctypes.c_size_t, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()


# ---------------------------------------------------------------------------
# Same-name wrappers of the C ABI (pointers are ints or None; stream is a
# cudaStream_t handle as an int, 0 / None for the legacy default stream).
# ---------------------------------------------------------------------------

def dcn4_version() -> int:
    return lib.dcn4_version()


def dcn4_num_points(p: dcn4_params) -> int:
    return lib.dcn4_num_points(ctypes.byref(p))


def dcn4_padded_offset_dim(G: int, K: int) -> int:
    return lib.dcn4_padded_offset_dim(G, K)


def dcn4_output_dims(p: dcn4_params) -> tuple[int, int, int]:
    ho, wo = ctypes.c_int(), ctypes.c_int()
    st = lib.dcn4_output_dims(ctypes.byref(p), ctypes.byref(ho), ctypes.byref(wo))
    return st, ho.value, wo.value


def dcn4_check_params(p: dcn4_params) -> int:
    return lib.dcn4_check_params(ctypes.byref(p))


def dcn4_forward(p: dcn4_params, value, offset_mask, out, stream=None) -> int:
    return lib.dcn4_forward(ctypes.byref(p), value, offset_mask, out, stream)


def dcn4_forward_linear(p: dcn4_params, Cx: int, value, x, weight, bias, out, offset_mask_out=None,
                        stream=None) -> int:
    return lib.dcn4_forward_linear(ctypes.byref(p), int(Cx), value, x, weight, bias, out, offset_mask_out, stream)


def dcn4_forward_proj(p: dcn4_params, Cout: int, value, offset_mask, weight, bias, out, core_out=None,
                      stream=None) -> int:
    return lib.dcn4_forward_proj(ctypes.byref(p), int(Cout), value, offset_mask, weight, bias, out, core_out, stream)


def dcn4_forward_tc_status(reset: bool = False) -> int:
    return lib.dcn4_forward_tc_status(1 if reset else 0)


def dcn4_backward_proj_workspace_size(p: dcn4_params, Cout: int) -> int:
    return lib.dcn4_backward_proj_workspace_size(ctypes.byref(p), int(Cout))


def dcn4_backward_proj(p: dcn4_params, Cout: int, value, offset_mask, core_out, weight, grad_out, grad_value,
                       grad_offset_mask, grad_weight, grad_bias, workspace, workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_backward_proj(ctypes.byref(p), int(Cout), value, offset_mask, core_out, weight, grad_out,
                                  grad_value, grad_offset_mask, grad_weight, grad_bias, workspace, workspace_bytes,
                                  stream)


def dcn4_backward_workspace_size(p: dcn4_params) -> int:
    return lib.dcn4_backward_workspace_size(ctypes.byref(p))


def dcn4_backward(p: dcn4_params, value, offset_mask, grad_out, grad_value, grad_offset_mask,
                  workspace, workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_backward(ctypes.byref(p), value, offset_mask, grad_out, grad_value,
                             grad_offset_mask, workspace, workspace_bytes, stream)


def dcn4_backward_offset_mask(p: dcn4_params, value, offset_mask, grad_out, grad_offset_mask, workspace,
                              workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_backward_offset_mask(ctypes.byref(p), value, offset_mask, grad_out, grad_offset_mask,
                                         workspace, workspace_bytes, stream)


def dcn4_backward_value(p: dcn4_params, offset_mask, grad_out, grad_value, workspace, workspace_bytes: int,
                        stream=None) -> int:
    return lib.dcn4_backward_value(ctypes.byref(p), offset_mask, grad_out, grad_value, workspace,
                                   workspace_bytes, stream)


def dcn4_backward_diagnostics(p: dcn4_params, workspace, workspace_bytes: int, stream=None):
    """(status, [corrupt bucket tiles, rescanned tiles, direct-path tiles]) of the last
    backward run on `workspace`; waits for `stream`."""
    counts = (ctypes.c_int * 3)()
    st = lib.dcn4_backward_diagnostics(ctypes.byref(p), workspace, workspace_bytes, counts, stream)
    return st, list(counts)


def dcn4_backward_linear_workspace_size(p: dcn4_params, Cx: int) -> int:
    return lib.dcn4_backward_linear_workspace_size(ctypes.byref(p), int(Cx))


def dcn4_backward_linear(p: dcn4_params, Cx: int, value, offset_mask, x, weight, grad_out, grad_value,
                         grad_offset_mask, grad_x, grad_weight, grad_bias, workspace, workspace_bytes: int,
                         stream=None) -> int:
    return lib.dcn4_backward_linear(ctypes.byref(p), int(Cx), value, offset_mask, x, weight, grad_out, grad_value,
                                    grad_offset_mask, grad_x, grad_weight, grad_bias, workspace, workspace_bytes,
                                    stream)


def dcn4_attn_check_params(p: dcn4_attn_params) -> int:
    return lib.dcn4_attn_check_params(ctypes.byref(p))


def dcn4_attn_forward(p: dcn4_attn_params, value, ref_points, offset_logits, out, stream=None) -> int:
    return lib.dcn4_attn_forward(ctypes.byref(p), value, ref_points, offset_logits, out, stream)


def dcn4_attn_backward_workspace_size(p: dcn4_attn_params) -> int:
    return lib.dcn4_attn_backward_workspace_size(ctypes.byref(p))


def dcn4_attn_backward(p: dcn4_attn_params, value, ref_points, offset_logits, grad_out, grad_value,
                       grad_offset_logits, workspace, workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_attn_backward(ctypes.byref(p), value, ref_points, offset_logits, grad_out, grad_value,
                                  grad_offset_logits, workspace, workspace_bytes, stream)


def dcn4_band_check_params(p: dcn4_band_params) -> int:
    return lib.dcn4_band_check_params(ctypes.byref(p))


def dcn4_rel_buckets(nb: int, M: int, both: bool, table) -> int:
    """`table`: a ctypes array of 2 * M + 1 ints."""
    return lib.dcn4_rel_buckets(int(nb), int(M), 1 if both else 0, table)


def dcn4_band_forward_workspace_size(p: dcn4_band_params) -> int:
    return lib.dcn4_band_forward_workspace_size(ctypes.byref(p))


def dcn4_band_forward(p: dcn4_band_params, q, k, v, bias, buckets, q_start, q_len, k_len, out, lse, workspace,
                      workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_band_forward(ctypes.byref(p), q, k, v, bias, buckets, q_start, q_len, k_len, out, lse, workspace,
                                 workspace_bytes, stream)


def dcn4_band_backward_workspace_size(p: dcn4_band_params) -> int:
    return lib.dcn4_band_backward_workspace_size(ctypes.byref(p))


def dcn4_band_backward_frozen_workspace_size(p: dcn4_band_params) -> int:
    return lib.dcn4_band_backward_frozen_workspace_size(ctypes.byref(p))


def dcn4_band_backward(p: dcn4_band_params, q, k, v, bias, buckets, q_start, q_len, k_len, out, lse, grad_out, grad_q,
                       grad_k, grad_v, grad_bias, workspace, workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_band_backward(ctypes.byref(p), q, k, v, bias, buckets, q_start, q_len, k_len, out, lse, grad_out,
                                  grad_q, grad_k, grad_v, grad_bias, workspace, workspace_bytes, stream)


def dcn4_band_status(reset: bool = False) -> int:
    return lib.dcn4_band_status(1 if reset else 0)


def dcn4_qknorm_check_params(p: dcn4_qknorm_params) -> int:
    return lib.dcn4_qknorm_check_params(ctypes.byref(p))


def dcn4_qknorm_forward(p: dcn4_qknorm_params, q, k, wq, wk, pos, inv_freq, q_out, k_out, stream=None) -> int:
    return lib.dcn4_qknorm_forward(ctypes.byref(p), q, k, wq, wk, pos, inv_freq, q_out, k_out, stream)


def dcn4_qknorm_backward_workspace_size(p: dcn4_qknorm_params) -> int:
    return lib.dcn4_qknorm_backward_workspace_size(ctypes.byref(p))


def dcn4_qknorm_backward(p: dcn4_qknorm_params, q, k, wq, wk, pos, inv_freq, grad_q_out, grad_k_out, grad_q, grad_k,
                         grad_wq, grad_wk, workspace, workspace_bytes: int, stream=None) -> int:
    return lib.dcn4_qknorm_backward(ctypes.byref(p), q, k, wq, wk, pos, inv_freq, grad_q_out, grad_k_out, grad_q,
                                    grad_k, grad_wq, grad_wk, workspace, workspace_bytes, stream)


def dcn4_backward_noalloc(p: dcn4_params, value, offset_mask, grad_out, grad_value, grad_offset_mask,
                          stream=None) -> int:
    """dcn4_backward with the library's built-in scratch area instead of a workspace
    (for callers that cannot provide device memory when they call)."""
    return lib.dcn4_backward_noalloc(ctypes.byref(p), value, offset_mask, grad_out, grad_value,
                                     grad_offset_mask, stream)


def dcn4_backward_noalloc_capacity() -> int:
    return lib.dcn4_backward_noalloc_capacity()


def dcn4_noalloc_last_error() -> str:
    return lib.dcn4_noalloc_last_error().decode()


def dcn4_status_string(status: int) -> str:
    return lib.dcn4_status_string(status).decode()


def dcn4_last_error() -> str:
    return lib.dcn4_last_error().decode()


def check(status: int) -> None:
    """Raise Dcn4Error for a negative status."""
    if status != 0:
        raise Dcn4Error(status, dcn4_last_error())


# ---------------------------------------------------------------------------
# torch conveniences (device memory and the current stream come from torch)
# ---------------------------------------------------------------------------

_TORCH_DTYPES = None


def _torch_dtype(code: int):
    global _TORCH_DTYPES
    if _TORCH_DTYPES is None:
        import torch
        _TORCH_DTYPES = {DCN4_F32: torch.float32, DCN4_F16: torch.float16, DCN4_BF16: torch.bfloat16}
    return _TORCH_DTYPES[code]


def _stream_handle(device):
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a Stream object: 2 us less a call
    if raw is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return raw(device.index)


def forward(p: dcn4_params, value, offset_mask, out=None):
    """y[N,Ho,Wo,C] for CUDA tensors value[N,H,W,C] and offset_mask[N,Ho,Wo,P]."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    if out is None:
        out = torch.empty((p.N, Ho, Wo, p.G * p.Cg), dtype=_torch_dtype(p.dtype), device=value.device)
    check(dcn4_forward(p, value.data_ptr(), offset_mask.data_ptr(), out.data_ptr(),
                       _stream_handle(value.device)))
    return out


def forward_linear(p: dcn4_params, value, x, weight, bias=None, out=None, offset_mask_out=None):
    """y[N,Ho,Wo,C] with the offset_mask formed in the kernel as x @ weight.T + bias
    (x [N,Ho,Wo,Cx], weight [P,Cx], bias [P] or None); offset_mask_out, when given
    ([N,Ho,Wo,P]), receives that offset_mask.  CUDA tensors, fp16 or bf16."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    if out is None:
        out = torch.empty((p.N, Ho, Wo, p.G * p.Cg), dtype=_torch_dtype(p.dtype), device=value.device)
    check(dcn4_forward_linear(p, x.shape[-1], value.data_ptr(), x.data_ptr(), weight.data_ptr(),
                              bias.data_ptr() if bias is not None else None, out.data_ptr(),
                              offset_mask_out.data_ptr() if offset_mask_out is not None else None,
                              _stream_handle(value.device)))
    return out


def backward(p: dcn4_params, value, offset_mask, grad_out, grad_value=None, grad_offset_mask=None,
             workspace=None):
    """(grad_value[N,H,W,C], grad_offset_mask[N,Ho,Wo,P]) for CUDA tensors.  `workspace`
    (a uint8 CUDA tensor of dcn4_backward_workspace_size bytes) is allocated when not
    given; pass one to read the call's fallback counters with backward_diagnostics."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    dt = _torch_dtype(p.dtype)
    if grad_value is None:
        grad_value = torch.empty_like(value, dtype=dt)
    if grad_offset_mask is None:
        grad_offset_mask = torch.empty((p.N, Ho, Wo, p.P), dtype=dt, device=value.device)
    need = dcn4_backward_workspace_size(p)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=value.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    check(dcn4_backward(p, value.data_ptr(), offset_mask.data_ptr(), grad_out.data_ptr(),
                        grad_value.data_ptr(), grad_offset_mask.data_ptr(), ws_ptr, ws_bytes,
                        _stream_handle(value.device)))
    return grad_value, grad_offset_mask


def backward_linear(p: dcn4_params, value, offset_mask, x, weight, grad_out, with_bias: bool = True,
                    want_x: bool = True, want_weight: bool = True, workspace=None):
    """Backward of forward_linear for CUDA tensors (offset_mask: the one the forward
    formed): (grad_value, grad_offset_mask, grad_x or None, grad_weight or None,
    grad_bias or None), all computed in libdcn4."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    dt = _torch_dtype(p.dtype)
    dev = value.device
    Cx = x.shape[-1]
    gv = torch.empty_like(value, dtype=dt)
    gom = torch.empty((p.N, Ho, Wo, p.P), dtype=dt, device=dev)
    gx = torch.empty_like(x) if want_x else None
    gw = torch.empty_like(weight) if want_weight else None
    gb = torch.empty((p.P,), dtype=dt, device=dev) if with_bias else None
    need = dcn4_backward_linear_workspace_size(p, Cx)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def ptr(t):
        return t.data_ptr() if t is not None else None

    check(dcn4_backward_linear(p, Cx, value.data_ptr(), offset_mask.data_ptr(), x.data_ptr(), weight.data_ptr(),
                               grad_out.data_ptr(), gv.data_ptr(), gom.data_ptr(), ptr(gx), ptr(gw), ptr(gb),
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _stream_handle(dev)))
    return gv, gom, gx, gw, gb


def forward_proj(p: dcn4_params, value, offset_mask, weight, bias=None, out=None, core_out=None):
    """y[N,Ho,Wo,Cout] = (aggregation of value at offset_mask) @ weight.T + bias, the
    projection formed inside the forward kernel (weight [Cout,C], bias [Cout] or None);
    core_out, when given ([N,Ho,Wo,C]), receives the aggregation's own output.  CUDA
    tensors, fp16 or bf16."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    Cout = weight.shape[0]
    if out is None:
        out = torch.empty((p.N, Ho, Wo, Cout), dtype=_torch_dtype(p.dtype), device=value.device)
    check(dcn4_forward_proj(p, Cout, value.data_ptr(), offset_mask.data_ptr(), weight.data_ptr(),
                            bias.data_ptr() if bias is not None else None, out.data_ptr(),
                            core_out.data_ptr() if core_out is not None else None, _stream_handle(value.device)))
    return out


def backward_proj(p: dcn4_params, value, offset_mask, core_out, weight, grad_out, with_bias: bool = True,
                  want_weight: bool = True, workspace=None):
    """Backward of forward_proj for CUDA tensors (core_out: the aggregation output the
    forward saved): (grad_value, grad_offset_mask, grad_weight or None, grad_bias or
    None), all computed in libdcn4."""
    import torch
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    dt = _torch_dtype(p.dtype)
    dev = value.device
    Cout = weight.shape[0]
    gv = torch.empty_like(value, dtype=dt)
    gom = torch.empty((p.N, Ho, Wo, p.P), dtype=dt, device=dev)
    gw = torch.empty_like(weight) if want_weight else None
    gb = torch.empty((Cout,), dtype=dt, device=dev) if with_bias else None
    need = dcn4_backward_proj_workspace_size(p, Cout)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)

    def ptr(t):
        return t.data_ptr() if t is not None else None

    check(dcn4_backward_proj(p, Cout, value.data_ptr(), offset_mask.data_ptr(), ptr(core_out), weight.data_ptr(),
                             grad_out.data_ptr(), gv.data_ptr(), gom.data_ptr(), ptr(gw), ptr(gb),
                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                             _stream_handle(dev)))
    return gv, gom, gw, gb


def attn_forward(p: dcn4_attn_params, value, ref_points, offset_logits, out=None):
    """y[N,Nq,C] of single-scale deformable attention for CUDA tensors value [N,H,W,C],
    ref_points [N,Nq,2] (float32) and offset_logits [N,Nq,P]."""
    import torch
    if out is None:
        out = torch.empty((p.N, p.Nq, p.G * p.Cg), dtype=_torch_dtype(p.dtype), device=value.device)
    check(dcn4_attn_forward(p, value.data_ptr(), ref_points.data_ptr(), offset_logits.data_ptr(), out.data_ptr(),
                            _stream_handle(value.device)))
    return out


def attn_backward(p: dcn4_attn_params, value, ref_points, offset_logits, grad_out):
    """(grad_value[N,H,W,C], grad_offset_logits[N,Nq,P]) for CUDA tensors."""
    import torch
    dt = _torch_dtype(p.dtype)
    gv = torch.empty((p.N, p.H, p.W, p.G * p.Cg), dtype=dt, device=value.device)
    gol = torch.empty((p.N, p.Nq, p.P), dtype=dt, device=value.device)
    need = dcn4_attn_backward_workspace_size(p)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=value.device)
    check(dcn4_attn_backward(p, value.data_ptr(), ref_points.data_ptr(), offset_logits.data_ptr(),
                             grad_out.data_ptr(), gv.data_ptr(), gol.data_ptr(), ws.data_ptr(), need,
                             _stream_handle(value.device)))
    return gv, gol


def rel_buckets(nb: int, M: int, both: bool = True, device="cuda"):
    """int32 tensor [2M + 1] of the buckets of relative positions -M..M (dcn4_rel_buckets)."""
    import torch
    table = (ctypes.c_int * (2 * max(M, 0) + 1))()
    check(dcn4_rel_buckets(nb, M, both, table))
    return torch.tensor(list(table), dtype=torch.int32, device=device)


def _launch(device, call, *args):
    """check(call(*args, stream)) with `device` the current one and its current stream."""
    import torch
    here = torch.cuda.current_device()
    if device.index == here:
        check(call(*args, _stream_handle(device)))
        return
    with torch.cuda.device(device):
        check(call(*args, _stream_handle(device)))


def _dense_like(t, shape):
    """An uninitialised contiguous tensor of `shape`, of t's type and device."""
    import torch
    return torch.empty_like(t) if t.shape == shape and t.is_contiguous() else t.new_empty(shape)


def _upstream(t):
    """An upstream gradient as the kernels take it: contiguous and from a 16-byte boundary on."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _workspace(need: int, like):
    import torch
    return torch.empty(need, dtype=torch.uint8, device=like.device) if need else None


def _heads_strides(name, t, dtype, device):
    """(batch, row) element strides of t [N, L, H, D] whose heads are contiguous; ValueError otherwise.
    A dimension of length 1 has no stride that matters."""
    if t.dim() != 4:
        raise ValueError(f"{name} must be [N, L, H, D]")
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on the same CUDA device as the others")
    if t.dtype != dtype:
        raise ValueError(f"{name} must have the same dtype as the others")
    N, L, H, D = t.shape
    sb, sl, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    row = sl if L > 1 else H * D
    batch = sb if N > 1 else row * L
    if t.numel() and ((L > 1 and row < H * D) or (N > 1 and batch < H * D)):
        raise ValueError(f"{name}: tokens must not overlap (expand()ed tensors need .contiguous())")
    return batch, row


def _int_vector(name, t, N, device):
    import torch
    if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (N,) or not t.is_contiguous() or t.device != device):
        raise ValueError(f"{name} must be a contiguous int32 tensor [{N}] on q's device")


def _dense(name, t, shape, dtype, device):
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on q's device")


def band_params_for(q, k, v, *, left=-1, right=-1, sinks=0, scale=None, bias=None, buckets=None, q_start=None,
                    q_len=None, k_len=None) -> dcn4_band_params:
    """dcn4_band_params for CUDA tensors q [N, Lq, Hq, D], k and v [N, Lk, Hk, D] (views whose heads are
    contiguous, such as parts of one packed projection or of a cache), bias [nb, Hq], buckets [2M + 1]
    (int32) and q_start, q_len, k_len [N] (int32); checks them on the host (ValueError, Dcn4Error)."""
    import torch
    qb, qr = _heads_strides("q", q, q.dtype, q.device)
    kb, kr = _heads_strides("k", k, q.dtype, q.device)
    vb, vr = _heads_strides("v", v, q.dtype, q.device)
    N, Lq, Hq, D = q.shape
    if k.shape != v.shape or k.shape[0] != N or k.shape[3] != D:
        raise ValueError("k and v must be [N, Lk, Hk, D] with q's N and D")
    nb = M = 0
    if (bias is None) != (buckets is None):
        raise ValueError("bias and buckets come together")
    if bias is not None:
        if bias.dim() != 2 or bias.shape[0] < 1 or buckets.dim() != 1 or buckets.shape[0] < 3 or buckets.shape[0] % 2 == 0:
            raise ValueError("bias must be [nb, Hq] and buckets [2M + 1]")
        nb, M = bias.shape[0], buckets.shape[0] // 2
        _dense("bias", bias, (nb, Hq), q.dtype, q.device)
        _dense("buckets", buckets, (2 * M + 1,), torch.int32, q.device)
    for name, t in (("q_start", q_start), ("q_len", q_len), ("k_len", k_len)):
        _int_vector(name, t, N, q.device)
    p = dcn4_band_params(N, Lq, k.shape[1], Hq, k.shape[2], D, left, right, sinks,
                         D ** -0.5 if scale is None else float(scale), nb, M, _dtype_code(q), qb, qr, kb, kr, vb, vr)
    check(dcn4_band_check_params(p))
    return p


def _same(name, t, shape, dtype, device, batch, row):
    """ValueError unless t is the tensor (its shape, device and all strides, 0 for dense ones) that the parameters
    are for.  A dimension of length 1 has no stride that matters."""
    N, L, H, D = shape
    row = row or H * D
    batch = batch or row * L
    ok = t.shape == shape and t.dtype == dtype and t.device == device
    if ok and t.stride() != (batch, row, D, 1) and t.numel():
        sb, sl, sh, sd = t.stride()
        ok = (N == 1 or sb == batch) and (L == 1 or sl == row) and (H == 1 or sh == D) and (D == 1 or sd == 1)
    if not ok:
        raise ValueError(f"{name} is not the tensor these parameters were made for")


def _on_gpu(q):
    if not q.is_cuda:
        raise ValueError("q and the other tensors must be on a CUDA device")


def _band_call(p, q, k, v, bias, buckets, *vectors):
    dt, keys = _torch_dtype(p.dtype), (p.N, p.Lk, p.Hk, p.D)
    _same("q", q, (p.N, p.Lq, p.Hq, p.D), dt, q.device, p.q_batch, p.q_row)
    _same("k", k, keys, dt, q.device, p.k_batch, p.k_row)
    _same("v", v, keys, dt, q.device, p.v_batch, p.v_row)
    if bias is not None and buckets is not None:
        _dense("bias", bias, (p.nb, p.Hq), dt, q.device)
        _int_vector("buckets", buckets, 2 * p.M + 1, q.device)
    for t in vectors:
        if t is not None:
            _int_vector("q_start, q_len or k_len", t, p.N, q.device)
    _on_gpu(q)


def band_forward(p: dcn4_band_params, q, k, v, bias=None, buckets=None, q_start=None, q_len=None, k_len=None, out=None):
    """(out [N, Lq, Hq, D], lse [N, Hq, Lq] fp32) of the dense attention over a band of keys,
    for CUDA tensors as band_params_for takes them."""
    import torch
    _band_call(p, q, k, v, bias, buckets, q_start, q_len, k_len)
    shape = (p.N, p.Lq, p.Hq, p.D)
    if out is None:
        out = _dense_like(q, shape)
    else:
        _dense("out", out, shape, q.dtype, q.device)
    lse = q.new_empty((p.N, p.Hq, p.Lq), dtype=torch.float32)
    need = dcn4_band_forward_workspace_size(p)
    ws = _workspace(need, q)
    _launch(q.device, dcn4_band_forward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(bias), _ptr(buckets),
            _ptr(q_start), _ptr(q_len), _ptr(k_len), out.data_ptr(), lse.data_ptr(), _ptr(ws), need)
    return out, lse


def band_backward(p: dcn4_band_params, q, k, v, out, lse, grad_out, bias=None, buckets=None, q_start=None, q_len=None,
                  k_len=None, want_bias: bool = True):
    """(grad_q, grad_k, grad_v, grad_bias or None) of band_forward, from its out and lse;
    grad_out [N, Lq, Hq, D] contiguous.  The gradients are dense."""
    import torch
    dev, dt = q.device, q.dtype
    _band_call(p, q, k, v, bias, buckets, q_start, q_len, k_len)
    for name, t in (("out", out), ("grad_out", grad_out)):
        _dense(name, t, (p.N, p.Lq, p.Hq, p.D), dt, dev)
    _dense("lse", lse, (p.N, p.Hq, p.Lq), torch.float32, dev)
    gq = torch.empty_like(grad_out)
    keys = (p.N, p.Lk, p.Hk, p.D)
    gk, gv = _dense_like(k, keys), _dense_like(v, keys)
    gb = torch.empty_like(bias) if bias is not None and want_bias else None
    need = dcn4_band_backward_workspace_size(p) if gb is not None else dcn4_band_backward_frozen_workspace_size(p)
    ws = _workspace(need, q)
    _launch(dev, dcn4_band_backward, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(bias), _ptr(buckets), _ptr(q_start),
            _ptr(q_len), _ptr(k_len), out.data_ptr(), lse.data_ptr(), grad_out.data_ptr(), gq.data_ptr(), gk.data_ptr(),
            gv.data_ptr(), _ptr(gb), _ptr(ws), need)
    return gq, gk, gv, gb


def qknorm_params_for(q, k, wq=None, wk=None, pos=None, inv_freq=None, *, interleaved: bool = False,
                      eps: float = 1e-6) -> dcn4_qknorm_params:
    """dcn4_qknorm_params for CUDA tensors q [N, L, Hq, D] and k [N, L, Hk, D] (views whose heads are
    contiguous), weights [D] or None, and for a rotation pos [N, L] or [N, L, axes] (float32) and
    inv_freq [R / 2] (float32); checks them on the host (ValueError, Dcn4Error)."""
    import torch
    qb, qr = _heads_strides("q", q, q.dtype, q.device)
    kb, kr = _heads_strides("k", k, q.dtype, q.device)
    N, L, Hq, D = q.shape
    if k.shape[:2] != q.shape[:2] or k.shape[3] != D:
        raise ValueError("q and k must be [N, L, Hq, D] and [N, L, Hk, D]")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _dense(name, w, (D,), q.dtype, q.device)
    if (pos is None) != (inv_freq is None):
        raise ValueError("pos and inv_freq come together")
    R, axes = 0, 1
    if pos is not None:
        if inv_freq.dim() != 1 or pos.dim() not in (2, 3):
            raise ValueError("pos must be [N, L] or [N, L, axes] and inv_freq [R / 2]")
        R, axes = 2 * inv_freq.shape[0], (pos.shape[2] if pos.dim() == 3 else 1)
        _dense("pos", pos, (N, L) + ((axes,) if pos.dim() == 3 else ()), torch.float32, q.device)
        _dense("inv_freq", inv_freq, (R // 2,), torch.float32, q.device)
    p = dcn4_qknorm_params(N, L, Hq, k.shape[2], D, R, axes, 1 if interleaved else 0, float(eps), _dtype_code(q),
                           qb, qr, kb, kr)
    check(dcn4_qknorm_check_params(p))
    return p


def _qknorm_call(p, q, k, wq, wk, pos, inv_freq):
    dt = _torch_dtype(p.dtype)
    _same("q", q, (p.N, p.L, p.Hq, p.D), dt, q.device, p.q_batch, p.q_row)
    _same("k", k, (p.N, p.L, p.Hk, p.D), dt, q.device, p.k_batch, p.k_row)
    for t, n, of in ((wq, p.D, dt), (wk, p.D, dt), (pos, p.N * p.L * p.axes, None), (inv_freq, p.R // 2, None)):
        if t is not None and (t.numel() != n or t.dtype != (of or _torch_dtype(DCN4_F32)) or not t.is_contiguous() or t.device != q.device):
            raise ValueError("a weight, pos or inv_freq is not the tensor these parameters were made for")
    _on_gpu(q)


def qknorm_forward(p: dcn4_qknorm_params, q, k, wq=None, wk=None, pos=None, inv_freq=None):
    """(q_out [N, L, Hq, D], k_out [N, L, Hk, D]): the heads of q and k RMS-normed, weighted and
    rotated by their positions, for CUDA tensors as qknorm_params_for takes them."""
    _qknorm_call(p, q, k, wq, wk, pos, inv_freq)
    qo, ko = _dense_like(q, (p.N, p.L, p.Hq, p.D)), _dense_like(k, (p.N, p.L, p.Hk, p.D))
    _launch(q.device, dcn4_qknorm_forward, p, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(pos), _ptr(inv_freq),
            qo.data_ptr(), ko.data_ptr())
    return qo, ko


def qknorm_backward(p: dcn4_qknorm_params, q, k, wq, wk, pos, inv_freq, grad_q_out, grad_k_out,
                    want_wq: bool = True, want_wk: bool = True):
    """(grad_q, grad_k, grad_wq or None, grad_wk or None) of qknorm_forward for contiguous
    gradients of its outputs; a weight that was None, or is not wanted, gets no gradient."""
    import torch
    dev, dt = q.device, q.dtype
    _qknorm_call(p, q, k, wq, wk, pos, inv_freq)
    _dense("grad_q_out", grad_q_out, (p.N, p.L, p.Hq, p.D), dt, dev)
    _dense("grad_k_out", grad_k_out, (p.N, p.L, p.Hk, p.D), dt, dev)
    gq, gk = torch.empty_like(grad_q_out), torch.empty_like(grad_k_out)
    gwq = torch.empty_like(wq) if wq is not None and want_wq else None
    gwk = torch.empty_like(wk) if wk is not None and want_wk else None
    need = dcn4_qknorm_backward_workspace_size(p) if gwq is not None or gwk is not None else 0
    ws = _workspace(need, q)
    _launch(dev, dcn4_qknorm_backward, p, q.data_ptr(), k.data_ptr(), _ptr(wq), _ptr(wk), _ptr(pos), _ptr(inv_freq),
            grad_q_out.data_ptr(), grad_k_out.data_ptr(), gq.data_ptr(), gk.data_ptr(), _ptr(gwq), _ptr(gwk), _ptr(ws), need)
    return gq, gk, gwq, gwk


def backward_diagnostics(p: dcn4_params, workspace) -> dict:
    """Fallback counters of the last backward on `workspace` (a uint8 CUDA tensor)."""
    st, c = dcn4_backward_diagnostics(p, workspace.data_ptr(), workspace.numel(), _stream_handle(workspace.device))
    check(st)
    return {"corrupt_bucket_tiles": c[0], "rescanned_tiles": c[1], "direct_tiles": c[2]}


# ---------------------------------------------------------------------------
# torch.autograd wrapper (argument marshalling only: both passes run in libdcn4)
# ---------------------------------------------------------------------------

_TORCH_CODES = None


def _dtype_code(t) -> int:
    import torch
    global _TORCH_CODES
    if _TORCH_CODES is None:
        _TORCH_CODES = {torch.float32: DCN4_F32, torch.float16: DCN4_F16, torch.bfloat16: DCN4_BF16}
    if t.dtype not in _TORCH_CODES:
        raise ValueError(f"dtype {t.dtype} is not float32, float16 or bfloat16")
    return _TORCH_CODES[t.dtype]


def _pair(v):
    return (v, v) if isinstance(v, int) else tuple(v)


def params_for_tensors(value, offset_mask, *, group: int, kernel=3, stride=1, pad=1, dilation=1,
                       offset_scale: float = 1.0, remove_center: bool = False,
                       softmax: bool = False) -> dcn4_params:
    """dcn4_params for NHWC value [N,H,W,C] and offset_mask [N,Ho,Wo,P]; checks shapes,
    dtypes, devices and contiguity on the host (ValueError) before anything is launched."""
    if value.dim() != 4 or offset_mask.dim() != 4:
        raise ValueError("value must be [N,H,W,C] and offset_mask [N,Ho,Wo,P]")
    if value.dtype != offset_mask.dtype:
        raise ValueError("value and offset_mask must have the same dtype")
    if not (value.is_contiguous() and offset_mask.is_contiguous()):
        raise ValueError("value and offset_mask must be contiguous (channels last)")
    N, H, W, C = value.shape
    if group < 1 or C % group != 0:
        raise ValueError(f"C={C} is not a multiple of group={group}")
    if not (value.is_cuda and offset_mask.is_cuda):
        raise ValueError("value and offset_mask must be CUDA tensors")
    if value.device != offset_mask.device:
        raise ValueError("value and offset_mask must be on the same device")
    (kh, kw), (sh, sw), (ph, pw), (dh, dw) = _pair(kernel), _pair(stride), _pair(pad), _pair(dilation)
    p = make_params(N=N, H=H, W=W, G=group, Cg=C // group, kh=kh, kw=kw, sh=sh, sw=sw, ph=ph, pw=pw, dh=dh,
                    dw=dw, offset_scale=float(offset_scale), remove_center=int(bool(remove_center)),
                    P=offset_mask.shape[-1], dtype={DCN4_F32: "f32", DCN4_F16: "f16", DCN4_BF16: "bf16"}[_dtype_code(value)],
                    softmax=int(bool(softmax)))
    st, Ho, Wo = dcn4_output_dims(p)
    check(st)
    if tuple(offset_mask.shape[:3]) != (N, Ho, Wo):
        raise ValueError(f"offset_mask must be [N={N}, Ho={Ho}, Wo={Wo}, P], got {tuple(offset_mask.shape)}")
    check(dcn4_check_params(p))
    return p


def _autograd_function():
    import torch

    class DCNv4Core(torch.autograd.Function):
        """The DCNv4 core aggregation as a torch.autograd.Function: forward and backward
        are dcn4_forward and dcn4_backward on the tensors' device and current stream."""

        @staticmethod
        def forward(ctx, value, offset_mask, p):
            ctx.save_for_backward(value, offset_mask)
            ctx.p = p
            return forward(p, value, offset_mask)

        @staticmethod
        def backward(ctx, grad_out):
            value, offset_mask = ctx.saved_tensors
            grad_value, grad_offset_mask = backward(ctx.p, value, offset_mask, grad_out.contiguous())
            return grad_value, grad_offset_mask, None

    return DCNv4Core


_DCNV4_CORE = None
_DCNV4_CORE_LINEAR = None
_DCNV4_CORE_PROJ = None
_BAND = None
_QKNORM = None


def _autograd_function_proj():
    import torch

    class DCNv4CoreProj(torch.autograd.Function):
        """The aggregation with the output projection fused behind it as a
        torch.autograd.Function.  Forward: dcn4_forward_proj, keeping the core output.
        Backward: dcn4_backward_proj (the projection's gradients in libdcn4's
        tensor-core kernels, then dcn4_backward with grad_core = grad_out W)."""

        @staticmethod
        def forward(ctx, value, offset_mask, weight, bias, p):
            st, Ho, Wo = dcn4_output_dims(p)
            check(st)
            core = torch.empty((p.N, Ho, Wo, p.G * p.Cg), dtype=value.dtype, device=value.device)
            y = forward_proj(p, value, offset_mask, weight, bias, core_out=core)
            ctx.save_for_backward(value, offset_mask, weight, core)
            ctx.p = p
            ctx.has_bias = bias is not None
            return y

        @staticmethod
        def backward(ctx, grad_out):
            value, offset_mask, weight, core = ctx.saved_tensors
            grad_value, grad_om, grad_w, grad_b = backward_proj(
                ctx.p, value, offset_mask, core, weight, grad_out.contiguous(), with_bias=ctx.has_bias,
                want_weight=ctx.needs_input_grad[2])
            return grad_value, grad_om, grad_w, grad_b, None

    return DCNv4CoreProj


def _autograd_function_linear():
    import torch

    class DCNv4CoreLinear(torch.autograd.Function):
        """The offset/mask linear layer fused into the aggregation as a
        torch.autograd.Function.  Forward: dcn4_forward_linear, keeping the
        offset_mask it formed.  Backward: dcn4_backward_linear, i.e. dcn4_backward on
        that offset_mask, then the linear layer's gradients (grad_x = g W,
        grad_W = g^T x, grad_b = sum g, with g = grad_offset_mask as [M, P]) in
        libdcn4's tensor-core kernels."""

        @staticmethod
        def forward(ctx, value, x, weight, bias, p):
            st, Ho, Wo = dcn4_output_dims(p)
            check(st)
            om = torch.empty((p.N, Ho, Wo, p.P), dtype=value.dtype, device=value.device)
            y = forward_linear(p, value, x, weight, bias, offset_mask_out=om)
            ctx.save_for_backward(value, x, weight, om)
            ctx.p = p
            ctx.has_bias = bias is not None
            return y

        @staticmethod
        def backward(ctx, grad_out):
            value, x, weight, om = ctx.saved_tensors
            grad_value, _, grad_x, grad_w, grad_b = backward_linear(
                ctx.p, value, om, x, weight, grad_out.contiguous(), with_bias=ctx.has_bias,
                want_x=ctx.needs_input_grad[1], want_weight=ctx.needs_input_grad[2])
            return grad_value, grad_x, grad_w, grad_b, None

    return DCNv4CoreLinear


def _autograd_function_band():
    import torch
    from torch.autograd.function import once_differentiable

    class BandAttention(torch.autograd.Function):
        """Dense attention over a band of keys as a torch.autograd.Function: dcn4_band_forward,
        keeping its output and log sums, and dcn4_band_backward."""

        @staticmethod
        def forward(ctx, q, k, v, bias, buckets, q_start, q_len, k_len, p):
            out, lse = band_forward(p, q, k, v, bias, buckets, q_start, q_len, k_len)
            ctx.save_for_backward(q, k, v, bias, buckets, q_start, q_len, k_len, out, lse)
            ctx.p = p
            return out

        @staticmethod
        @once_differentiable
        def backward(ctx, grad_out):
            q, k, v, bias, buckets, q_start, q_len, k_len, out, lse = ctx.saved_tensors
            grads = band_backward(ctx.p, q, k, v, out, lse, _upstream(grad_out), bias, buckets, q_start, q_len,
                                  k_len, want_bias=ctx.needs_input_grad[3])
            return grads + (None,) * 5

    return BandAttention


def _autograd_function_qknorm():
    import torch
    from torch.autograd.function import once_differentiable

    class QkNorm(torch.autograd.Function):
        """RMS norm and rotation of query and key heads as a torch.autograd.Function:
        dcn4_qknorm_forward and dcn4_qknorm_backward, which reads the inputs again."""

        @staticmethod
        def forward(ctx, q, k, wq, wk, pos, inv_freq, p):
            ctx.save_for_backward(q, k, wq, wk, pos, inv_freq)
            ctx.p = p
            return qknorm_forward(p, q, k, wq, wk, pos, inv_freq)

        @staticmethod
        @once_differentiable
        def backward(ctx, grad_q_out, grad_k_out):
            q, k, wq, wk, pos, inv_freq = ctx.saved_tensors
            grads = qknorm_backward(ctx.p, q, k, wq, wk, pos, inv_freq, _upstream(grad_q_out),
                                    _upstream(grad_k_out), *ctx.needs_input_grad[2:4])
            return grads + (None,) * 3

    return QkNorm


def band_attention(q, k, v, *, left=-1, right=-1, sinks=0, scale=None, bias=None, buckets=None, q_start=None,
                   q_len=None, k_len=None):
    """out [N, Lq, Hq, D] = dense attention of q [N, Lq, Hq, D] to the keys k, v [N, Lk, Hk, D] in a band
    around each query (`left` behind and `right` ahead of it, -1: all; the first `sinks` keys stay
    visible behind the window), with a learned bias [nb, Hq] by the buckets [2M + 1] of the relative
    position; differentiable in q, k, v and bias (torch.autograd)."""
    global _BAND
    p = band_params_for(q, k, v, left=left, right=right, sinks=sinks, scale=scale, bias=bias, buckets=buckets,
                        q_start=q_start, q_len=q_len, k_len=k_len)
    if _BAND is None:
        _BAND = _autograd_function_band()
    return _BAND.apply(q, k, v, bias, buckets, q_start, q_len, k_len, p)


def qk_norm_rotate(q, k, wq=None, wk=None, pos=None, inv_freq=None, *, interleaved: bool = False, eps: float = 1e-6):
    """(q, k) with every head RMS-normed, weighted (wq, wk [D] or None) and its first 2 * len(inv_freq)
    entries rotated by pos [N, L] or [N, L, axes]; differentiable in q, k, wq and wk (torch.autograd)."""
    global _QKNORM
    p = qknorm_params_for(q, k, wq, wk, pos, inv_freq, interleaved=interleaved, eps=eps)
    if _QKNORM is None:
        _QKNORM = _autograd_function_qknorm()
    return _QKNORM.apply(q, k, wq, wk, pos, inv_freq, p)


def dcnv4_core(value, offset_mask, *, group: int, kernel=3, stride=1, pad=1, dilation=1,
               offset_scale: float = 1.0, remove_center: bool = False, softmax: bool = False):
    """y = DCNv4 core aggregation of value [N,H,W,C] at the offsets and masks of
    offset_mask [N,Ho,Wo,P], differentiable in both (torch.autograd).  softmax=True
    takes the masks as logits normalised over the K points (the DCNv3 form)."""
    global _DCNV4_CORE
    p = params_for_tensors(value, offset_mask, group=group, kernel=kernel, stride=stride, pad=pad,
                           dilation=dilation, offset_scale=offset_scale, remove_center=remove_center,
                           softmax=softmax)
    if _DCNV4_CORE is None:
        _DCNV4_CORE = _autograd_function()
    return _DCNV4_CORE.apply(value, offset_mask, p)


def dcnv4_core_linear(value, x, weight, bias=None, *, group: int, kernel=3, stride=1, pad=1, dilation=1,
                      offset_scale: float = 1.0, remove_center: bool = False, softmax: bool = False):
    """y = DCNv4 core aggregation of value [N,H,W,C] at offset_mask = x @ weight.T + bias,
    formed inside the forward kernel (x [N,Ho,Wo,Cx], weight [P,Cx], bias [P] or None;
    fp16/bf16), differentiable in value, x, weight and bias (torch.autograd)."""
    global _DCNV4_CORE_LINEAR
    if weight.dim() != 2 or x.dim() != 4 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x must be [N,Ho,Wo,Cx] and weight [P,Cx]")
    if bias is not None and tuple(bias.shape) != (weight.shape[0],):
        raise ValueError("bias must be [P]")
    for name, t in (("x", x), ("weight", weight)) + ((("bias", bias),) if bias is not None else ()):
        if t.dtype != value.dtype or not t.is_contiguous() or t.device != value.device:
            raise ValueError(f"{name} must be contiguous, on value's device and of value's dtype")
    # the shape checks of the operator itself, on an offset_mask-shaped view of the producer
    N = value.shape[0]
    p = params_for_tensors(value, _OffsetMaskShape(x.shape[:3], weight.shape[0], value), group=group, kernel=kernel,
                           stride=stride, pad=pad, dilation=dilation, offset_scale=offset_scale,
                           remove_center=remove_center, softmax=softmax)
    if x.shape[0] != N:
        raise ValueError("x and value must have the same batch")
    if _DCNV4_CORE_LINEAR is None:
        _DCNV4_CORE_LINEAR = _autograd_function_linear()
    return _DCNV4_CORE_LINEAR.apply(value, x, weight, bias, p)


def dcnv4_core_proj(value, offset_mask, weight, bias=None, *, group: int, kernel=3, stride=1, pad=1, dilation=1,
                    offset_scale: float = 1.0, remove_center: bool = False, softmax: bool = False):
    """y = (DCNv4 core aggregation of value [N,H,W,C] at offset_mask [N,Ho,Wo,P]) @ weight.T
    + bias, the output projection (weight [Cout,C], bias [Cout] or None; fp16/bf16)
    formed inside the forward kernel; differentiable in value, offset_mask, weight and
    bias (torch.autograd)."""
    global _DCNV4_CORE_PROJ
    if weight.dim() != 2 or weight.shape[1] != value.shape[-1]:
        raise ValueError("weight must be [Cout, C]")
    if bias is not None and tuple(bias.shape) != (weight.shape[0],):
        raise ValueError("bias must be [Cout]")
    for name, t in (("weight", weight),) + ((("bias", bias),) if bias is not None else ()):
        if t.dtype != value.dtype or not t.is_contiguous() or t.device != value.device:
            raise ValueError(f"{name} must be contiguous, on value's device and of value's dtype")
    p = params_for_tensors(value, offset_mask, group=group, kernel=kernel, stride=stride, pad=pad,
                           dilation=dilation, offset_scale=offset_scale, remove_center=remove_center,
                           softmax=softmax)
    if _DCNV4_CORE_PROJ is None:
        _DCNV4_CORE_PROJ = _autograd_function_proj()
    return _DCNV4_CORE_PROJ.apply(value, offset_mask, weight, bias, p)


class _OffsetMaskShape:
    """Stands in for an offset_mask tensor [N,Ho,Wo,P] in params_for_tensors' checks."""

    def __init__(self, lead, P, like):
        self.shape = tuple(lead) + (int(P),)
        self.dtype = like.dtype
        self.is_cuda = like.is_cuda
        self.device = like.device

    def dim(self):
        return 4

    def is_contiguous(self):
        return True
