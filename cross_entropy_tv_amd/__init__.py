"""Fused cross-entropy + total-variation-distance loss for MI355X (gfx950).

Thin Python binding over the C ABI declared in ``include/lx_ce_tvd.h``: every
function here has the name of the C entry point it calls and only marshals
arguments (PyTorch tensors supply device memory and the HIP stream).  All of
the loss is computed by the HIP kernels in ``liblx_ce_tvd.so``; there is no
other code path.  Importing this package fails if the library is not built
(``python cross_entropy_tv_amd/build.py``).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblx_ce_tvd.so")

LX_OK = 0
LX_ERR_INVALID_ARG = 1
LX_ERR_UNSUPPORTED_DTYPE = 2
LX_ERR_ALIAS = 3
LX_ERR_WORKSPACE = 4
LX_ERR_HIP = 5
LX_ERR_TOO_LARGE = 6
LX_F32 = 0
LX_BF16 = 1
LX_F16 = 2


class LxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = lib.lx_status_string(status).decode()
        extra = f" (hipError {lib.lx_last_hip_error()})" if status == LX_ERR_HIP else ""
        super().__init__(f"{where}: {name}{extra}")


def _load() -> ctypes.CDLL:
    # PyTorch-ROCm ships its own HIP runtime and links it as "libamdhip64.so";
    # the library links "libamdhip64.so.7".  Importing torch first puts torch's
    # runtime in the process under that soname, so the library binds to it.
    # Loading the library first would start a second HIP runtime, whose
    # launches then fail with hipErrorNoDevice.
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python cross_entropy_tv_amd/build.py` "
                          "(the HIP library is the only implementation)")
    L = ctypes.CDLL(LIB_PATH)
    p, i64, f32, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    L.lx_status_string.argtypes = [i32]
    L.lx_status_string.restype = ctypes.c_char_p
    L.lx_abi_version.argtypes = []
    L.lx_abi_version.restype = i32
    L.lx_last_hip_error.argtypes = []
    L.lx_last_hip_error.restype = i32
    L.lx_ce_tvd_workspace_bytes.argtypes = [i64, i64, i32, i32]
    L.lx_ce_tvd_workspace_bytes.restype = sz
    L.lx_ce_tvd_forward.argtypes = [p, p, p, i64, i64, i64, p, p, p, p, p, i32, p, sz, p]
    L.lx_ce_tvd_forward.restype = i32
    L.lx_ce_tvd_backward.argtypes = [p, p, p, p, i64, i64, i64, p, p, p, f32, f32, p, i32, p]
    L.lx_ce_tvd_backward.restype = i32
    L.lx_ce_tvd_reduce_mean.argtypes = [p, p, p, i64, i64, p, p, p, p]
    L.lx_ce_tvd_reduce_mean.restype = i32
    L.lx_ce_tvd_forward_backward_workspace_bytes.argtypes = [i64, i64, i32, i32]
    L.lx_ce_tvd_forward_backward_workspace_bytes.restype = sz
    L.lx_ce_tvd_forward_backward.argtypes = [p, p, p, i64, i64, i64, p, p, p, p, p, p, f32, f32, p, i32, p, sz, p]
    L.lx_ce_tvd_forward_backward.restype = i32
    L.lx_ce_tvd_forward_backward_noalloc.argtypes = [p, p, p, i64, i64, i64, p, p, p, p, p, p, f32, f32, p, i32, p]
    L.lx_ce_tvd_forward_backward_noalloc.restype = i32
    L.lx_stream_read.argtypes = [p, i64, p, p]
    L.lx_stream_read.restype = i32
    L.lx_stream_read2_write.argtypes = [p, p, p, i64, p]
    L.lx_stream_read2_write.restype = i32
    L.lx_ce_tvd_count_valid.argtypes = [p, i64, i64, p, p, p]
    L.lx_ce_tvd_count_valid.restype = i32
    L.lx_ce_tvd_vp_stats.argtypes = [p, p, p, i64, i64, i64, i64, i32, p, p]
    L.lx_ce_tvd_vp_stats.restype = i32
    L.lx_ce_tvd_vp_merge_stats.argtypes = [p, i64, p, i64, i64, i64, i32, p, p, p, p]
    L.lx_ce_tvd_vp_merge_stats.restype = i32
    L.lx_ce_tvd_vp_tv.argtypes = [p, p, p, i64, i64, i64, p, p, i32, p, p]
    L.lx_ce_tvd_vp_tv.restype = i32
    L.lx_ce_tvd_vp_merge_tv.argtypes = [p, i64, p, i64, i64, p, p, p]
    L.lx_ce_tvd_vp_merge_tv.restype = i32
    L.lx_ce_tvd_backward_shard.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, p, p, p, f32, f32, p, i32, p]
    L.lx_ce_tvd_backward_shard.restype = i32
    L.lx_ce_tvd_forward_ex.argtypes = [p, i64, p, i64, p, i64, i64, i64, p, p, p, p, p, i32, p, sz, p]
    L.lx_ce_tvd_forward_ex.restype = i32
    L.lx_ce_tvd_backward_ex.argtypes = [p, i64, p, i64, p, i64, p, i64, i64, i64, p, p, p, f32, f32, p, p, p, i32, p]
    L.lx_ce_tvd_backward_ex.restype = i32
    L.lx_ce_tvd_forward_backward_ex.argtypes = [p, i64, p, i64, p, i64, i64, i64, p, p, p, p, p, p, i64, f32, f32,
                                                p, p, p, i32, p, sz, p]
    L.lx_ce_tvd_forward_backward_ex.restype = i32
    L.lx_gemm_bf16.argtypes = [p, i64, i32, p, i64, i32, p, i64, i64, i64, i64, i32, p]
    L.lx_gemm_bf16.restype = i32
    L.lx_ce_tvd_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i64]
    L.lx_ce_tvd_linear_workspace_bytes.restype = sz
    L.lx_ce_tvd_linear_forward_backward.argtypes = [p, p, i64, p, p, i64, p, i64, i64, i64, p, p, p, p, p, p, p,
                                                    f32, f32, p, i64, p, sz, p]
    L.lx_ce_tvd_linear_forward_backward.restype = i32
    L.lx_draft_verify_workspace_bytes.argtypes = [i64, i64, i64]
    L.lx_draft_verify_workspace_bytes.restype = sz
    L.lx_draft_verify.argtypes = [p, i64, p, i64, p, p, i64, i64, i64, i64, p, p, p, p, p, p, i32, p, sz, p]
    L.lx_draft_verify.restype = i32
    L.lx_lora_forward_workspace_bytes.argtypes = [i64] * 5
    L.lx_lora_forward_workspace_bytes.restype = sz
    L.lx_lora_forward.argtypes = [p, i64, p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, p, i64, i32, p, i64, i32, p, sz,
                                  p]
    L.lx_lora_forward.restype = i32
    L.lx_lora_backward_workspace_bytes.argtypes = [i64] * 6
    L.lx_lora_backward_workspace_bytes.restype = sz
    L.lx_lora_backward.argtypes = [p, i64, p, i64, p, p, p, p, p, p, i64, i64, i64, i64, i64, i64, p, i64, p, i64, p, p, p,
                                   sz, p]
    L.lx_lora_backward.restype = i32
    L.lx_top_logits_workspace_bytes.argtypes = [i64, i64, i64]
    L.lx_top_logits_workspace_bytes.restype = sz
    L.lx_top_logits.argtypes = [p, i64, i64, i64, i64, f32, p, p, p, p, i32, p, sz, p]
    L.lx_top_logits.restype = i32
    for name in ("lx_ce_kd_workspace_bytes", "lx_ce_kd_forward_backward_workspace_bytes"):
        getattr(L, name).argtypes = [i64, i64, i32]
        getattr(L, name).restype = sz
    L.lx_ce_kd_forward.argtypes = [p, i64, p, p, p, p, i64, i64, i64, i64, f32, p, p, p, p, i32, p, sz, p]
    L.lx_ce_kd_forward.restype = i32
    L.lx_ce_kd_backward.argtypes = [p, i64, p, i64, p, p, p, i64, i64, i64, i64, f32, p, p, f32, f32, p, p, p, i32, p]
    L.lx_ce_kd_backward.restype = i32
    L.lx_ce_kd_forward_backward.argtypes = [p, i64, p, p, p, p, i64, i64, i64, i64, f32, p, p, p, p, p, i64, f32, f32, p, p,
                                            p, i32, p, sz, p]
    L.lx_ce_kd_forward_backward.restype = i32
    L.lx_ce_kd_linear_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i32]
    L.lx_ce_kd_linear_workspace_bytes.restype = sz
    L.lx_ce_kd_linear_forward_backward.argtypes = [p, p, i64, p, p, p, p, i64, i64, i64, i64, f32, p, p, p, p, p, p, i32,
                                                   f32, f32, p, p, p, i64, p, sz, p]
    L.lx_ce_kd_linear_forward_backward.restype = i32
    return L


lib = _load()

import torch  # noqa: E402  (already loaded, see _load)


# ------------------------------------------------------------------ marshalling helpers

def _ptr(t):
    return None if t is None else t.data_ptr()


_DTYPE_CODES = {torch.float32: LX_F32, torch.bfloat16: LX_BF16, torch.float16: LX_F16}


def _dtype_code(t) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _stream(stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _logits2d(t, name):
    if t.dim() != 2 or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous 2-D (BT, V) device tensor")
    return t.shape


def _rows2d(t, name):
    """(BT, V, row stride) of a 2-D device tensor whose rows are contiguous."""
    if t.dim() != 2 or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D (BT, V) device tensor with contiguous rows")
    BT, V = t.shape
    return BT, V, (t.stride(0) if BT > 1 else V)


def _arg(t, name, dtype, shape, device):
    """Refuses t unless it is a contiguous tensor of this dtype and shape on this device."""
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


# The current stream's handle, without the stream object around it (3 us a call).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Launch:
    """The device, stream and workspace of one call: the device of its tensors is made
    current (a stream belongs to a device), the stream is the given one or that device's
    current one, and a workspace allocated here comes from the memory of the stream that
    uses it."""

    __slots__ = ("device", "stream", "guard", "ptr")

    def __init__(self, device, stream):
        self.device, self.stream, self.guard = device, stream, None

    def __enter__(self):
        index = self.device.index
        if self.stream is None:
            self.ptr = _current_raw_stream(index)
        else:
            if getattr(self.stream, "device", self.device) != self.device:
                raise ValueError(f"stream must be one of {self.device}, got one of {self.stream.device}")
            self.ptr = _stream(self.stream)
        if _current_device() != index:  # (last: nothing behind it can fail and leave the device changed)
            self.guard = torch.cuda.device(index)
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def workspace(self, given, need):
        """(address, bytes, the tensor that holds them) of the given workspace or of a new one."""
        if given is not None:
            if given.device != self.device:
                raise ValueError(f"workspace must be on {self.device}")
        elif self.stream is None:
            given = torch.empty(need, dtype=torch.uint8, device=self.device)
            return given.data_ptr(), need, given
        else:
            s = self.stream if hasattr(self.stream, "cuda_stream") else torch.cuda.ExternalStream(self.ptr)
            with torch.cuda.stream(s):
                given = torch.empty(need, dtype=torch.uint8, device=self.device)
        return given.data_ptr(), given.numel() * given.element_size(), given


def _check(status: int, where: str) -> None:
    if status != LX_OK:
        raise LxError(status, where)


# ------------------------------------------------------------------ entry points

def lx_status_string(status: int) -> str:
    return lib.lx_status_string(status).decode()


def lx_abi_version() -> int:
    return lib.lx_abi_version()


def lx_ce_tvd_workspace_bytes(BT: int, V: int, dt: int, has_teacher: bool) -> int:
    return lib.lx_ce_tvd_workspace_bytes(BT, V, dt, int(bool(has_teacher)))


def lx_ce_tvd_forward(student, teacher, target, ignore_index, ce, tvd, lse_s, lse_t, sigma,
                      workspace=None, stream=None) -> None:
    """Forward pass into the caller's float32 [BT] output tensors (tvd, lse_t, sigma
    may be None in CE-only mode, i.e. teacher=None).  ``workspace`` is a uint8
    device tensor of at least lx_ce_tvd_workspace_bytes bytes; when None and the
    shape needs one, it is allocated here with torch."""
    BT, V = _logits2d(student, "student")
    dt = _dtype_code(student)
    if teacher is not None and (teacher.shape != student.shape or teacher.dtype != student.dtype):
        raise ValueError("teacher must match student in shape and dtype")
    need = lx_ce_tvd_workspace_bytes(BT, V, dt, teacher is not None)
    if workspace is None and need:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=student.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.lx_ce_tvd_forward(_ptr(student), _ptr(teacher), _ptr(target), BT, V, int(ignore_index),
                                 _ptr(ce), _ptr(tvd), _ptr(lse_s), _ptr(lse_t), _ptr(sigma), dt,
                                 _ptr(workspace), wbytes, _stream(stream)), "lx_ce_tvd_forward")


def lx_ce_tvd_backward(grad, student, teacher, target, ignore_index, lse_s, lse_t, sigma,
                       g_ce: float, g_tvd: float, g_scale=None, stream=None) -> None:
    """Backward pass into ``grad`` (may be ``student`` itself).  ``g_scale`` is an
    optional float32 device tensor of one element multiplying g_ce and g_tvd."""
    BT, V = _logits2d(student, "student")
    dt = _dtype_code(student)
    if grad.shape != student.shape or grad.dtype != student.dtype or not grad.is_contiguous():
        raise ValueError("grad must match student in shape and dtype and be contiguous")
    _check(lib.lx_ce_tvd_backward(_ptr(grad), _ptr(student), _ptr(teacher), _ptr(target), BT, V,
                                  int(ignore_index), _ptr(lse_s), _ptr(lse_t), _ptr(sigma),
                                  float(g_ce), float(g_tvd), _ptr(g_scale), dt, _stream(stream)),
           "lx_ce_tvd_backward")


def lx_ce_tvd_forward_backward_workspace_bytes(BT: int, V: int, dt: int, has_teacher: bool) -> int:
    return lib.lx_ce_tvd_forward_backward_workspace_bytes(BT, V, dt, int(bool(has_teacher)))


def lx_ce_tvd_forward_backward(student, teacher, target, ignore_index, ce, tvd, lse_s, lse_t, sigma, grad,
                               g_ce: float, g_tvd: float, g_scale=None, workspace=None, stream=None) -> None:
    """Forward outputs and the student gradient in one call (``grad`` may be
    ``student``).  ``workspace`` as in lx_ce_tvd_forward, sized by
    lx_ce_tvd_forward_backward_workspace_bytes."""
    BT, V = _logits2d(student, "student")
    dt = _dtype_code(student)
    if teacher is not None and (teacher.shape != student.shape or teacher.dtype != student.dtype):
        raise ValueError("teacher must match student in shape and dtype")
    if grad.shape != student.shape or grad.dtype != student.dtype or not grad.is_contiguous():
        raise ValueError("grad must match student in shape and dtype and be contiguous")
    need = lx_ce_tvd_forward_backward_workspace_bytes(BT, V, dt, teacher is not None)
    if workspace is None and need:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=student.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.lx_ce_tvd_forward_backward(_ptr(student), _ptr(teacher), _ptr(target), BT, V, int(ignore_index),
                                          _ptr(ce), _ptr(tvd), _ptr(lse_s), _ptr(lse_t), _ptr(sigma), _ptr(grad),
                                          float(g_ce), float(g_tvd), _ptr(g_scale), dt, _ptr(workspace), wbytes,
                                          _stream(stream)), "lx_ce_tvd_forward_backward")


def lx_ce_tvd_forward_backward_noalloc(student, teacher, target, ignore_index, ce, tvd, lse_s, lse_t, sigma, grad,
                                       g_ce: float, g_tvd: float, g_scale=None, stream=None) -> None:
    """lx_ce_tvd_forward_backward with its scratch memory in the library's static
    device buffer instead of a workspace (nothing is allocated; calls that
    overlap on one device race)."""
    BT, V = _logits2d(student, "student")
    dt = _dtype_code(student)
    if teacher is not None and (teacher.shape != student.shape or teacher.dtype != student.dtype):
        raise ValueError("teacher must match student in shape and dtype")
    if grad.shape != student.shape or grad.dtype != student.dtype or not grad.is_contiguous():
        raise ValueError("grad must match student in shape and dtype and be contiguous")
    _check(lib.lx_ce_tvd_forward_backward_noalloc(_ptr(student), _ptr(teacher), _ptr(target), BT, V,
                                                  int(ignore_index), _ptr(ce), _ptr(tvd), _ptr(lse_s), _ptr(lse_t),
                                                  _ptr(sigma), _ptr(grad), float(g_ce), float(g_tvd), _ptr(g_scale),
                                                  dt, _stream(stream)), "lx_ce_tvd_forward_backward_noalloc")


def lx_ce_tvd_count_valid(target, ignore_index, n_valid=None, inv_n_valid=None, stream=None) -> None:
    """Number of non-ignored rows (int64 [1]) and its reciprocal (float32 [1])."""
    BT = target.shape[0]
    _check(lib.lx_ce_tvd_count_valid(_ptr(target), BT, int(ignore_index), _ptr(n_valid), _ptr(inv_n_valid),
                                     _stream(stream)), "lx_ce_tvd_count_valid")


def lx_ce_tvd_reduce_mean(ce, tvd, target, ignore_index, mean_out, n_valid=None, inv_n_valid=None,
                          stream=None) -> None:
    """Mean of ce (and tvd) over non-ignored rows into mean_out (float32 [2])."""
    BT = target.shape[0]
    _check(lib.lx_ce_tvd_reduce_mean(_ptr(ce), _ptr(tvd), _ptr(target), BT, int(ignore_index),
                                     _ptr(mean_out), _ptr(n_valid), _ptr(inv_n_valid), _stream(stream)),
           "lx_ce_tvd_reduce_mean")


def lx_vp_stats_floats(has_teacher: bool) -> int:
    return 5 if has_teacher else 3


def lx_ce_tvd_vp_stats(student, teacher, target, v0, ignore_index, stats, stream=None) -> None:
    """Step-1 partials of a column shard (student / teacher (BT, V_shard), the shard's
    first column v0) into ``stats``, float32 [BT, 5] (CE-only: [BT, 3])."""
    BT, Vs = _logits2d(student, "student")
    dt = _dtype_code(student)
    if teacher is not None and (teacher.shape != student.shape or teacher.dtype != student.dtype):
        raise ValueError("teacher must match student in shape and dtype")
    _check(lib.lx_ce_tvd_vp_stats(_ptr(student), _ptr(teacher), _ptr(target), BT, Vs, int(v0), int(ignore_index),
                                  dt, _ptr(stats), _stream(stream)), "lx_ce_tvd_vp_stats")


def lx_ce_tvd_vp_merge_stats(stats, target, V, ignore_index, ce, lse_s, lse_t=None, stream=None) -> None:
    """Merge of gathered step-1 partials, ``stats`` float32 [n_shards, BT, 5 or 3]."""
    n, BT, P = stats.shape
    _check(lib.lx_ce_tvd_vp_merge_stats(_ptr(stats), n, _ptr(target), BT, int(V), int(ignore_index), int(P == 5),
                                        _ptr(ce), _ptr(lse_s), _ptr(lse_t), _stream(stream)),
           "lx_ce_tvd_vp_merge_stats")


def lx_ce_tvd_vp_tv(student, teacher, target, ignore_index, lse_s, lse_t, tv, stream=None) -> None:
    """Step-2 partials of a column shard into ``tv``, float32 [BT, 2]."""
    BT, Vs = _logits2d(student, "student")
    dt = _dtype_code(student)
    if teacher is None or teacher.shape != student.shape or teacher.dtype != student.dtype:
        raise ValueError("teacher must be given and match student in shape and dtype")
    _check(lib.lx_ce_tvd_vp_tv(_ptr(student), _ptr(teacher), _ptr(target), BT, Vs, int(ignore_index), _ptr(lse_s),
                               _ptr(lse_t), dt, _ptr(tv), _stream(stream)), "lx_ce_tvd_vp_tv")


def lx_ce_tvd_vp_merge_tv(tv, target, ignore_index, tvd, sigma, stream=None) -> None:
    """Merge of gathered step-2 partials, ``tv`` float32 [n_shards, BT, 2]."""
    n, BT, _ = tv.shape
    _check(lib.lx_ce_tvd_vp_merge_tv(_ptr(tv), n, _ptr(target), BT, int(ignore_index), _ptr(tvd), _ptr(sigma),
                                     _stream(stream)), "lx_ce_tvd_vp_merge_tv")


def lx_ce_tvd_backward_shard(grad, student, teacher, target, v0, V, ignore_index, lse_s, lse_t, sigma,
                             g_ce: float, g_tvd: float, g_scale=None, stream=None) -> None:
    """Backward of a column shard (columns [v0, v0 + V_shard) of rows of V)."""
    BT, Vs = _logits2d(student, "student")
    dt = _dtype_code(student)
    if grad.shape != student.shape or grad.dtype != student.dtype or not grad.is_contiguous():
        raise ValueError("grad must match student in shape and dtype and be contiguous")
    _check(lib.lx_ce_tvd_backward_shard(_ptr(grad), _ptr(student), _ptr(teacher), _ptr(target), BT, Vs, int(v0),
                                        int(V), int(ignore_index), _ptr(lse_s), _ptr(lse_t), _ptr(sigma),
                                        float(g_ce), float(g_tvd), _ptr(g_scale), dt, _stream(stream)),
           "lx_ce_tvd_backward_shard")


def lx_ce_tvd_forward_ex(student, teacher, target, ignore_index, ce, tvd, lse_s, lse_t, sigma,
                         workspace=None, stream=None) -> None:
    """lx_ce_tvd_forward on row-strided views: each of student / teacher may be any
    2-D view with contiguous rows (its stride(0) is passed as the row stride)."""
    BT, V, lds = _rows2d(student, "student")
    dt = _dtype_code(student)
    ldt = V
    if teacher is not None:
        if teacher.shape != student.shape or teacher.dtype != student.dtype:
            raise ValueError("teacher must match student in shape and dtype")
        ldt = _rows2d(teacher, "teacher")[2]
    need = lx_ce_tvd_workspace_bytes(BT, V, dt, teacher is not None)
    if workspace is None and need:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=student.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.lx_ce_tvd_forward_ex(_ptr(student), lds, _ptr(teacher), ldt, _ptr(target), BT, V, int(ignore_index),
                                    _ptr(ce), _ptr(tvd), _ptr(lse_s), _ptr(lse_t), _ptr(sigma), dt,
                                    _ptr(workspace), wbytes, _stream(stream)), "lx_ce_tvd_forward_ex")


def lx_ce_tvd_backward_ex(grad, student, teacher, target, ignore_index, lse_s, lse_t, sigma, g_ce: float,
                          g_tvd: float, grad_ce_rows=None, grad_tvd_rows=None, g_scale=None, stream=None) -> None:
    """lx_ce_tvd_backward on row-strided views, with optional per-row factors
    ``grad_ce_rows`` / ``grad_tvd_rows`` (float32 [BT] device tensors)."""
    BT, V, lds = _rows2d(student, "student")
    dt = _dtype_code(student)
    if grad.shape != student.shape or grad.dtype != student.dtype:
        raise ValueError("grad must match student in shape and dtype")
    ldg = _rows2d(grad, "grad")[2]
    ldt = V if teacher is None else _rows2d(teacher, "teacher")[2]
    _check(lib.lx_ce_tvd_backward_ex(_ptr(grad), ldg, _ptr(student), lds, _ptr(teacher), ldt, _ptr(target), BT, V,
                                     int(ignore_index), _ptr(lse_s), _ptr(lse_t), _ptr(sigma), float(g_ce),
                                     float(g_tvd), _ptr(grad_ce_rows), _ptr(grad_tvd_rows), _ptr(g_scale), dt,
                                     _stream(stream)), "lx_ce_tvd_backward_ex")


def lx_ce_tvd_forward_backward_ex(student, teacher, target, ignore_index, ce, tvd, lse_s, lse_t, sigma, grad,
                                  g_ce: float, g_tvd: float, grad_ce_rows=None, grad_tvd_rows=None, g_scale=None,
                                  workspace=None, stream=None) -> None:
    """lx_ce_tvd_forward_backward on row-strided views, with optional per-row factors."""
    BT, V, lds = _rows2d(student, "student")
    dt = _dtype_code(student)
    ldt = V
    if teacher is not None:
        if teacher.shape != student.shape or teacher.dtype != student.dtype:
            raise ValueError("teacher must match student in shape and dtype")
        ldt = _rows2d(teacher, "teacher")[2]
    if grad.shape != student.shape or grad.dtype != student.dtype:
        raise ValueError("grad must match student in shape and dtype")
    ldg = _rows2d(grad, "grad")[2]
    need = lx_ce_tvd_forward_backward_workspace_bytes(BT, V, dt, teacher is not None)
    if workspace is None and need:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=student.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.lx_ce_tvd_forward_backward_ex(_ptr(student), lds, _ptr(teacher), ldt, _ptr(target), BT, V,
                                             int(ignore_index), _ptr(ce), _ptr(tvd), _ptr(lse_s), _ptr(lse_t),
                                             _ptr(sigma), _ptr(grad), ldg, float(g_ce), float(g_tvd),
                                             _ptr(grad_ce_rows), _ptr(grad_tvd_rows), _ptr(g_scale), dt,
                                             _ptr(workspace), wbytes, _stream(stream)),
           "lx_ce_tvd_forward_backward_ex")


def lx_gemm_bf16(A, a_k_contiguous: bool, B, b_k_contiguous: bool, C, M: int, N: int, K: int,
                 accumulate: bool = False, stream=None) -> None:
    """C[m][n] (+)= sum_k A(m, k) B(n, k) on bf16 device tensors A, B (2-D, rows contiguous)
    and a float32 2-D C.  A(m, k) is A[m, k] when a_k_contiguous else A[k, m]; likewise B."""
    import torch
    for t, name in ((A, "A"), (B, "B")):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError(f"{name} must be a 2-D bfloat16 tensor with contiguous rows")
    if C.dtype != torch.float32 or C.dim() != 2 or C.stride(1) != 1:
        raise ValueError("C must be a 2-D float32 tensor with contiguous rows")
    _check(lib.lx_gemm_bf16(_ptr(A), A.stride(0), int(bool(a_k_contiguous)), _ptr(B), B.stride(0),
                            int(bool(b_k_contiguous)), _ptr(C), C.stride(0), int(M), int(N), int(K),
                            int(bool(accumulate)), _stream(stream)), "lx_gemm_bf16")


def lx_ce_tvd_linear_workspace_bytes(BT: int, V: int, H_s: int, has_teacher: bool, chunk_rows: int) -> int:
    return lib.lx_ce_tvd_linear_workspace_bytes(BT, V, H_s, int(bool(has_teacher)), chunk_rows)


def lx_ce_tvd_linear_forward_backward(x_s, w_s, x_t, w_t, target, ignore_index, ce, tvd, lse_s, lse_t, sigma,
                                      grad_x_s, grad_w_s, g_ce: float, g_tvd: float, g_scale=None,
                                      chunk_rows: int | None = None, workspace=None, stream=None) -> None:
    """lm_head products and the CE + TVD loss: x_s (BT, H_s), w_s (V, H_s), x_t / w_t (or None)
    contiguous bfloat16; grad_x_s (BT, H_s) / grad_w_s (V, H_s) float32 or None.  The workspace
    (uint8 device tensor) is allocated here with torch when not given."""
    import torch
    BT, H_s = x_s.shape
    V = w_s.shape[0]
    H_t = 0 if x_t is None else x_t.shape[1]
    for t, name in ((x_s, "x_s"), (w_s, "w_s"), (x_t, "x_t"), (w_t, "w_t")):
        if t is not None and (t.dtype != torch.bfloat16 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous bfloat16 tensor")
    chunk = BT if chunk_rows is None else int(chunk_rows)
    need = lx_ce_tvd_linear_workspace_bytes(BT, V, x_s.shape[1], x_t is not None, chunk)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x_s.device)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.lx_ce_tvd_linear_forward_backward(_ptr(x_s), _ptr(w_s), H_s, _ptr(x_t), _ptr(w_t), H_t, _ptr(target),
                                                 BT, V, int(ignore_index), _ptr(ce), _ptr(tvd), _ptr(lse_s),
                                                 _ptr(lse_t), _ptr(sigma), _ptr(grad_x_s), _ptr(grad_w_s),
                                                 float(g_ce), float(g_tvd), _ptr(g_scale), chunk, _ptr(workspace),
                                                 wbytes, _stream(stream)), "lx_ce_tvd_linear_forward_backward")


def lx_draft_verify_workspace_bytes(S: int, max_draft: int, V: int) -> int:
    return lib.lx_draft_verify_workspace_bytes(S, max_draft, V)


def lx_draft_verify(target, draft, draft_tokens, draft_start, max_draft: int, temperature, u_accept, u_sample,
                    n_accepted, tokens, logprobs=None, workspace=None, stream=None) -> None:
    """Verification of S sequences' drafted tokens: ``target`` (N + S, V) and ``draft`` (N, V)
    or None, 2-D with contiguous rows; ``draft_tokens`` int64 [N], ``draft_start`` int64
    [S + 1]; ``temperature`` float32 [S] or None, ``u_accept`` float32 [N], ``u_sample``
    float32 [S]; into ``n_accepted`` int64 [S], ``tokens`` int64 [S, max_draft + 1] and
    ``logprobs`` float32 [S, max_draft + 1] or None.  The workspace (uint8 device tensor) is
    allocated here with torch when not given."""
    rows, V, ldt = _rows2d(target, "target")
    dt, dev, max_draft = _dtype_code(target), target.device, int(max_draft)
    N, S = draft_tokens.shape[0], u_sample.shape[0]
    if rows != N + S:
        raise ValueError(f"target must have a row per draft and one per sequence, {N} + {S}, got {rows}")
    ldd = V
    if draft is not None:
        if draft.shape != (N, V) or draft.dtype != target.dtype or draft.device != dev:
            raise ValueError(f"draft must be ({N}, {V}), of target's dtype and on its device")
        ldd = _rows2d(draft, "draft")[2]
    f32, i64 = torch.float32, torch.int64
    _arg(draft_tokens, "draft_tokens", i64, (N,), dev)
    _arg(draft_start, "draft_start", i64, (S + 1,), dev)
    if temperature is not None:
        _arg(temperature, "temperature", f32, (S,), dev)
    _arg(u_accept, "u_accept", f32, (N,), dev)
    _arg(u_sample, "u_sample", f32, (S,), dev)
    _arg(n_accepted, "n_accepted", i64, (S,), dev)
    _arg(tokens, "tokens", i64, (S, max_draft + 1), dev)
    if logprobs is not None:
        _arg(logprobs, "logprobs", f32, (S, max_draft + 1), dev)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_draft_verify_workspace_bytes(S, max_draft, V))
        _check(lib.lx_draft_verify(_ptr(target), ldt, _ptr(draft), ldd, _ptr(draft_tokens), _ptr(draft_start), S, N,
                                   max_draft, V, _ptr(temperature), _ptr(u_accept), _ptr(u_sample),
                                   _ptr(n_accepted), _ptr(tokens), _ptr(logprobs), dt, ws, wbytes, at.ptr),
               "lx_draft_verify")


def lx_lora_forward_workspace_bytes(T: int, R: int, H: int, N: int, r: int) -> int:
    return lib.lx_lora_forward_workspace_bytes(T, R, H, N, r)


def lx_lora_backward_workspace_bytes(T: int, R: int, n_adapters: int, H: int, N: int, r: int) -> int:
    return lib.lx_lora_backward_workspace_bytes(T, R, n_adapters, H, N, r)


def _rows_of(t, name, dtypes, rows, cols, dev):
    """The row stride of a 2-D (rows, cols) device tensor with contiguous rows, of one of these dtypes."""
    if t.dtype not in dtypes or t.shape != (rows, cols) or t.device != dev:
        raise ValueError(f"{name} must be ({rows}, {cols}) on {dev}, {' or '.join(map(str, dtypes))}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if rows > 1 else cols


_ONLY_BF16, _ONLY_F32, _F32_OR_BF16 = (torch.bfloat16,), (torch.float32,), (torch.float32, torch.bfloat16)


def _lora_set(x, A, B, adapter, req_start, scale, rank):
    """(T, R, n_adapters, H, N, r, device, x's row stride, the pointers of A .. rank) of the arguments that both
    directions take, checked."""
    dev, bf16, i64, a, b = x.device, torch.bfloat16, torch.int64, A.shape, B.shape
    if len(a) != 3 or len(b) != 3 or a[0] != b[0] or a[1] != b[2]:
        raise ValueError("A must be (n_adapters, r, H) and B (n_adapters, N, r)")
    (n, r, H), N, R, T = a, b[1], adapter.shape[0], x.shape[0]
    ldx = _rows_of(x, "x", _ONLY_BF16, T, H, dev)
    _arg(A, "A", bf16, a, dev)
    _arg(B, "B", bf16, b, dev)
    _arg(adapter, "adapter", i64, (R,), dev)
    _arg(req_start, "req_start", i64, (R + 1,), dev)
    _arg(scale, "scale", torch.float32, (n,), dev)
    if rank is not None:
        _arg(rank, "rank", i64, (n,), dev)
    if not x.is_cuda:
        raise ValueError("x must be a device tensor, and the others on its device")
    return T, R, n, H, N, r, dev, ldx, (A.data_ptr(), B.data_ptr(), adapter.data_ptr(), req_start.data_ptr(),
                                        scale.data_ptr(), None if rank is None else rank.data_ptr())


def lx_lora_forward(x, A, B, adapter, req_start, scale, rank, base, y, workspace=None, stream=None) -> None:
    """y = base + scale (x A^T) B^T with each request's adapter: ``x`` (T, H) bfloat16; ``A``
    (n_adapters, r, H) and ``B`` (n_adapters, N, r) bfloat16; ``adapter`` int64 [R],
    ``req_start`` int64 [R + 1]; ``scale`` float32 [n_adapters], ``rank`` int64 [n_adapters]
    or None; ``base`` (T, N) or None and ``y`` (T, N), float32 or bfloat16 each (``y`` may be
    ``base``).  The workspace is allocated here with torch when not given."""
    T, R, n, H, N, r, dev, ldx, set_ = _lora_set(x, A, B, adapter, req_start, scale, rank)
    base_ptr, ldb, base_dt = None, N, LX_F32
    if base is not None:
        base_ptr, ldb, base_dt = base.data_ptr(), _rows_of(base, "base", _F32_OR_BF16, T, N, dev), _dtype_code(base)
    ldy = _rows_of(y, "y", _F32_OR_BF16, T, N, dev)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_lora_forward_workspace_bytes(T, R, H, N, r))
        _check(lib.lx_lora_forward(x.data_ptr(), ldx, *set_, T, R, n, H, N, r, base_ptr, ldb, base_dt, y.data_ptr(), ldy,
                                   _dtype_code(y), ws, wbytes, at.ptr), "lx_lora_forward")


def lx_lora_backward(grad_y, x, A, B, adapter, req_start, scale, rank, base, grad_x, grad_A, grad_B, workspace=None,
                     stream=None) -> None:
    """The gradients of lx_lora_forward: ``grad_y`` (T, N) bfloat16 and its inputs, into
    ``grad_x`` (T, H) (``base`` or 0 added; may be ``base``), ``grad_A`` and ``grad_B`` (as A
    and B), float32, each or None; grad_A and grad_B are overwritten."""
    T, R, n, H, N, r, dev, ldx, set_ = _lora_set(x, A, B, adapter, req_start, scale, rank)
    lddy = _rows_of(grad_y, "grad_y", _ONLY_BF16, T, N, dev)
    ldb = H if base is None else _rows_of(base, "base", _ONLY_F32, T, H, dev)
    ldgx = H if grad_x is None else _rows_of(grad_x, "grad_x", _ONLY_F32, T, H, dev)
    if grad_A is not None:
        _arg(grad_A, "grad_A", torch.float32, (n, r, H), dev)
    if grad_B is not None:
        _arg(grad_B, "grad_B", torch.float32, (n, N, r), dev)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_lora_backward_workspace_bytes(T, R, n, H, N, r))
        _check(lib.lx_lora_backward(grad_y.data_ptr(), lddy, x.data_ptr(), ldx, *set_, T, R, n, H, N, r, _ptr(base), ldb,
                                    _ptr(grad_x), ldgx, _ptr(grad_A), _ptr(grad_B), ws, wbytes, at.ptr),
               "lx_lora_backward")


LX_KD_MAX_TOP, LX_KD_STATE_FLOATS = 256, 4


def lx_top_logits_workspace_bytes(BT: int, V: int, K: int) -> int:
    return lib.lx_top_logits_workspace_bytes(BT, V, K)


def lx_top_logits(logits, temperature: float, top, ids, lse=None, lse_rest=None, workspace=None, stream=None) -> None:
    """The K largest logits of every row of ``logits`` (BT, V, contiguous rows) into ``top`` float32 and ``ids`` int32
    (BT, K), and, each or None, the log-sum-exp of the row's logits / temperature and of those outside the K into
    ``lse`` and ``lse_rest`` float32 [BT].  The workspace (uint8 device tensor) is allocated here with torch when not
    given."""
    BT, V, ld = _rows2d(logits, "logits")
    dt, dev, f32 = _dtype_code(logits), logits.device, torch.float32
    K = top.shape[1] if top.dim() == 2 else 0
    _arg(top, "top", f32, (BT, K), dev)
    _arg(ids, "ids", torch.int32, (BT, K), dev)
    for t, name in ((lse, "lse"), (lse_rest, "lse_rest")):
        if t is not None:
            _arg(t, name, f32, (BT,), dev)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_top_logits_workspace_bytes(BT, V, K))
        _check(lib.lx_top_logits(_ptr(logits), ld, BT, V, K, float(temperature), _ptr(top), _ptr(ids), _ptr(lse),
                                 _ptr(lse_rest), dt, ws, wbytes, at.ptr), "lx_top_logits")


def _kd_set(student, target, ids, top, lse_rest, per_row, state, grad=None):
    """(BT, V, K, dtype code, device, student's row stride, grad's) of the arguments that the entry points over
    logits share, checked; ``per_row``: (name, float32 [BT] tensor or None) pairs."""
    BT, V, ld = _rows2d(student, "student")
    dt, dev, f32 = _dtype_code(student), student.device, torch.float32
    K = ids.shape[1] if ids.dim() == 2 else 0
    _arg(target, "target", torch.int64, (BT,), dev)
    _arg(ids, "ids", torch.int32, (BT, K), dev)
    _arg(top, "top", f32, (BT, K), dev)
    if lse_rest is not None:
        _arg(lse_rest, "lse_rest", f32, (BT,), dev)
    for name, t in per_row:
        if t is not None:
            _arg(t, name, f32, (BT,), dev)
    _arg(state, "state", f32, (BT, LX_KD_STATE_FLOATS), dev)
    ldg = V
    if grad is not None:
        if grad.shape != student.shape or grad.dtype != student.dtype or grad.device != dev:
            raise ValueError("grad must match student in shape and dtype and lie on its device")
        ldg = _rows2d(grad, "grad")[2]
    return BT, V, K, dt, dev, ld, ldg


def _scale_ptr(g_scale, dev):
    if g_scale is None:
        return None
    if g_scale.dtype is not torch.float32 or g_scale.numel() != 1 or g_scale.device != dev:
        raise ValueError(f"g_scale must be one float32 on {dev}")
    return g_scale.data_ptr()


def lx_ce_kd_workspace_bytes(BT: int, V: int, dt: int) -> int:
    return lib.lx_ce_kd_workspace_bytes(BT, V, dt)


def lx_ce_kd_forward_backward_workspace_bytes(BT: int, V: int, dt: int) -> int:
    return lib.lx_ce_kd_forward_backward_workspace_bytes(BT, V, dt)


def lx_ce_kd_forward(student, target, ignore_index, ids, top, lse_rest, temperature: float, ce, kd, lse, state,
                     workspace=None, stream=None) -> None:
    """Cross entropy and the divergence from a teacher's top logits: ``student`` (BT, V) with contiguous rows;
    ``ids`` int32 and ``top`` float32 (BT, K), ``lse_rest`` float32 [BT] or None, as lx_top_logits writes them;
    into ``ce``, ``kd``, ``lse`` float32 [BT] and ``state`` float32 [BT, 4].  The workspace (uint8 device
    tensor) is allocated here with torch when not given."""
    BT, V, K, dt, dev, ld, _ = _kd_set(student, target, ids, top, lse_rest, (("ce", ce), ("kd", kd), ("lse", lse)), state)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_ce_kd_workspace_bytes(BT, V, dt))
        _check(lib.lx_ce_kd_forward(_ptr(student), ld, _ptr(target), _ptr(ids), _ptr(top), _ptr(lse_rest), BT, V, K,
                                    int(ignore_index), float(temperature), _ptr(ce), _ptr(kd), _ptr(lse), _ptr(state), dt,
                                    ws, wbytes, at.ptr), "lx_ce_kd_forward")


def lx_ce_kd_backward(grad, student, target, ignore_index, ids, top, temperature: float, lse, state, g_ce: float,
                      g_kd: float, grad_ce_rows=None, grad_kd_rows=None, g_scale=None, stream=None) -> None:
    """The gradient of g_ce ce + g_kd kd into ``grad`` (may be ``student``), from lx_ce_kd_forward's ``lse`` and
    ``state``; ``grad_ce_rows``, ``grad_kd_rows`` float32 [BT] factors or None, ``g_scale`` one float32 or None."""
    BT, V, K, dt, dev, ld, ldg = _kd_set(student, target, ids, top, None, (
        ("lse", lse), ("grad_ce_rows", grad_ce_rows), ("grad_kd_rows", grad_kd_rows)), state, grad)
    with _Launch(dev, stream) as at:
        _check(lib.lx_ce_kd_backward(_ptr(grad), ldg, _ptr(student), ld, _ptr(target), _ptr(ids), _ptr(top), BT, V, K,
                                     int(ignore_index), float(temperature), _ptr(lse), _ptr(state), float(g_ce), float(g_kd),
                                     _ptr(grad_ce_rows), _ptr(grad_kd_rows), _scale_ptr(g_scale, dev), dt, at.ptr),
               "lx_ce_kd_backward")


def lx_ce_kd_forward_backward(student, target, ignore_index, ids, top, lse_rest, temperature: float, ce, kd, lse, state,
                              grad, g_ce: float, g_kd: float, grad_ce_rows=None, grad_kd_rows=None, g_scale=None,
                              workspace=None, stream=None) -> None:
    """lx_ce_kd_forward and lx_ce_kd_backward in one call (``grad`` may be ``student``)."""
    BT, V, K, dt, dev, ld, ldg = _kd_set(student, target, ids, top, lse_rest, (
        ("ce", ce), ("kd", kd), ("lse", lse), ("grad_ce_rows", grad_ce_rows), ("grad_kd_rows", grad_kd_rows)), state, grad)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_ce_kd_forward_backward_workspace_bytes(BT, V, dt))
        _check(lib.lx_ce_kd_forward_backward(_ptr(student), ld, _ptr(target), _ptr(ids), _ptr(top), _ptr(lse_rest), BT, V, K,
                                             int(ignore_index), float(temperature), _ptr(ce), _ptr(kd), _ptr(lse),
                                             _ptr(state), _ptr(grad), ldg, float(g_ce), float(g_kd), _ptr(grad_ce_rows),
                                             _ptr(grad_kd_rows), _scale_ptr(g_scale, dev), dt, ws, wbytes, at.ptr),
               "lx_ce_kd_forward_backward")


def lx_ce_kd_linear_workspace_bytes(BT: int, V: int, H: int, K: int, piece: int, grads: bool) -> int:
    return lib.lx_ce_kd_linear_workspace_bytes(BT, V, H, K, piece, int(bool(grads)))


def lx_ce_kd_linear_piece(BT: int, V: int) -> int:
    """The columns of a piece that lx_ce_kd_linear_forward_backward takes when none are given: at most 2^27 elements
    of the gradient of the logits at once, and at least 2048 columns."""
    return max(1, min(V, max(2048, (1 << 27) // max(1, BT) // 256 * 256), 1 << 22))


def lx_ce_kd_linear_forward_backward(x, w, target, ignore_index, ids, top, lse_rest, temperature: float, ce, kd, lse, state,
                                     grad_x, grad_w, g_ce: float, g_kd: float, grad_ce_rows=None, grad_kd_rows=None,
                                     g_scale=None, piece: int | None = None, workspace=None, stream=None) -> None:
    """The loss of lx_ce_kd_forward (``ids`` None: cross entropy alone, ``top``, ``lse_rest``, ``kd`` and ``state`` None
    too) of the logits x w^T, and their gradients, in pieces of ``piece`` columns of the vocabulary: ``x`` (BT, H) and
    ``w`` (V, H) contiguous bfloat16; ``grad_x`` and ``grad_w`` of the same shapes, both float32 or both bfloat16, or
    None.  The workspace (uint8 device tensor) is allocated here with torch when not given."""
    f32, bf16, dev = torch.float32, torch.bfloat16, x.device
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1] or not x.is_cuda:
        raise ValueError("x must be (BT, H) and w (V, H), device tensors")
    (BT, H), V = x.shape, w.shape[0]
    _arg(x, "x", bf16, (BT, H), dev)
    _arg(w, "w", bf16, (V, H), dev)
    _arg(target, "target", torch.int64, (BT,), dev)
    K = 0
    if ids is not None:
        K = ids.shape[1] if ids.dim() == 2 else 0
        if K < 1:
            raise ValueError("ids must be (BT, K), K at least 1")
        _arg(ids, "ids", torch.int32, (BT, K), dev)
        _arg(top, "top", f32, (BT, K), dev)
        _arg(state, "state", f32, (BT, LX_KD_STATE_FLOATS), dev)
        _arg(kd, "kd", f32, (BT,), dev)
    elif top is not None or lse_rest is not None or kd is not None or state is not None:
        raise ValueError("without ids there are no top, lse_rest, kd and state")
    for name, t in (("lse_rest", lse_rest), ("ce", ce), ("lse", lse), ("grad_ce_rows", grad_ce_rows),
                    ("grad_kd_rows", grad_kd_rows)):
        if t is not None or name in ("ce", "lse"):
            _arg(t, name, f32, (BT,), dev)
    kinds = {t.dtype for t in (grad_x, grad_w) if t is not None}
    if kinds - {f32, bf16} or len(kinds) > 1:
        raise ValueError("grad_x and grad_w must both be float32 or both bfloat16")
    grad_dt = kinds.pop() if kinds else f32
    for name, t, like in (("grad_x", grad_x, x), ("grad_w", grad_w, w)):
        if t is not None:
            _arg(t, name, grad_dt, like.shape, dev)
    piece = lx_ce_kd_linear_piece(BT, V) if piece is None else int(piece)
    with _Launch(dev, stream) as at:
        ws, wbytes, _held = at.workspace(workspace, lib.lx_ce_kd_linear_workspace_bytes(
            BT, V, H, K, piece, int(grad_x is not None or grad_w is not None)))
        _check(lib.lx_ce_kd_linear_forward_backward(
            _ptr(x), _ptr(w), H, _ptr(target), _ptr(ids), _ptr(top), _ptr(lse_rest), BT, V, K, int(ignore_index),
            float(temperature), _ptr(ce), _ptr(kd), _ptr(lse), _ptr(state), _ptr(grad_x), _ptr(grad_w),
            _DTYPE_CODES[grad_dt], float(g_ce), float(g_kd), _ptr(grad_ce_rows), _ptr(grad_kd_rows),
            _scale_ptr(g_scale, dev), piece, ws, wbytes, at.ptr), "lx_ce_kd_linear_forward_backward")


__all__ = [
    "LxError", "lib", "LIB_PATH", "LX_OK", "LX_ERR_INVALID_ARG", "LX_ERR_UNSUPPORTED_DTYPE", "LX_ERR_ALIAS",
    "LX_ERR_WORKSPACE", "LX_ERR_HIP", "LX_F32", "LX_BF16", "LX_F16", "lx_status_string", "lx_abi_version",
    "lx_ce_tvd_workspace_bytes", "lx_ce_tvd_forward", "lx_ce_tvd_backward", "lx_ce_tvd_reduce_mean",
    "lx_ce_tvd_forward_backward_workspace_bytes", "lx_ce_tvd_forward_backward", "lx_ce_tvd_count_valid",
    "lx_vp_stats_floats", "lx_ce_tvd_vp_stats", "lx_ce_tvd_vp_merge_stats", "lx_ce_tvd_vp_tv", "lx_ce_tvd_vp_merge_tv",
    "lx_ce_tvd_backward_shard", "lx_ce_tvd_forward_ex", "lx_ce_tvd_backward_ex", "lx_ce_tvd_forward_backward_ex",
    "lx_gemm_bf16", "lx_ce_tvd_linear_workspace_bytes", "lx_ce_tvd_linear_forward_backward",
    "lx_draft_verify_workspace_bytes", "lx_draft_verify", "lx_lora_forward_workspace_bytes", "lx_lora_forward",
    "lx_lora_backward_workspace_bytes", "lx_lora_backward", "LX_KD_MAX_TOP", "LX_KD_STATE_FLOATS",
    "lx_top_logits_workspace_bytes", "lx_top_logits",
    "lx_ce_kd_workspace_bytes", "lx_ce_kd_forward", "lx_ce_kd_backward", "lx_ce_kd_forward_backward_workspace_bytes",
    "lx_ce_kd_forward_backward", "lx_ce_kd_linear_workspace_bytes", "lx_ce_kd_linear_piece",
    "lx_ce_kd_linear_forward_backward",
]


def lx_stream_read(src, sink, stream=None) -> None:
    """Reference stream: read every byte of src once (sink: int32/uint32 [1])."""
    _check(lib.lx_stream_read(_ptr(src), src.numel() * src.element_size(), _ptr(sink), _stream(stream)),
           "lx_stream_read")


def lx_stream_read2_write(a, b, out, stream=None) -> None:
    """Reference stream: out = a XOR b over their bytes (all the same size)."""
    nb = a.numel() * a.element_size()
    if b.numel() * b.element_size() != nb or out.numel() * out.element_size() != nb:
        raise ValueError("a, b and out must have the same number of bytes")
    _check(lib.lx_stream_read2_write(_ptr(a), _ptr(b), _ptr(out), nb, _stream(stream)), "lx_stream_read2_write")
