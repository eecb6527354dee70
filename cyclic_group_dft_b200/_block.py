"""ctypes binding of the handle-free operators of libeqlin.so (C ABI in include/eqlin.h):
attention over packed sequences, residual addition with root-mean-square norm, and rotary
positions.  Argument marshalling only, as in ``_capi``: torch supplies memory and streams.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _capi
from ._capi import _TORCH_TO_EQLIN, _check, _lib, _stream_ptr

_vp, _i64, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _AttentionShape(ctypes.Structure):
    _fields_ = [("q_rows", _i64), ("k_rows", _i64), ("sequences", _i64), ("heads", _i64), ("kv_heads", _i64),
                ("head_dim", _i64), ("q_offsets", _vp), ("k_offsets", _vp), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("o_stride", _i64), ("io_dtype", _int), ("causal", _int), ("scale", _f32)]


class _GradStrides(ctypes.Structure):
    _fields_ = [("dout", _i64), ("dq", _i64), ("dk", _i64), ("dv", _i64)]


_lib.eqlin_add_rmsnorm.argtypes = [_vp] * 5 + [_i64] * 3 + [_f32, _int, _int, _vp]
_lib.eqlin_add_rmsnorm_fp8.argtypes = [_vp] * 6 + [_i64] * 3 + [_f32, _int, _int, _vp]
_lib.eqlin_rmsnorm_backward_workspace_size.argtypes = [_i64] * 3 + [_int, ctypes.POINTER(_sz)]
_lib.eqlin_rmsnorm_backward.argtypes = [_vp] * 6 + [_i64] * 3 + [_f32, _int, _int, _vp, _sz, _vp]
_lib.eqlin_rope.argtypes = ([_vp] * 3 + [_i64] * 4
                            + [ctypes.POINTER(ctypes.c_int32), _int, ctypes.c_double, _i64, _i64, _int, _int, _vp])
_lib.eqlin_attention_workspace_size.argtypes = [ctypes.POINTER(_AttentionShape), _int, ctypes.POINTER(_sz)]
_lib.eqlin_attention_forward.argtypes = [ctypes.POINTER(_AttentionShape)] + [_vp] * 6 + [_sz, _vp]
_lib.eqlin_attention_backward.argtypes = ([ctypes.POINTER(_AttentionShape), ctypes.POINTER(_GradStrides)]
                                          + [_vp] * 10 + [_sz, _vp])
_lib.eqlin_attention_device_status.argtypes = [ctypes.POINTER(_int)]
for _f in ("eqlin_attention_device_status", "eqlin_add_rmsnorm", "eqlin_add_rmsnorm_fp8", "eqlin_rmsnorm_backward_workspace_size",
           "eqlin_rmsnorm_backward", "eqlin_rope", "eqlin_attention_workspace_size", "eqlin_attention_forward",
           "eqlin_attention_backward"):
    getattr(_lib, _f).restype = _int


_current_stream = torch._C._cuda_getCurrentRawStream   # of a device number; the public call makes a Stream object


def _run(name: str, device: torch.device, stream, *args) -> None:
    """Calls library function `name` with `args` and the stream, with `device` current."""
    f = getattr(_lib, name)
    if torch.cuda.current_device() == device.index:
        status = f(*args, _current_stream(device.index) if stream is None else _stream_ptr(stream))
    else:
        with torch.cuda.device(device):
            status = f(*args, _stream_ptr(stream))
    if status:
        _check(status, name)


def _features(t: torch.Tensor, name: str) -> None:
    if t.dim() != 3:
        raise ValueError(f"{name} must be [N, C, G], got {tuple(t.shape)}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _TORCH_TO_EQLIN:
        raise ValueError(f"unsupported dtype {t.dtype}")


def _like(t: torch.Tensor, name: str, ref: torch.Tensor, dtype: torch.dtype | None = None) -> None:
    want = ref.dtype if dtype is None else dtype
    if t.shape != ref.shape or t.dtype != want or t.device != ref.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(ref.shape)} {want} tensor on {ref.device}")


def _rows(t: torch.Tensor, name: str) -> int:
    """The features between two rows of a [N, C, G] tensor whose rows are contiguous."""
    N, C, G = t.shape
    if (G > 1 and t.stride(2) != 1) or (C > 1 and t.stride(1) != G):
        raise ValueError(f"{name} must have contiguous rows (a [N, C, G] tensor or a channel slice of one)")
    return t.stride(0) if N > 1 else C * G


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _norm_args(x: torch.Tensor, residual, weight, sum_out) -> None:
    _features(x, "x")
    _like(x, "x", x)
    if residual is not None:
        _like(residual, "residual", x)
    _weight(weight, x)
    if sum_out is not None:
        _like(sum_out, "sum_out", x)


def _weight(weight: torch.Tensor | None, x: torch.Tensor) -> None:
    if weight is None:
        return
    if weight.shape != (x.shape[1],) or weight.device != x.device or not weight.is_contiguous() \
            or weight.dtype not in _TORCH_TO_EQLIN:
        raise ValueError(f"weight must be a contiguous [{x.shape[1]}] tensor of a supported dtype on {x.device}")


def _w_code(weight: torch.Tensor | None) -> int:
    return _capi.EQLIN_F32 if weight is None else _TORCH_TO_EQLIN[weight.dtype]


def eqlin_add_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                      eps: float = 1e-6, y: torch.Tensor | None = None, sum_out: torch.Tensor | None = None,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(y, r) with r = x + residual and y = r * weight[c] / sqrt(mean(r^2) + eps) over the
    channels and group elements of a token; x, residual, y and r are [N, C, G], weight [C] or
    None (ones).  Without a residual r is x itself, unless sum_out is given.  y and sum_out may
    be x or residual (in place)."""
    _norm_args(x, residual, weight, sum_out)
    N, C, G = x.shape
    if y is None:
        y = torch.empty_like(x)
    _like(y, "y", x)
    if sum_out is None and residual is not None:
        sum_out = torch.empty_like(x)
    if sum_out is not None and N > 0 and sum_out.data_ptr() == y.data_ptr():
        raise ValueError("y and sum_out must not be the same tensor")
    _run("eqlin_add_rmsnorm", x.device, stream, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(), _ptr(sum_out),
         N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[x.dtype])
    return y, (x if sum_out is None else sum_out)


def eqlin_add_rmsnorm_fp8(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                          eps: float = 1e-6, y: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                          sum_out: torch.Tensor | None = None,
                          stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y8, scale, r): eqlin_add_rmsnorm with y as float8_e4m3fn and one fp32 scale per token,
    y = y8 * scale[:, None, None], scale = max|y| / 448 (1 for a row of zeros)."""
    _norm_args(x, residual, weight, sum_out)
    N, C, G = x.shape
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    _like(y, "y", x, torch.float8_e4m3fn)
    if scale is None:
        scale = torch.empty((N,), dtype=torch.float32, device=x.device)
    elif scale.shape != (N,) or scale.dtype != torch.float32 or scale.device != x.device or not scale.is_contiguous():
        raise ValueError(f"scale must be a contiguous [{N}] fp32 tensor on {x.device}")
    if sum_out is None and residual is not None:
        sum_out = torch.empty_like(x)
    _run("eqlin_add_rmsnorm_fp8", x.device, stream, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(),
         scale.data_ptr(), _ptr(sum_out), N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[x.dtype])
    return y, scale, (x if sum_out is None else sum_out)


def eqlin_rmsnorm_backward_workspace_size(N: int, C: int, G: int, io_dtype=torch.bfloat16) -> int:
    v = _sz()
    _check(_lib.eqlin_rmsnorm_backward_workspace_size(N, C, G, _capi._as_code(io_dtype), ctypes.byref(v)),
           "eqlin_rmsnorm_backward_workspace_size")
    return int(v.value)


def eqlin_rmsnorm_backward(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor | None = None,
                           dsum: torch.Tensor | None = None, eps: float = 1e-6, with_weight: bool = True,
                           dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None,
                           stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(dx [N, C, G], dweight [C] fp32 or None) from dy and the stored sum r of
    eqlin_add_rmsnorm; dx is the gradient of x and of the residual alike and includes dsum, the
    gradient that reaches r through the residual stream.  The workspace (a uint8 CUDA tensor) is
    allocated by torch when not given."""
    _features(r, "r")
    _like(r, "r", r)
    _like(dy, "dy", r)
    _weight(weight, r)
    if dsum is not None:
        _like(dsum, "dsum", r)
    N, C, G = r.shape
    if dx is None:
        dx = torch.empty_like(r)
    _like(dx, "dx", r)
    if with_weight and dweight is None:
        dweight = torch.empty((C,), dtype=torch.float32, device=r.device)
    if dweight is not None:
        if dweight.shape != (C,) or dweight.dtype != torch.float32 or dweight.device != r.device \
                or not dweight.is_contiguous():
            raise ValueError(f"dweight must be a contiguous [{C}] fp32 tensor on {r.device}")
        if workspace is None:
            need = eqlin_rmsnorm_backward_workspace_size(N, C, G, r.dtype)
            workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=r.device)
    _workspace(workspace, r)
    _run("eqlin_rmsnorm_backward", r.device, stream, dy.data_ptr(), r.data_ptr(), _ptr(weight), _ptr(dsum), dx.data_ptr(),
         _ptr(dweight), N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[r.dtype], _ptr(workspace),
         0 if workspace is None else workspace.numel())
    return dx, dweight


def _workspace(workspace: torch.Tensor | None, ref: torch.Tensor) -> None:
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.device != ref.device
                                  or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {ref.device}")


def eqlin_rope(x: torch.Tensor, positions: torch.Tensor, heads: int, sections, base: float = 10000.0,
               inverse: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions with several axes on x [N, heads * Dh, G] (a channel slice of a wider
    tensor will do): channel pair (c, c + Dh/2) of each head turns by positions[n, axis] *
    base^(-j / sections[axis]).  positions is [N, axes] int32; the sections add up to Dh/2.
    inverse turns back, which is also the gradient.  out may be x (in place)."""
    _features(x, "x")
    N, C, G = x.shape
    sections = [int(n) for n in sections]
    if heads < 1 or C % heads:
        raise ValueError(f"{C} channels are not {heads} heads")
    if positions.shape != (N, len(sections)) or positions.dtype != torch.int32 or positions.device != x.device \
            or not positions.is_contiguous():
        raise ValueError(f"positions must be a contiguous [{N}, {len(sections)}] int32 tensor on {x.device}")
    if any(n < 0 or n > C for n in sections):
        raise ValueError("the sections must be counts that add up to half the channels of a head")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out has the wrong shape, dtype or device")
    xs, ys = _rows(x, "x"), _rows(out, "out")
    table = (ctypes.c_int32 * max(len(sections), 1))(*sections)
    _run("eqlin_rope", x.device, stream, x.data_ptr(), positions.data_ptr(), out.data_ptr(), N, heads, C // heads, G, table,
         len(sections), base, xs, ys, int(bool(inverse)), _TORCH_TO_EQLIN[x.dtype])
    return out


def _attention_shape(q, k, v, o, heads, kv_heads, q_offsets, k_offsets, causal, scale) -> _AttentionShape:
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _features(t, name)
        if t.dtype != q.dtype or t.device != q.device or t.shape[2] != q.shape[2]:
            raise ValueError("q, k, v and o must share a dtype, a device and G")
    kv_heads = heads if kv_heads is None else kv_heads
    if heads < 1 or kv_heads < 1 or q.shape[1] % heads:
        raise ValueError(f"{q.shape[1]} channels are not {heads} heads")
    Dh = q.shape[1] // heads
    if k.shape[1] != kv_heads * Dh or v.shape != k.shape:
        raise ValueError(f"k and v must be [Nk, {kv_heads * Dh}, G] (kv_heads heads of {Dh} channels)")
    if o.shape != q.shape:
        raise ValueError("o must have q's shape")
    if (q_offsets is None) != (k_offsets is None):
        raise ValueError("q_offsets and k_offsets go together")
    n = 1
    if q_offsets is not None:
        for t, name in ((q_offsets, "q_offsets"), (k_offsets, "k_offsets")):
            if t.dim() != 1 or t.dtype != torch.int32 or t.device != q.device or not t.is_contiguous() \
                    or t.numel() < 2 or t.numel() != q_offsets.numel():
                raise ValueError(f"{name} must be a contiguous [sequences + 1] int32 tensor on {q.device}")
        n = q_offsets.numel() - 1
    D = Dh * q.shape[2]
    return _AttentionShape(q.shape[0], k.shape[0], n, heads, kv_heads, D, _ptr(q_offsets), _ptr(k_offsets),
                           _rows(q, "q"), _rows(k, "k"), _rows(v, "v"), _rows(o, "o"), _TORCH_TO_EQLIN[q.dtype],
                           int(bool(causal)), 1.0 / math.sqrt(D) if scale is None else scale)


def _attention_workspace(shape: _AttentionShape, backward: int, workspace, ref: torch.Tensor):
    v = _sz()
    _check(_lib.eqlin_attention_workspace_size(ctypes.byref(shape), backward, ctypes.byref(v)),
           "eqlin_attention_workspace_size")
    if workspace is None and v.value:
        workspace = torch.empty((v.value,), dtype=torch.uint8, device=ref.device)
    _workspace(workspace, ref)
    return workspace


def eqlin_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, heads: int,
                            kv_heads: int | None = None, q_offsets: torch.Tensor | None = None,
                            k_offsets: torch.Tensor | None = None, causal: bool = False, scale: float | None = None,
                            o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None,
                            stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(o [Nq, heads * Dh, G], lse [heads, Nq] fp32) of attention over packed sequences.

    q is [Nq, heads * Dh, G], k and v are [Nk, kv_heads * Dh, G] (channel slices of a joint
    projection will do); a head's Dh * G features are a multiple of 8 up to 128.  q_offsets and
    k_offsets are [sequences + 1] int32 on the device: sequence b has the rows offsets[b] ..
    offsets[b + 1]; None means one sequence.  causal: the last query of a sequence sees its last
    key.  scale defaults to 1 / sqrt(Dh * G)."""
    _features(q, "q")
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    shape = _attention_shape(q, k, v, o, heads, kv_heads, q_offsets, k_offsets, causal, scale)
    if lse is None:
        lse = torch.empty((heads, q.shape[0]), dtype=torch.float32, device=q.device)
    elif lse.shape != (heads, q.shape[0]) or lse.dtype != torch.float32 or lse.device != q.device \
            or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous [{heads}, {q.shape[0]}] fp32 tensor on {q.device}")
    workspace = _attention_workspace(shape, 0, workspace, q)
    _run("eqlin_attention_forward", q.device, stream, ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         o.data_ptr(), lse.data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel())
    return o, lse


def eqlin_attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                             lse: torch.Tensor, heads: int, kv_heads: int | None = None,
                             q_offsets: torch.Tensor | None = None, k_offsets: torch.Tensor | None = None,
                             causal: bool = False, scale: float | None = None,
                             grads: tuple[torch.Tensor, torch.Tensor, torch.Tensor] | None = None,
                             workspace: torch.Tensor | None = None,
                             stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) from do = dL/do and the forward's inputs, o and lse.  grads gives the three
    outputs (channel slices of one joint gradient will do); they are allocated when not given."""
    _features(q, "q")
    shape = _attention_shape(q, k, v, o, heads, kv_heads, q_offsets, k_offsets, causal, scale)
    if grads is None:
        grads = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    dq, dk, dv = grads
    for t, ref, name in ((do, q, "do"), (dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError(f"{name} must be a {tuple(ref.shape)} {ref.dtype} tensor on {ref.device}")
    if lse.shape != (heads, q.shape[0]) or lse.dtype != torch.float32 or lse.device != q.device \
            or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous [{heads}, {q.shape[0]}] fp32 tensor on {q.device}")
    strides = _GradStrides(_rows(do, "do"), _rows(dq, "dq"), _rows(dk, "dk"), _rows(dv, "dv"))
    workspace = _attention_workspace(shape, 1, workspace, q)
    _run("eqlin_attention_backward", q.device, stream, ctypes.byref(shape), ctypes.byref(strides), do.data_ptr(),
         q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
         dv.data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel())
    return dq, dk, dv


def eqlin_attention_device_status(device=None) -> int:
    """Synchronises the device (default: the current one), then reads and clears its word for errors of
    the attention kernels: EQLIN_OK, or EQLIN_ERR_TIMEOUT when a wait inside one ran out."""
    v = _int()
    with torch.cuda.device(torch.cuda.current_device() if device is None else device):
        _check(_lib.eqlin_attention_device_status(ctypes.byref(v)), "eqlin_attention_device_status")
    return int(v.value)
