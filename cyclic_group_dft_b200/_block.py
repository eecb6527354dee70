"""ctypes binding of the handle-free operators of libeqlin.so (C ABI in include/eqlin.h):
attention over packed sequences, residual addition with root-mean-square norm, and rotary
positions.  Argument marshalling only, as in ``_capi``: torch supplies memory and streams.
Every function of tensors takes the keyword ``stream`` as well (see ``_in_stream``).
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi
from ._capi import _TORCH_TO_EQLIN, _check, _lib

_vp, _i64, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


class _AttentionShape(ctypes.Structure):
    _fields_ = [("q_rows", _i64), ("k_rows", _i64), ("sequences", _i64), ("heads", _i64), ("kv_heads", _i64),
                ("head_dim", _i64), ("q_offsets", _vp), ("k_offsets", _vp), ("q_stride", _i64), ("k_stride", _i64),
                ("v_stride", _i64), ("o_stride", _i64), ("io_dtype", _int), ("causal", _int), ("scale", _f32)]


_Sections = ctypes.c_int32 * 4   # pairs of each rotary axis


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


# the current device, and a device's current stream, as numbers (the tensors show that CUDA is set up)
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _run(name: str, device: int, *args) -> None:
    """Calls library function `name` with `args` and the current stream, with device number `device` current."""
    f = getattr(_lib, name)
    if _current_device() == device:
        status = f(*args, _current_stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _current_stream(device))
    if status:
        _check(status, name)


def _in_stream(f):
    """Gives a function its keyword `stream` (a torch Stream of the tensors' device or a cudaStream_t as a number;
    default: the current stream): the whole call, its allocations among it, is made with that stream current.
    What it allocates then belongs to that stream, and a workspace that is given up on return is not reused
    before the kernels are done with it."""

    @functools.wraps(f)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return f(*args, **kwargs)
        device = next((t.device for t in (*args, *kwargs.values()) if isinstance(t, torch.Tensor)), None)
        if device is None or device.type != "cuda":
            return f(*args, **kwargs)               # which says what is wrong with the tensors
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else \
                torch.cuda.default_stream(device)
        elif stream.device != device:
            raise ValueError(f"stream must be a stream of {device}, got one of {stream.device}")
        with torch.cuda.stream(stream):
            return f(*args, **kwargs)

    return call


# These checks run on every call, whose kernels may take a few microseconds: each asks a tensor for as little as
# it can (shape and strides once, the device as a number).

def _features(t: torch.Tensor, name: str) -> torch.Size:
    """The shape of a [N, C, G] CUDA tensor of a supported dtype."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [N, C, G], got {tuple(shape)}")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _TORCH_TO_EQLIN:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return shape


def _like(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device: int) -> None:
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on cuda:{device}")


def _rows(t: torch.Tensor, name: str, shape, dtype: torch.dtype, device: int) -> int:
    """The features between two rows of a [N, C, G] tensor whose rows are contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on cuda:{device}")
    N, C, G = shape
    row, channel, element = t.stride()
    if (G > 1 and element != 1) or (C > 1 and channel != G):
        raise ValueError(f"{name} must have contiguous rows (a [N, C, G] tensor or a channel slice of one)")
    return row if N > 1 else C * G


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _norm_args(x: torch.Tensor, residual, weight, sum_out):
    shape, dtype, device = _features(x, "x"), x.dtype, x.get_device()
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if residual is not None:
        _like(residual, "residual", shape, dtype, device)
    if weight is not None:
        _weight(weight, shape[1], device)
    if sum_out is not None:
        _like(sum_out, "sum_out", shape, dtype, device)
    return shape, dtype, device


def _weight(weight: torch.Tensor, C: int, device: int) -> None:
    if weight.shape != (C,) or weight.get_device() != device or weight.dtype not in _TORCH_TO_EQLIN \
            or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{C}] tensor of a supported dtype on cuda:{device}")


def _w_code(weight: torch.Tensor | None) -> int:
    return _capi.EQLIN_F32 if weight is None else _TORCH_TO_EQLIN[weight.dtype]


@_in_stream
def eqlin_add_rmsnorm(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                      eps: float = 1e-6, y: torch.Tensor | None = None, sum_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(y, r) with r = x + residual and y = r * weight[c] / sqrt(mean(r^2) + eps) over the
    channels and group elements of a token; x, residual, y and r are [N, C, G], weight [C] or
    None (ones).  Without a residual r is x itself, unless sum_out is given or y is written over x: then r
    has memory of its own.  y and sum_out may be x or residual (in place)."""
    shape, dtype, device = _norm_args(x, residual, weight, sum_out)
    N, C, G = shape
    if y is None:
        y = torch.empty_like(x)
    else:
        _like(y, "y", shape, dtype, device)
    if sum_out is None and (residual is not None or y.data_ptr() == x.data_ptr()):
        sum_out = torch.empty_like(x)
    if sum_out is not None and N > 0 and sum_out.data_ptr() == y.data_ptr():
        raise ValueError("y and sum_out must not be the same tensor")
    _run("eqlin_add_rmsnorm", device, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(), _ptr(sum_out),
         N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[dtype])
    return y, (x if sum_out is None else sum_out)


@_in_stream
def eqlin_add_rmsnorm_fp8(x: torch.Tensor, residual: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                          eps: float = 1e-6, y: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                          sum_out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(y8, scale, r): eqlin_add_rmsnorm with y as float8_e4m3fn and one fp32 scale per token,
    y = y8 * scale[:, None, None], scale = max|y| / 448 (1 for a row of zeros)."""
    shape, dtype, device = _norm_args(x, residual, weight, sum_out)
    N, C, G = shape
    if y is None:
        y = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _like(y, "y", shape, torch.float8_e4m3fn, device)
    if scale is None:
        scale = torch.empty((N,), dtype=torch.float32, device=x.device)
    else:
        _like(scale, "scale", (N,), torch.float32, device)
    if sum_out is None and residual is not None:
        sum_out = torch.empty_like(x)
    _run("eqlin_add_rmsnorm_fp8", device, x.data_ptr(), _ptr(residual), _ptr(weight), y.data_ptr(),
         scale.data_ptr(), _ptr(sum_out), N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[dtype])
    return y, scale, (x if sum_out is None else sum_out)


def eqlin_rmsnorm_backward_workspace_size(N: int, C: int, G: int, io_dtype=torch.bfloat16) -> int:
    v = _sz()
    _check(_lib.eqlin_rmsnorm_backward_workspace_size(N, C, G, _capi._as_code(io_dtype), ctypes.byref(v)),
           "eqlin_rmsnorm_backward_workspace_size")
    return int(v.value)


@_in_stream
def eqlin_rmsnorm_backward(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor | None = None,
                           dsum: torch.Tensor | None = None, eps: float = 1e-6, with_weight: bool = True,
                           dx: torch.Tensor | None = None, dweight: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(dx [N, C, G], dweight [C] fp32 or None) from dy and the stored sum r of
    eqlin_add_rmsnorm; dx is the gradient of x and of the residual alike and includes dsum, the
    gradient that reaches r through the residual stream.  The workspace (a uint8 CUDA tensor) is
    allocated by torch when not given."""
    shape, dtype, device = _features(r, "r"), r.dtype, r.get_device()
    if not r.is_contiguous():
        raise ValueError("r must be contiguous")
    _like(dy, "dy", shape, dtype, device)
    N, C, G = shape
    if weight is not None:
        _weight(weight, C, device)
    if dsum is not None:
        _like(dsum, "dsum", shape, dtype, device)
    if dx is None:
        dx = torch.empty_like(r)
    else:
        _like(dx, "dx", shape, dtype, device)
    if dweight is not None:
        _like(dweight, "dweight", (C,), torch.float32, device)
    elif with_weight:
        dweight = torch.empty((C,), dtype=torch.float32, device=r.device)
    if dweight is not None and workspace is None:
        need = eqlin_rmsnorm_backward_workspace_size(N, C, G, dtype)
        workspace = torch.empty((max(need, 16),), dtype=torch.uint8, device=r.device)
    _run("eqlin_rmsnorm_backward", device, dy.data_ptr(), r.data_ptr(), _ptr(weight), _ptr(dsum), dx.data_ptr(),
         _ptr(dweight), N, C, G, eps, _w_code(weight), _TORCH_TO_EQLIN[dtype], _ptr(workspace), _workspace(workspace, device))
    return dx, dweight


def _workspace(workspace: torch.Tensor | None, device: int) -> int:
    """Bytes of a workspace (a contiguous uint8 tensor on the device)."""
    if workspace is None:
        return 0
    if workspace.dtype is not torch.uint8 or workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{device}")
    return workspace.numel()


@_in_stream
def eqlin_rope(x: torch.Tensor, positions: torch.Tensor, heads: int, sections, base: float = 10000.0,
               inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotary positions with several axes on x [N, heads * Dh, G] (a channel slice of a wider
    tensor will do): channel pair (c, c + Dh/2) of each head turns by positions[n, axis] *
    base^(-j / sections[axis]).  positions is [N, axes] int32; the sections add up to Dh/2.
    inverse turns back, which is also the gradient.  out may be x (in place)."""
    shape, dtype, device = _features(x, "x"), x.dtype, x.get_device()
    N, C, G = shape
    axes = len(sections)
    if heads < 1 or C % heads:
        raise ValueError(f"{C} channels are not {heads} heads")
    if not 1 <= axes <= 4 or min(sections) < 0 or 2 * heads * sum(sections) != C:
        raise ValueError("the sections must be 1 to 4 counts that add up to half the channels of a head")
    _like(positions, "positions", (N, axes), torch.int32, device)
    xs = _rows(x, "x", shape, dtype, device)
    if out is None:
        out, ys = torch.empty(shape, dtype=dtype, device=x.device), C * G
    else:
        ys = _rows(out, "out", shape, dtype, device)
    _run("eqlin_rope", device, x.data_ptr(), positions.data_ptr(), out.data_ptr(), N, heads, C // heads, G,
         _Sections(*sections), axes, base, xs, ys, int(bool(inverse)), _TORCH_TO_EQLIN[dtype])
    return out


def _attention_shape(q, k, v, heads, kv_heads, q_offsets, k_offsets, causal, scale):
    """(the C struct but for o's stride, q's shape, k's shape, dtype, device number)"""
    q_shape, dtype, device = _features(q, "q"), q.dtype, q.get_device()
    Nq, C, G = q_shape
    kv_heads = heads if kv_heads is None else kv_heads
    if heads < 1 or kv_heads < 1 or C % heads:
        raise ValueError(f"{C} channels are not {heads} heads")
    Dh = C // heads
    k_shape = k.shape
    if len(k_shape) != 3 or k_shape[1] != kv_heads * Dh or k_shape[2] != G:
        raise ValueError(f"k and v must be [Nk, {kv_heads * Dh}, {G}] ({kv_heads} heads of {Dh} channels)")
    n = 1
    if q_offsets is not None and k_offsets is not None:
        n = len(q_offsets) - 1
        for t, name in ((q_offsets, "q_offsets"),) if k_offsets is q_offsets else ((q_offsets, "q_offsets"),
                                                                                  (k_offsets, "k_offsets")):
            if n < 1 or t.shape != (n + 1,) or t.dtype is not torch.int32 or t.get_device() != device \
                    or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [sequences + 1] int32 tensor on cuda:{device}")
    elif q_offsets is not None or k_offsets is not None:
        raise ValueError("q_offsets and k_offsets go together")
    D = Dh * G
    s = _AttentionShape(Nq, k_shape[0], n, heads, kv_heads, D, _ptr(q_offsets), _ptr(k_offsets),
                        _rows(q, "q", q_shape, dtype, device), _rows(k, "k", k_shape, dtype, device),
                        _rows(v, "v", k_shape, dtype, device), C * G, _TORCH_TO_EQLIN[dtype], 1 if causal else 0,
                        D ** -0.5 if scale is None else scale)
    return s, q_shape, k_shape, dtype, device


def _attention_workspace(shape: _AttentionShape, backward: int, workspace, ref: torch.Tensor):
    v = _sz()
    status = _lib.eqlin_attention_workspace_size(ctypes.byref(shape), backward, ctypes.byref(v))
    if status:
        _check(status, "eqlin_attention_workspace_size")
    if workspace is None and v.value:
        workspace = torch.empty((v.value,), dtype=torch.uint8, device=ref.device)
    return workspace


@_in_stream
def eqlin_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, heads: int,
                            kv_heads: int | None = None, q_offsets: torch.Tensor | None = None,
                            k_offsets: torch.Tensor | None = None, causal: bool = False, scale: float | None = None,
                            o: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(o [Nq, heads * Dh, G], lse [heads, Nq] fp32) of attention over packed sequences.

    q is [Nq, heads * Dh, G], k and v are [Nk, kv_heads * Dh, G] (channel slices of a joint
    projection will do); a head's Dh * G features are a multiple of 8 up to 128.  q_offsets and
    k_offsets are [sequences + 1] int32 on the device: sequence b has the rows offsets[b] ..
    offsets[b + 1]; None means one sequence.  causal: the last query of a sequence sees its last
    key.  scale defaults to 1 / sqrt(Dh * G)."""
    shape, q_shape, _, dtype, device = _attention_shape(q, k, v, heads, kv_heads, q_offsets, k_offsets, causal, scale)
    if o is None:
        o = torch.empty(q_shape, dtype=dtype, device=q.device)
    else:
        shape.o_stride = _rows(o, "o", q_shape, dtype, device)
    if lse is None:
        lse = torch.empty((heads, q_shape[0]), dtype=torch.float32, device=q.device)
    else:
        _like(lse, "lse", (heads, q_shape[0]), torch.float32, device)
    workspace = _attention_workspace(shape, 0, workspace, q)
    _run("eqlin_attention_forward", device, ctypes.byref(shape), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         o.data_ptr(), lse.data_ptr(), _ptr(workspace), _workspace(workspace, device))
    return o, lse


@_in_stream
def eqlin_attention_backward(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                             lse: torch.Tensor, heads: int, kv_heads: int | None = None,
                             q_offsets: torch.Tensor | None = None, k_offsets: torch.Tensor | None = None,
                             causal: bool = False, scale: float | None = None,
                             grads: tuple[torch.Tensor, torch.Tensor, torch.Tensor] | None = None,
                             workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) from do = dL/do and the forward's inputs, o and lse.  grads gives the three
    outputs (channel slices of one joint gradient will do); they are allocated when not given."""
    shape, q_shape, k_shape, dtype, device = _attention_shape(q, k, v, heads, kv_heads, q_offsets, k_offsets, causal,
                                                              scale)
    shape.o_stride = _rows(o, "o", q_shape, dtype, device)
    _like(lse, "lse", (heads, q_shape[0]), torch.float32, device)
    if grads is None:
        dq, dk, dv = (torch.empty(t, dtype=dtype, device=q.device) for t in (q_shape, k_shape, k_shape))
    else:
        dq, dk, dv = grads
    strides = _GradStrides(_rows(do, "do", q_shape, dtype, device), _rows(dq, "dq", q_shape, dtype, device),
                           _rows(dk, "dk", k_shape, dtype, device), _rows(dv, "dv", k_shape, dtype, device))
    workspace = _attention_workspace(shape, 1, workspace, q)
    _run("eqlin_attention_backward", device, ctypes.byref(shape), ctypes.byref(strides), do.data_ptr(),
         q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
         dv.data_ptr(), _ptr(workspace), _workspace(workspace, device))
    return dq, dk, dv


def eqlin_attention_device_status(device=None) -> int:
    """Synchronises the device (default: the current one), then reads and clears its word for errors of
    the attention kernels: EQLIN_OK, or EQLIN_ERR_TIMEOUT when a wait inside one ran out."""
    v = _int()
    with torch.cuda.device(torch.cuda.current_device() if device is None else device):
        _check(_lib.eqlin_attention_device_status(ctypes.byref(v)), "eqlin_attention_device_status")
    return int(v.value)
