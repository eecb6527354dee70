"""Refusals of the transformer-block operators, checked on the host (no GPU needed): the C entry
points validate sizes, dtypes, pointers, alignment and workspaces before any CUDA work."""
from __future__ import annotations

import contextlib
import ctypes
import glob
import os

import pytest
import torch

import cyclic_group_dft_b200 as eq
from cyclic_group_dft_b200 import _block, build

LIB = eq.library()
BF, F16, F32 = eq.EQLIN_BF16, eq.EQLIN_F16, eq.EQLIN_F32
OK, BAD, UNSUP, MISAL = eq.EQLIN_OK, eq.EQLIN_ERR_INVALID_ARG, eq.EQLIN_ERR_UNSUPPORTED, eq.EQLIN_ERR_MISALIGNED


def test_header_declares_the_binding_s_functions():
    declared = eq.header_functions()
    for name in ("eqlin_add_rmsnorm", "eqlin_add_rmsnorm_fp8", "eqlin_rmsnorm_backward",
                 "eqlin_rmsnorm_backward_workspace_size", "eqlin_rope", "eqlin_attention_workspace_size",
                 "eqlin_attention_forward", "eqlin_attention_backward"):
        assert name in declared
    assert "eqlin_attention_forward" in dir(eq)


# -------------------------------------------------------------------------------- norm
@pytest.mark.parametrize("change,status", [
    (dict(N=-1), BAD), (dict(C=0), BAD), (dict(io=9), BAD), (dict(wd=7), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(x=None), BAD), (dict(y=None), BAD),
    (dict(G=3), UNSUP), (dict(G=32), UNSUP), (dict(C=3, G=2), UNSUP), (dict(C=8192, G=4), UNSUP),
    (dict(C=4096, G=4, io=F32), UNSUP), (dict(C=4099, G=1, io=F32), UNSUP), (dict(N=1 << 31), UNSUP),
    (dict(x=24), MISAL), (dict(residual=8), MISAL), (dict(y=40), MISAL), (dict(sum_out=4), MISAL),
    (dict(N=0, x=None, y=None), OK),
])
def test_norm_refusals(change, status):
    a = dict(x=256, residual=256, w=256, y=512, sum_out=1024, N=4, C=96, G=4, eps=1e-6, wd=BF, io=BF)
    a.update(change)
    args = (a["x"], a["residual"], a["w"], a["y"])
    sizes = (a["N"], a["C"], a["G"], a["eps"], a["wd"], a["io"], None)
    assert LIB.eqlin_add_rmsnorm(*args, a["sum_out"], *sizes) == status
    assert LIB.eqlin_add_rmsnorm_fp8(*args, 2048, a["sum_out"], *sizes) == status
    if status != OK:
        assert eq.eqlin_last_error()
    assert LIB.eqlin_rmsnorm_backward(a["x"], a["y"], a["w"], a["residual"], 512 if a["sum_out"] == 1024 else 4, None,
                                      *sizes[:-1], None, 0, None) == status


def test_norm_fp8_needs_scales():
    assert LIB.eqlin_add_rmsnorm_fp8(256, None, None, 512, None, None, 4, 96, 4, 1e-6, BF, BF, None) == BAD
    assert LIB.eqlin_add_rmsnorm_fp8(256, None, None, 512, 1026, None, 4, 96, 4, 1e-6, BF, BF, None) == MISAL


def test_norm_refuses_outputs_over_one_another():
    sizes = (4, 96, 4, 1e-6, BF, BF, None)
    assert LIB.eqlin_add_rmsnorm(256, 512, None, 1024, 1024, *sizes) == BAD
    assert LIB.eqlin_add_rmsnorm_fp8(256, 512, None, 1024, 2048, 1024, *sizes) == BAD
    for y in (256, 512):
        assert LIB.eqlin_add_rmsnorm_fp8(256, 512, None, y, 2048, None, *sizes) == BAD


def test_norm_backward_workspace():
    n = eq.eqlin_rmsnorm_backward_workspace_size(1000, 96, 4)
    assert n > 0 and n % (96 * 4) == 0
    assert eq.eqlin_rmsnorm_backward_workspace_size(0, 96, 4) == 0
    args = (256, 512, None, None, 1024, 2048, 1000, 96, 4, 1e-6, BF, BF)
    assert LIB.eqlin_rmsnorm_backward(*args, None, 0, None) == BAD
    assert LIB.eqlin_rmsnorm_backward(*args, 4096, n - 1, None) == BAD
    assert LIB.eqlin_rmsnorm_backward(*args, 4100, n, None) == MISAL
    assert LIB.eqlin_rmsnorm_backward_workspace_size(4, 96, 4, BF, None) == BAD
    assert LIB.eqlin_rmsnorm_backward(256, 512, None, None, 1024, 2050, 4, 96, 4, 1e-6, BF, BF, 4096, n, None) == MISAL


# -------------------------------------------------------------------------------- rope
def _rope(x=256, pos=256, y=512, N=4, heads=2, channels=8, G=4, sections=(2, 2), axes=None, base=100.0, xs=64, ys=64,
          inverse=0, io=BF):
    t = None if sections is None else (ctypes.c_int32 * max(len(sections), 1))(*sections)
    return LIB.eqlin_rope(x, pos, y, N, heads, channels, G, t, len(sections or ()) if axes is None else axes, base, xs,
                          ys, inverse, io, None)


@pytest.mark.parametrize("change,status", [
    (dict(N=-1), BAD), (dict(heads=0), BAD), (dict(channels=0), BAD), (dict(io=5), BAD), (dict(sections=None), BAD),
    (dict(axes=0), BAD), (dict(sections=(1, 1, 1, 1, 0)), BAD), (dict(sections=(2, 1)), BAD),
    (dict(sections=(5, -1)), BAD), (dict(base=0.5), BAD), (dict(base=float("nan")), BAD), (dict(xs=63), BAD),
    (dict(ys=32), BAD), (dict(xs=1 << 50), BAD), (dict(x=None), BAD), (dict(pos=None), BAD), (dict(y=None), BAD),
    (dict(G=3), UNSUP), (dict(channels=7), UNSUP), (dict(channels=258, sections=(129,), xs=4096, ys=4096), UNSUP),
    (dict(N=1 << 31), UNSUP), (dict(x=257), MISAL), (dict(y=513), MISAL), (dict(pos=258), MISAL),
    (dict(N=0, x=None, y=None, pos=None), OK),
])
def test_rope_refusals(change, status):
    assert _rope(**change) == status


# --------------------------------------------------------------------------- attention
def _shape(**change):
    a = dict(q_rows=10, k_rows=12, sequences=1, heads=6, kv_heads=2, head_dim=64, q_offsets=None, k_offsets=None,
             q_stride=384, k_stride=128, v_stride=128, o_stride=384, io_dtype=BF, causal=0, scale=0.125)
    a.update(change)
    return _block._AttentionShape(**a)


SHAPE_REFUSALS = [
    (dict(q_rows=-1), BAD), (dict(k_rows=-1), BAD), (dict(sequences=0), BAD), (dict(heads=0), BAD),
    (dict(kv_heads=0), BAD), (dict(kv_heads=4), BAD), (dict(head_dim=0), BAD), (dict(io_dtype=4), BAD),
    (dict(scale=0.0), BAD), (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(causal=2), BAD),
    (dict(sequences=2), BAD), (dict(q_offsets=256), BAD), (dict(k_offsets=256), BAD),
    (dict(head_dim=63), UNSUP), (dict(head_dim=136), UNSUP), (dict(q_rows=1 << 31), UNSUP),
    (dict(heads=1 << 16, kv_heads=1), UNSUP), (dict(sequences=1 << 24, q_offsets=256, k_offsets=256), UNSUP),
    (dict(q_offsets=258, k_offsets=256), MISAL),
]
TENSOR_REFUSALS = [
    (dict(q_stride=383), BAD), (dict(o_stride=376), BAD), (dict(k_stride=1 << 41), BAD), (dict(v_stride=0), BAD),
    (dict(q_stride=388), MISAL), (dict(v_stride=130), MISAL),
]


@pytest.mark.parametrize("change,status", SHAPE_REFUSALS + TENSOR_REFUSALS)
def test_attention_refusals(change, status):
    s = _shape(**change)
    n = ctypes.c_size_t()
    if (change, status) in SHAPE_REFUSALS:
        assert LIB.eqlin_attention_workspace_size(ctypes.byref(s), 1, ctypes.byref(n)) == status
    big = 1 << 40
    assert LIB.eqlin_attention_forward(ctypes.byref(s), 256, 256, 256, 512, None, 1024, big, None) == status
    g = _block._GradStrides(384, 384, 128, 128)
    assert LIB.eqlin_attention_backward(ctypes.byref(s), ctypes.byref(g), 256, 256, 256, 256, 512, 256, 512, 512, 512,
                                        1024, big, None) == status
    assert eq.eqlin_last_error()


@pytest.mark.parametrize("side", ["q_rows", "k_rows"])
def test_attention_row_limit_leaves_room_for_the_last_tile(side):
    """Kernels count rows in 32 bits, up to the end of a tile that begins before the last row."""
    n = ctypes.c_size_t()
    for rows, status in (((1 << 31) - 1, UNSUP), ((1 << 31) - 1024, UNSUP), ((1 << 31) - 1025, OK)):
        s = _shape(heads=1, kv_heads=1, head_dim=8, q_stride=8, k_stride=8, v_stride=8, o_stride=8, **{side: rows})
        for backward in (0, 1):
            assert LIB.eqlin_attention_workspace_size(ctypes.byref(s), backward, ctypes.byref(n)) == status


def test_attention_pointer_refusals():
    s, big = _shape(), 1 << 30
    ref = ctypes.byref(s)
    assert LIB.eqlin_attention_forward(None, 256, 256, 256, 512, None, None, 0, None) == BAD
    for k in range(4):
        ptrs = [256, 256, 256, 512]
        ptrs[k] = None
        assert LIB.eqlin_attention_forward(ref, *ptrs, None, 1024, big, None) == BAD
        ptrs[k] = 264
        assert LIB.eqlin_attention_forward(ref, *ptrs, None, 1024, big, None) == MISAL
    assert LIB.eqlin_attention_forward(ref, 256, 256, 256, 512, 514, 1024, big, None) == MISAL
    empty = _shape(q_rows=0)
    assert LIB.eqlin_attention_forward(ctypes.byref(empty), None, 256, 256, None, None, None, 0, None) == OK
    g = _block._GradStrides(384, 384, 128, 128)
    good = [256] * 5 + [512] + [1024] * 3
    for k in range(9):
        ptrs = list(good)
        ptrs[k] = None
        assert LIB.eqlin_attention_backward(ref, ctypes.byref(g), *ptrs, 4096, big, None) == BAD, k
    n = ctypes.c_size_t()
    assert LIB.eqlin_attention_workspace_size(ref, 1, ctypes.byref(n)) == OK and n.value >= 10 * 6 * 4
    assert LIB.eqlin_attention_backward(ref, ctypes.byref(g), *good, None, 0, None) == BAD
    assert LIB.eqlin_attention_backward(ref, ctypes.byref(g), *good, 4096, n.value - 1, None) == BAD
    assert LIB.eqlin_attention_backward(ref, ctypes.byref(g), *good, 4100, n.value, None) == MISAL
    assert LIB.eqlin_attention_backward(ref, None, *good, 4096, big, None) == BAD
    for bad in (_block._GradStrides(380, 384, 128, 128), _block._GradStrides(384, 384, 64, 128)):
        assert LIB.eqlin_attention_backward(ref, ctypes.byref(bad), *good, 4096, big, None) == BAD
    bad = _block._GradStrides(384, 388, 128, 128)
    assert LIB.eqlin_attention_backward(ref, ctypes.byref(bad), *good, 4096, big, None) == MISAL
    assert LIB.eqlin_attention_workspace_size(ref, 1, None) == BAD


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8, 4, dtype=torch.bfloat16)
    for call in (lambda: eq.eqlin_add_rmsnorm(x), lambda: eq.eqlin_add_rmsnorm_fp8(x),
                 lambda: eq.eqlin_rmsnorm_backward(x, x),
                 lambda: eq.eqlin_rope(x, torch.zeros(4, 1, dtype=torch.int32), heads=1, sections=(4,)),
                 lambda: eq.eqlin_attention_forward(x, x, x, heads=1),
                 lambda: eq.eqlin_attention_backward(x, x, x, x, x, torch.zeros(1, 4), heads=1),
                 lambda: eq.eqlin_add_rmsnorm(torch.zeros(4, 8))):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    """With stand-ins for the stream and the tensor, so that one device or none is enough."""

    class Stream:
        device = torch.device("cuda:1")

    class Tensor:
        device = torch.device("cuda:0")

    called = []
    with monkeypatch.context() as m:
        m.setattr(_block.torch.cuda, "Stream", Stream)
        m.setattr(_block.torch, "Tensor", Tensor)
        m.setattr(_block.torch.cuda, "stream", lambda s: contextlib.nullcontext(called.append(s)))
        call = _block._in_stream(lambda *a, **k: "done")
        for args, kwargs in (((Tensor(),), {}), ((), {"heads": 2, "x": Tensor()})):
            with pytest.raises(ValueError, match="stream of cuda:0"):
                call(*args, stream=Stream(), **kwargs)
            right = Stream()
            right.device = Tensor.device
            assert call(*args, stream=right, **kwargs) == "done" and called == [right]
            called.clear()


def test_binding_with_a_stream_refuses_cpu_tensors():
    x = torch.zeros(4, 8, 4, dtype=torch.bfloat16)
    for stream in (0, 256):
        with pytest.raises(ValueError):
            eq.eqlin_attention_forward(heads=1, q=x, k=x, v=x, stream=stream)


def test_kernels_read_by_coherent_loads():
    """The block operators' kernels start while the kernel before them still runs, and read what it writes.  The
    non-coherent path is for memory that nothing writes while a kernel runs, and its loads may be moved
    before the wait for that kernel."""
    for path in glob.glob(os.path.join(build.CSRC, "eqlin_attn*")) + [os.path.join(build.CSRC, f"eqlin_{n}.cuh")
                                                                    for n in ("norm", "rope", "vec")]:
        with open(path) as f:
            text = f.read()
        for word in ("__ldg", "ld.global.nc", "__ldcs", "__restrict__"):
            assert word not in text, (path, word)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks behaviour without a GPU")
def test_without_a_gpu_the_calls_report_a_cuda_error():
    assert LIB.eqlin_add_rmsnorm(256, None, None, 512, None, 4, 96, 4, 1e-6, BF, BF, None) == eq.EQLIN_ERR_CUDA
    assert _rope() == eq.EQLIN_ERR_CUDA
    s = _shape()
    assert LIB.eqlin_attention_forward(ctypes.byref(s), 256, 256, 256, 512, None, 1024, 1 << 30,
                                       None) == eq.EQLIN_ERR_CUDA
