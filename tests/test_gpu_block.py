"""Attention over packed sequences, residual RMS norm and rotary positions on the GPU, against
their float64 definitions (block_reference.py) with bounds derived there."""
from __future__ import annotations

import math

import pytest
import torch

import cyclic_group_dft_b200 as eq
import block_reference as ref
from block_reference import within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _randn(*shape, seed, dtype, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


# ------------------------------------------------------------------------------------ norm
NORM_SHAPES = [(1, 8, 1), (3, 1, 8), (5, 96, 4), (257, 96, 4), (7, 64, 8), (33, 32, 16), (2, 100, 2), (4, 192, 4),
               (19, 136, 4), (3, 512, 8), (2, 1024, 16), (70, 4, 2)]
NORM_F32_ONLY = [(3, 3, 1), (9, 5, 2), (2, 2047, 1), (5, 2, 1)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,C,G", NORM_SHAPES + NORM_F32_ONLY)
def test_norm(N, C, G, dtype):
    if dtype != torch.float32 and (N, C, G) in NORM_F32_ONLY:
        pytest.skip("16-byte rows only")
    if dtype == torch.float32 and C * G > 8192:
        pytest.skip("fp32 rows of at most 8192 features")
    eps, u = 1e-6, ref.unit(dtype)
    x, res = _randn(N, C, G, seed=N, dtype=dtype), _randn(N, C, G, seed=C, dtype=dtype, std=3.0)
    w = _randn(C, seed=G, dtype=torch.float32)
    for residual, weight in ((res, w), (None, None), (res, w.to(dtype))):
        y64, r64, _ = ref.add_rmsnorm(x, residual, weight, eps)
        y, r = eq.eqlin_add_rmsnorm(x.to(DEV), None if residual is None else residual.to(DEV),
                                    None if weight is None else weight.to(DEV), eps=eps)
        within(y, y64, (u + ref.E) * y64.abs() + ref.tiny(dtype), "y")
        within(r, r64, (u + 2.0 ** -23) * r64.abs() + ref.tiny(dtype), "r")
    y8, scale, r = eq.eqlin_add_rmsnorm_fp8(x.to(DEV), res.to(DEV), w.to(DEV), eps=eps)
    y64, r64, _ = ref.add_rmsnorm(x, res, w, eps)
    top = y64.abs().amax((1, 2))
    within(scale, torch.where(top > 0, top / 448, torch.ones_like(top)), ref.E * (top / 448 + 1), "scale")
    # e4m3: half a step is 2^-4 of the value, at least 2^-10 (half the smallest subnormal), in scale units
    s = (top / 448)[:, None, None]
    within(y8.float().cpu().double() * scale.cpu().double()[:, None, None], y64,
           (2.0 ** -4 + 4 * ref.E) * y64.abs() + (2.0 ** -10 + ref.E) * s, "y8 * scale")
    within(r, r64, (u + 2.0 ** -23) * r64.abs() + ref.tiny(dtype), "r")
    dy, dsum = _randn(N, C, G, seed=5, dtype=dtype), _randn(N, C, G, seed=6, dtype=dtype)
    for weight, ds in ((w, dsum), (None, None), (w.to(dtype), dsum)):
        dx64, dw64, dx_b, dw_b = ref.rmsnorm_backward(dy, r.cpu(), weight, ds, eps)
        dx, dw = eq.eqlin_rmsnorm_backward(dy.to(DEV), r, None if weight is None else weight.to(DEV),
                                           None if ds is None else ds.to(DEV), eps=eps)
        within(dx, dx64, dx_b, "dx")
        within(dw, dw64, dw_b, "dweight")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("C,G", [(96, 4), (512, 8), (3, 1)])
@pytest.mark.parametrize("size", [1e-34, 1e-36, 1e-38, 1e-40, 1e-42, 1e-44])
def test_norm_fp8_of_tiny_rows(C, G, size, dtype):
    """Rows whose scale is a subnormal number, zeros among them: still y8 * scale within half a step of y."""
    if dtype != torch.float32 and C * G % 8:
        pytest.skip("16-byte rows only")
    N = 5
    x = _randn(N, C, G, seed=1, dtype=dtype)
    x[:, ::3] = 0
    x[0] = 0
    w = torch.full((C,), size)
    y64, _, _ = ref.add_rmsnorm(x, None, w, 1e-6)
    y8, scale, _ = eq.eqlin_add_rmsnorm_fp8(x.to(DEV), None, w.to(DEV))
    top = y64.abs().amax((1, 2))
    # fp32 below 2^-126 has steps of 2^-149: y is off by half of one beside its relative error, the scale by one step
    step = 2.0 ** -149
    want = torch.where(top > step / 2, top / 448, torch.ones_like(top))
    within(scale, want, ref.E * want + 1.01 * step, "scale")
    s = scale.cpu().double()[:, None, None]
    # e4m3: half a step is 2^-4 of the value, at least 2^-10 of the scale
    within(y8.float().cpu().double() * s, y64, (2.0 ** -4 + 4 * ref.E) * y64.abs() + (2.0 ** -10 + ref.E) * s + 2 * step,
           "y8 * scale")


def test_norm_zero_rows_and_empty_batches():
    x = torch.zeros(3, 16, 4, dtype=torch.bfloat16, device=DEV)
    y8, scale, r = eq.eqlin_add_rmsnorm_fp8(x, x)
    assert (scale == 1).all() and (y8.float() == 0).all() and (r == 0).all()
    e = x[:0]
    y, r = eq.eqlin_add_rmsnorm(e, e)
    assert y.shape == e.shape and r.shape == e.shape
    dx, dw = eq.eqlin_rmsnorm_backward(e, e)
    assert dx.shape == e.shape and (dw == 0).all()
    # infinities and NaN stay in their rows
    x = torch.ones(4, 16, 4, device=DEV)
    x[1, 3, 2], x[2, 0, 0] = float("nan"), float("inf")
    y, _ = eq.eqlin_add_rmsnorm(x, None)
    assert y[1].isnan().all() and y[2].isnan().any() and torch.isfinite(y[[0, 3]]).all()


def test_norm_in_place_and_large_values():
    x, res = _randn(50, 96, 4, seed=1, dtype=torch.bfloat16).to(DEV), _randn(50, 96, 4, seed=2, dtype=torch.bfloat16).to(DEV)
    y, r = eq.eqlin_add_rmsnorm(x, res)
    x2, res2 = x.clone(), res.clone()
    y2, r2 = eq.eqlin_add_rmsnorm(x2, res2, y=x2, sum_out=res2)      # y over x, the sum over the residual
    assert torch.equal(y, y2) and torch.equal(r, r2) and y2.data_ptr() == x2.data_ptr()
    dy = _randn(50, 96, 4, seed=3, dtype=torch.bfloat16).to(DEV)
    dx, dw = eq.eqlin_rmsnorm_backward(dy, r, dsum=dy)
    dx2, dw2 = eq.eqlin_rmsnorm_backward(dy, r, dsum=dy, dx=dy)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    with pytest.raises(ValueError):
        eq.eqlin_add_rmsnorm(x, res, y=x, sum_out=x)
    big = torch.full((2, 16, 4), 3e4, dtype=torch.float16, device=DEV)   # squares overflow fp16, not fp32
    y, _ = eq.eqlin_add_rmsnorm(big, None)
    assert (y.float() - 1).abs().max() <= 2.0 ** -11


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_in_place_without_a_residual_keeps_the_sum(dtype):
    """y over x and no residual: r is the sum that the gradients need, not what y left there."""
    x, w = _randn(50, 96, 4, seed=1, dtype=dtype).to(DEV), _randn(96, seed=2, dtype=torch.float32).to(DEV)
    y, r = eq.eqlin_add_rmsnorm(x, None, w)
    assert r.data_ptr() == x.data_ptr()                            # the sum is x itself
    x2 = x.clone()
    y2, r2 = eq.eqlin_add_rmsnorm(x2, None, w, y=x2)
    assert y2.data_ptr() == x2.data_ptr() and torch.equal(y2, y) and torch.equal(r2, x)
    e = x[:0]
    assert eq.eqlin_add_rmsnorm(e, None, w, y=e)[1].shape == e.shape


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C,G", [(96, 4), (8, 1), (512, 8)])      # 16 rows of a block at once, 64 (fp32) and more, one
@pytest.mark.parametrize("N", [1, 17, 50])
def test_norm_gradient_without_eps(N, C, G, dtype):
    """eps = 0 and rows that do not fill the blocks: places past the last row add nothing to dweight."""
    x, w = _randn(N, C, G, seed=N, dtype=dtype), _randn(C, seed=C, dtype=torch.float32)
    dy, dsum = _randn(N, C, G, seed=1, dtype=dtype), _randn(N, C, G, seed=2, dtype=dtype)
    for ds in (None, dsum):                                        # with the ring of copies and without
        dx64, dw64, dx_b, dw_b = ref.rmsnorm_backward(dy, x, w, ds, 0.0)
        dx, dw = eq.eqlin_rmsnorm_backward(dy.to(DEV), x.to(DEV), w.to(DEV), None if ds is None else ds.to(DEV), eps=0.0)
        within(dx, dx64, dx_b, "dx")
        within(dw, dw64, dw_b, "dweight")


def test_norm_gradient_against_differences():
    N, C, G, eps = 5, 24, 4, 1e-3
    x = _randn(N, C, G, seed=1, dtype=torch.float64)
    w, dy = _randn(C, seed=2, dtype=torch.float64), _randn(N, C, G, seed=3, dtype=torch.float64)
    f = lambda x, w: float((ref.add_rmsnorm(x, None, w, eps)[0] * dy).sum())   # noqa: E731
    r = x.float()
    dx, dw = eq.eqlin_rmsnorm_backward(dy.float().to(DEV), r.to(DEV), w.float().to(DEV), eps=eps)
    h = 1e-5   # central differences of a smooth function in float64: truncation and rounding below 1e-8
    for (n, c, g) in ((0, 0, 0), (4, 23, 3), (2, 11, 1)):
        d = torch.zeros_like(x)
        d[n, c, g] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[n, c, g].item()) < 2e-5
    for c in (0, 7, 23):
        d = torch.zeros_like(w)
        d[c] = h
        assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[c].item()) < 2e-4


# ------------------------------------------------------------------------------------ rope
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,heads,Dh,G,sections,base,far", [
    (1, 1, 2, 1, (1,), 100.0, 10), (5, 3, 8, 4, (2, 2), 100.0, 56), (300, 6, 32, 4, (8, 8), 10000.0, 1000),
    (17, 4, 8, 16, (2, 1, 1), 100.0, 14), (33, 2, 6, 2, (0, 3), 10.0, 1 << 20), (9, 5, 10, 1, (5,), 10000.0, 1 << 30),
    (2, 1, 256, 2, (100, 20, 7, 1), 500.0, 100000), (40, 12, 8, 8, (4,), 1.0, 7), (3, 2, 12, 2, (6,), 100.0, 50),
])
def test_rope(N, heads, Dh, G, sections, base, far, dtype):
    x = _randn(N, heads * Dh, G, seed=N, dtype=dtype)
    pos = torch.randint(-far, far, (N, len(sections)), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    y64, bound = ref.rope(x, pos, heads, sections, base)
    y = eq.eqlin_rope(x.to(DEV), pos.to(DEV), heads=heads, sections=sections, base=base)
    # beside the bound of the arithmetic: the reference's own angle, position * frequency rounded to
    # float64, is off by up to 2^-52 of up to `far` radians
    slack = far * 2.0 ** -51 * x.double().abs().max()
    within(y, y64, bound + slack, "y")
    back64, bound = ref.rope(y.cpu(), pos, heads, sections, base, inverse=True)
    back = eq.eqlin_rope(y, pos.to(DEV), heads=heads, sections=sections, base=base, inverse=True)
    within(back, back64, bound + 2 * slack, "inverse")


@pytest.mark.parametrize("offset,width", [(0, 96), (8, 104), (4, 100), (1, 97), (2, 98)])
def test_rope_slices_and_in_place(offset, width):
    """Channel slices of a wider tensor at every alignment, and y over x."""
    G, heads, Dh = 2, 3, 8
    joint = _randn(21, width, G, seed=3, dtype=torch.bfloat16).to(DEV)
    before = joint.clone()
    pos = torch.randint(0, 99, (21, 2), dtype=torch.int32).to(DEV)
    x = joint[:, offset:offset + heads * Dh]
    want = eq.eqlin_rope(x.contiguous(), pos, heads=heads, sections=(2, 2))
    assert torch.equal(eq.eqlin_rope(x, pos, heads=heads, sections=(2, 2)), want)
    eq.eqlin_rope(x, pos, heads=heads, sections=(2, 2), out=x)
    assert torch.equal(x, want)
    before[:, offset:offset + heads * Dh] = want
    assert torch.equal(joint, before)                       # nothing beside the slice changed
    with pytest.raises(ValueError):
        eq.eqlin_rope(joint.transpose(1, 2), pos, heads=1, sections=(1,))
    assert eq.eqlin_rope(x[:0], pos[:0], heads=heads, sections=(2, 2)).shape == (0, heads * Dh, G)


def test_rope_gradient_is_the_inverse():
    x, dy = _randn(7, 16, 4, seed=1, dtype=torch.float32).to(DEV), _randn(7, 16, 4, seed=2, dtype=torch.float32).to(DEV)
    pos = torch.randint(0, 50, (7, 2), dtype=torch.int32).to(DEV)
    kw = dict(heads=2, sections=(2, 2), base=100.0)
    left = (eq.eqlin_rope(x, pos, **kw).double() * dy.double()).sum()
    right = (x.double() * eq.eqlin_rope(dy, pos, inverse=True, **kw).double()).sum()
    assert abs(left - right) <= ref.E * (x.double().abs().sum() + dy.double().abs().sum())


# ------------------------------------------------------------------------------- attention
SELF = [
    ([1], 1, 1, 8, False), ([1], 2, 1, 64, True), ([49] * 5, 3, 3, 128, False), ([64], 2, 2, 64, True),
    ([63, 65, 1, 0, 128, 129, 200], 2, 1, 64, True), ([63, 65, 1, 0, 128, 129, 200], 2, 2, 128, False),
    ([5, 0, 0, 3], 6, 2, 40, True), ([256, 255, 257], 3, 1, 72, True), ([700], 2, 2, 96, False),
    ([130, 12], 4, 1, 16, False), ([31] * 9, 2, 1, 24, True), ([0, 0, 17], 1, 1, 32, False),
    ([385, 2, 640], 2, 1, 120, True), ([2] * 70, 1, 1, 56, True), ([16] * 7, 5, 1, 128, True),
    ([17, 30, 1, 32] * 3, 3, 3, 64, False), ([20] * 30 + [200, 0, 129], 6, 3, 80, True), ([1] * 40 + [300], 2, 1, 128, True),
]
CROSS = [
    ([1, 1, 1], [300, 0, 7], 4, 2, 64, False), ([10, 0, 130, 3], [0, 20, 50, 400], 2, 1, 128, True),
    ([1], [2000], 8, 2, 64, False), ([200], [70], 2, 2, 48, True), ([5, 129], [513, 128], 3, 1, 80, False),
    ([1, 0, 3, 1], [700, 50, 0, 1000], 6, 2, 128, True), ([2, 1], [300, 900], 12, 4, 72, False),
    ([1] * 20, [200 + 7 * i for i in range(20)], 2, 1, 40, False), ([1, 1], [4000, 3], 8, 1, 64, False),
    ([5, 1, 9], [600, 400, 8], 1, 1, 16, True), ([30], [5000], 1, 1, 128, True),
    ([0, 0], [5, 9], 2, 1, 64, True), ([5, 9], [0, 0], 2, 1, 64, True), ([2], [1500], 2, 1, 128, True),
]


def _attention(q_lens, k_lens, H, Hk, D, causal, dtype, G=4, seed=0, tail=0, std=1.0):
    """Runs forward and backward; returns the GPU's outputs and the reference's with their bounds."""
    G = math.gcd(G, D)
    Nq, Nk, Dh = sum(q_lens), sum(k_lens), D // G
    q = _randn(Nq + tail, H * Dh, G, seed=seed, dtype=dtype, std=std)
    k, v = (_randn(Nk + tail, Hk * Dh, G, seed=seed + i, dtype=dtype, std=s) for i, s in ((1, std), (2, 1.0)))
    do = _randn(Nq + tail, H * Dh, G, seed=seed + 3, dtype=dtype)
    want, bound = ref.attention(q, k, v, do, q_lens, k_lens, H, Hk, causal)
    kw = dict(heads=H, kv_heads=Hk, causal=causal, q_offsets=ref.offsets(q_lens, DEV),
              k_offsets=ref.offsets(k_lens, DEV))
    qd, kd, vd, dod = (t.to(DEV) for t in (q, k, v, do))
    o, lse = eq.eqlin_attention_forward(qd, kd, vd, **kw)
    # the gradients get the definition's o and lse, so that their bounds need not count the forward's
    o_ref = want["o"].to(dtype).to(DEV)
    lse_ref = want["lse"].float().to(DEV)
    dq, dk, dv = eq.eqlin_attention_backward(dod, qd, kd, vd, o_ref, lse_ref, **kw)
    torch.cuda.synchronize()
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, want, bound


def _check_attention(got, want, bound):
    for name in ("o", "lse", "dq", "dk", "dv"):
        within(got[name], want[name], bound[name], name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,H,Hk,D,causal", SELF)
def test_self_attention(lens, H, Hk, D, causal, dtype):
    _check_attention(*_attention(lens, lens, H, Hk, D, causal, dtype, seed=len(lens) * 7 + D))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("q_lens,k_lens,H,Hk,D,causal", CROSS)
def test_cross_attention(q_lens, k_lens, H, Hk, D, causal, dtype):
    _check_attention(*_attention(q_lens, k_lens, H, Hk, D, causal, dtype, seed=len(q_lens) + D))


@pytest.mark.parametrize("q_lens,k_lens,H,Hk,D,causal", [
    ([63, 65, 1, 0, 128, 129, 200], None, 6, 3, 64, True), ([49] * 5, None, 8, 8, 128, False),
    ([385, 2, 640], None, 16, 4, 120, True), ([65], None, 40, 8, 8, False), ([257, 3], None, 20, 20, 72, True),
    ([10, 0, 130, 3], [0, 20, 50, 400], 12, 6, 128, True), ([200], [70], 12, 4, 48, True),
    ([5, 9], [0, 0], 20, 20, 64, True), ([0, 0], [5, 9], 20, 10, 64, False), ([20, 70], [130, 61], 38, 2, 40, False),
])
def test_fp32_attention_of_many_tiles(q_lens, k_lens, H, Hk, D, causal):
    """Enough tiles of 64 rows that fp32 goes to the tensor cores."""
    k_lens = q_lens if k_lens is None else k_lens
    _check_attention(*_attention(q_lens, k_lens, H, Hk, D, causal, torch.float32, seed=D + H))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,most,H,Hk,D,causal,other", [
    (700, 64, 2, 2, 64, False, False), (650, 49, 2, 2, 128, True, True), (3000, 16, 1, 1, 8, False, True),
    (1300, 30, 2, 2, 24, True, False), (700, 60, 4, 2, 16, False, True),
])
def test_many_short_sequences(n, most, H, Hk, D, causal, other, dtype):
    """Mostly one tile each, with empty and longer ones between them; keys of other lengths than the queries'."""
    g = torch.Generator().manual_seed(n + D)
    lens = lambda: torch.randint(0, most + 1, (n,), generator=g).tolist()
    q_lens = lens()
    k_lens = lens() if other else list(q_lens)
    for i in (3, n // 2, n - 1):                      # each longer than a tile on one side or both
        q_lens[i] = 70 if i != 3 or not other else 5
        k_lens[i] = 131 if other else q_lens[i]
    _check_attention(*_attention(q_lens, k_lens, H, Hk, D, causal, dtype, seed=n))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,q_most,k_most,H,Hk,D,causal", [
    (60, 140, 0, 8, 8, 64, True), (57, 120, 0, 8, 2, 128, False),      # self-attention over about one and two tiles
    (60, 33, 500, 8, 8, 40, True), (60, 60, 400, 8, 4, 128, False),    # few tiles of queries over several of keys
    (70, 1, 900, 16, 2, 64, False), (64, 16, 700, 8, 8, 128, True),    # packed heads; one and a few queries
    (3, 40, 1500, 6, 2, 72, True), (2, 100, 1200, 4, 4, 64, False),    # split keys for more than 16 packed rows
])
def test_attention_of_many_tiles(n, q_most, k_most, H, Hk, D, causal, dtype):
    g = torch.Generator().manual_seed(n + D)
    q_lens = torch.randint(0, q_most + 1, (n,), generator=g).tolist() if q_most > 1 else [1] * n
    k_lens = torch.randint(k_most // 2, k_most + 1, (n,), generator=g).tolist() if k_most else q_lens
    _check_attention(*_attention(q_lens, k_lens, H, Hk, D, causal, dtype, seed=n))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens,k_lens,H,Hk,D,causal", [
    ([3] * 300 + [1500] + [7] * 200, None, 2, 1, 64, True),     # one long sequence among many short ones
    ([20] * 60 + [900], [20] * 60 + [1100], 2, 2, 128, False),
    ([1200], None, 6, 2, 128, True), ([900, 1, 700], None, 4, 1, 64, False),   # long ones with shared key heads
    ([700], [1900], 4, 2, 96, True),
])
def test_attention_of_outliers_and_long_sequences(lens, k_lens, H, Hk, D, causal, dtype):
    _check_attention(*_attention(lens, lens if k_lens is None else k_lens, H, Hk, D, causal, dtype, seed=D))


@pytest.mark.parametrize("q_len,k_len", [(30, 8192), (8192, 30)])
def test_fp32_attention_sums_do_not_drift(q_len, k_len):
    """Thousands of terms of one sign: roundings that all go one way would add up in o, or in dv."""
    H, D, G = 40, 16, 4
    q, k = _randn(q_len, H * D // G, G, seed=1, dtype=torch.float32), _randn(k_len, H * D // G, G, seed=2, dtype=torch.float32)
    v = 1 + _randn(k_len, H * D // G, G, seed=3, dtype=torch.float32).abs()
    do = 1 + _randn(q_len, H * D // G, G, seed=4, dtype=torch.float32).abs()
    want, bound = ref.attention(q, k, v, do, [q_len], [k_len], H, H, False)
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    o, lse = eq.eqlin_attention_forward(q, k, v, heads=H)
    dq, dk, dv = eq.eqlin_attention_backward(do, q, k, v, want["o"].float().to(DEV), want["lse"].float().to(DEV), heads=H)
    _check_attention({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, want, bound)


def test_fp32_not_a_number_stays_in_its_sequence_of_many_tiles():
    lens, H, D, G = [70, 5, 130], 16, 64, 4
    n = sum(lens)
    q, k, v, do = (_randn(n, H * D // G, G, seed=i, dtype=torch.float32) for i in range(4))
    for t in (q, k, v, do):
        t[70:75] = float("nan")
    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, q_offsets=off, k_offsets=off)
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    o, lse = eq.eqlin_attention_forward(q, k, v, **kw)
    grads = eq.eqlin_attention_backward(do, q, k, v, o, lse, **kw)
    torch.cuda.synchronize()
    for t in (o, lse.T, *grads):
        assert t[70:75].isnan().any()
        assert torch.isfinite(t[:70]).all() and torch.isfinite(t[75:]).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_with_one_weight_far_above_the_others(dtype):
    """Scores of several hundred: the running maximum moves far, most weights vanish."""
    got, want, bound = _attention([150, 260], [150, 260], 2, 2, 64, False, dtype, seed=3, std=6.0)
    _check_attention(got, want, bound)


@pytest.mark.parametrize("lens,k_lens,H,Hk,D,causal", [
    ([700], None, 2, 2, 64, False), ([700], None, 2, 1, 128, True), ([130, 300], None, 4, 2, 72, True),   # tiles of 128
    ([5, 200], [900, 640], 3, 3, 64, False),
    ([49] * 4, None, 3, 3, 128, False), ([30, 17], None, 2, 2, 64, True), ([12] * 5, None, 5, 5, 40, False),   # one tile
    ([60] * 3, None, 4, 2, 64, True), ([13, 16], None, 6, 2, 128, False), ([8, 8, 8, 150], None, 2, 2, 64, False),
])
@pytest.mark.parametrize("do_exp,v_exp,q_exp,k_exp", [
    (-14, -6, -8, 8), (-14, -6, 8, -8), (-12, 3, -6, 6),          # ds below fp16's smallest number, or among its subnormal ones
    (12, 8, -4, -4), (11, -2, -4, -4), (0, 9, -2, -2),            # and above its largest
])
def test_fp16_gradients_of_small_and_large_values(lens, k_lens, H, Hk, D, causal, do_exp, v_exp, q_exp, k_exp):
    """The gradients are linear in dO and, with o, in V: those of dO 2^a and V 2^b are 2^(a+b) times (dv: 2^a) those of
    values near 1, whose bounds hold for them too, but for the rounding of outputs (and of the given o) near zero: ds must
    not be lost because it is small, nor become infinite because it is large."""
    k_lens, dtype, G = lens if k_lens is None else k_lens, torch.float16, math.gcd(4, D)
    Dh, Nq, Nk = D // G, sum(lens), sum(k_lens)

    def pair(n, h, seed, e):         # values near 1, in steps of 2^-10, and the same times 2^e: both are fp16 numbers
        near = (_randn(n, h * Dh, G, seed=seed, dtype=torch.float16).float() * 1024).round() / 1024
        t = (near * 2.0 ** e).half()
        assert torch.isfinite(t).all() and torch.equal(near.double() * 2.0 ** e, t.double())
        return t.to(DEV), near.half()

    (q, q1), (k, k1), (v, v1), (do, do1) = pair(Nq, H, 1, q_exp), pair(Nk, Hk, 2, k_exp), pair(Nk, Hk, 3, v_exp), pair(Nq, H, 4, do_exp)
    scale = D ** -0.5
    want, bound = ref.attention(q1, k1, v1, do1, lens, k_lens, H, Hk, causal, scale=scale * 2.0 ** (q_exp + k_exp),
                                o_err=ref.tiny(dtype) * 2.0 ** -v_exp)
    o = (want["o"].half().float() * 2.0 ** v_exp).half()
    kw = dict(heads=H, kv_heads=Hk, causal=causal, q_offsets=ref.offsets(lens, DEV), k_offsets=ref.offsets(k_lens, DEV))
    got = eq.eqlin_attention_backward(do, q, k, v, o.to(DEV), want["lse"].float().to(DEV), **kw)
    # the reference has 2^(q_exp + k_exp) in its scale, and k or q near 1
    for name, t, e in (("dq", got[0], do_exp + v_exp - q_exp), ("dk", got[1], do_exp + v_exp - k_exp), ("dv", got[2], do_exp)):
        t = t.double().cpu()
        # a gradient itself may be above fp16's largest number: it may be infinite where its bound reaches that far
        most = torch.finfo(dtype).max
        past = t.isinf() & (t.sign() == want[name].sign()) & ((want[name].abs() + bound[name]) * 2.0 ** e > most)
        t = torch.where(past, want[name] * 2.0 ** e, t)
        assert past.double().mean() < 0.05
        within(t * 2.0 ** -e, want[name], bound[name] + ref.tiny(dtype) * 2.0 ** -e, name)


@pytest.mark.parametrize("D,H,Hk,a,b", [(128, 1, 1, 300, 4096), (64, 2, 1, 4096, 200), (64, 2, 2, 50, 3000)])
@pytest.mark.parametrize("which", ["dq", "dk", "dv"])
def test_fp16_gradients_keep_their_precision_over_long_sequences(D, H, Hk, a, b, which):
    """Thousands of keys (or queries) and dO of 2^-10: ds and small weights lie where fp16 has few bits left.  Normwise:
    ds and p are rounded once, the output once, each by at most u relative, independently and so by u / sqrt(3) in the
    mean square: u sqrt(2 / 3) together; twice u leaves room for fp32.  k, or q, is large so that the gradient itself
    is no subnormal number."""
    G, u, e = 4, ref.unit(torch.float16), {"dq": 7, "dk": -7, "dv": 0}[which]
    q, do = _randn(a, H * D // G, G, seed=1, dtype=torch.float16, std=2.0 ** -e), _randn(a, H * D // G, G, seed=2, dtype=torch.float16, std=2.0 ** -10)
    k, v = (_randn(b, Hk * D // G, G, seed=s, dtype=torch.float16, std=d) for s, d in ((3, 2.0 ** e), (4, 1.0)))
    if which == "dv":
        do = do * 64
    want, _ = ref.attention(q, k, v, do, [a], [b], H, Hk, False)
    got = eq.eqlin_attention_backward(do.to(DEV), q.to(DEV), k.to(DEV), v.to(DEV), want["o"].half().to(DEV),
                                      want["lse"].float().to(DEV), heads=H, kv_heads=Hk)[["dq", "dk", "dv"].index(which)]
    err = float((got.double().cpu() - want[which]).norm() / want[which].norm())
    assert err <= 2 * u, (err, u)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lens", [[49, 3, 20], [130, 5, 260]])
@pytest.mark.parametrize("causal", [False, True])
def test_not_a_number_stays_in_its_sequence(lens, causal, dtype):
    """The middle sequence holds NaN and infinities everywhere; so do the rows behind the last one."""
    H, D, G = 2, 64, 4
    n, tail = sum(lens), 9
    q, k, v, do = (_randn(n + tail, H * D // G, G, seed=i, dtype=dtype) for i in range(4))
    a, b = lens[0], lens[0] + lens[1]
    keep = torch.cat([torch.arange(a), torch.arange(b, n)])
    want, bound = ref.attention(q[keep], k[keep], v[keep], do[keep], [lens[0], lens[2]], [lens[0], lens[2]], H, H, causal,
                                chained=True)
    for t in (q, k, v, do):
        t[a:b] = float("nan")
        t[n:] = float("inf")
    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, causal=causal, q_offsets=off, k_offsets=off)
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    mark = [torch.full_like(q, 7.0) for _ in range(4)]
    lse = torch.full((H, n + tail), 7.0, device=DEV)
    eq.eqlin_attention_forward(q, k, v, o=mark[0], lse=lse, **kw)
    o = mark[0].clone()
    eq.eqlin_attention_backward(do, q, k, v, o, lse, grads=tuple(mark[1:]), **kw)
    for t in mark:
        assert (t[n:] == 7).all()                              # rows behind the last sequence: as they were
        assert t[a:b].isnan().any()
    assert (lse[:, n:] == 7).all()
    within(mark[0][keep.to(DEV)], want["o"], bound["o"], "o")
    within(lse[:, keep.to(DEV)], want["lse"], bound["lse"], "lse")
    for t, name in zip(mark[1:], ("dq", "dk", "dv")):
        within(t[keep.to(DEV)], want[name], bound[name], name)


def test_joint_projection_slices():
    """q, k, v as channel slices of one tensor and gradients into slices of another."""
    H, Hk, Dh, G = 3, 1, 16, 4
    lens = [100, 29, 150]
    n, C = sum(lens), (H + 2 * Hk) * Dh
    joint = _randn(n, C, G, seed=1, dtype=torch.bfloat16).to(DEV)
    q, k, v = joint[:, :H * Dh], joint[:, H * Dh:(H + Hk) * Dh], joint[:, (H + Hk) * Dh:]
    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, kv_heads=Hk, q_offsets=off, k_offsets=off, causal=True)
    o, lse = eq.eqlin_attention_forward(q, k, v, **kw)
    o2, lse2 = eq.eqlin_attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    wide = torch.zeros(n, H * Dh + 8, G, dtype=torch.bfloat16, device=DEV)
    eq.eqlin_attention_forward(q, k, v, o=wide[:, 4:4 + H * Dh], **kw)
    assert torch.equal(wide[:, 4:4 + H * Dh], o) and (wide[:, :4] == 0).all() and (wide[:, 4 + H * Dh:] == 0).all()
    do = _randn(n, H * Dh, G, seed=2, dtype=torch.bfloat16).to(DEV)
    dj = torch.zeros_like(joint)
    grads = (dj[:, :H * Dh], dj[:, H * Dh:(H + Hk) * Dh], dj[:, (H + Hk) * Dh:])
    eq.eqlin_attention_backward(do, q, k, v, o, lse, grads=grads, **kw)
    plain = eq.eqlin_attention_backward(do, q.contiguous(), k.contiguous(), v.contiguous(), o, lse, **kw)
    assert torch.equal(dj, torch.cat(plain, 1))
    # a single sequence: no offsets
    one = eq.eqlin_attention_forward(q[:100], k[:100], v[:100], heads=H, kv_heads=Hk, causal=True)[0]
    within(one, o[:100].double(), 2.0 ** -7 * o[:100].double().abs() + 2.0 ** -9, "one sequence")


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_is_deterministic_and_equivariant(dtype):
    H, Dh, G = 2, 16, 4
    lens = [200, 33, 129]
    n = sum(lens)
    q, k, v, do = (_randn(n, H * Dh, G, seed=i, dtype=dtype).to(DEV) for i in range(4))
    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, q_offsets=off, k_offsets=off)
    o, lse = eq.eqlin_attention_forward(q, k, v, **kw)
    g = eq.eqlin_attention_backward(do, q, k, v, o, lse, **kw)
    for _ in range(3):
        o2, lse2 = eq.eqlin_attention_forward(q, k, v, **kw)
        g2 = eq.eqlin_attention_backward(do, q, k, v, o, lse, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(g, g2))
    want, bound = ref.attention(q.cpu(), k.cpu(), v.cpu(), do.cpu(), lens, lens, H, H, False)
    turned = [t.roll(1, dims=2).contiguous() for t in (q, k, v)]
    o2, _ = eq.eqlin_attention_forward(*turned, **kw)
    within(o2, o.roll(1, dims=2).double(), 2 * bound["o"].roll(1, dims=2), "shifted o")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [[0, 50, 20, 130], [-5, 40, 90, 130], [10, 60, 200, 300], [130, 0, 130, 0],
                                 [2 ** 31 - 1, -2 ** 31, 0, 130]])
def test_bad_offsets_stay_inside_the_tensors(bad, dtype):
    """Offsets that decrease or point outside are clamped: the call returns, guard rows stay."""
    n, H, G = 130, 2, 4
    q, k, v, do = (_randn(n + 8, H * 16, G, seed=i, dtype=dtype).to(DEV) for i in range(4))
    off = torch.tensor(bad, dtype=torch.int32, device=DEV)
    kw = dict(heads=H, q_offsets=off, k_offsets=off, causal=True)
    outs = [torch.full_like(q, 7.0) for _ in range(4)]
    lse = torch.zeros(H, n, device=DEV)
    eq.eqlin_attention_forward(q[:n], k[:n], v[:n], o=outs[0][:n], lse=lse, **kw)
    eq.eqlin_attention_backward(do[:n], q[:n], k[:n], v[:n], outs[0][:n], lse, grads=tuple(t[:n] for t in outs[1:]), **kw)
    torch.cuda.synchronize()
    assert all((t[n:] == 7).all() for t in outs)


def test_attention_gradient_against_differences():
    lens, H, Dh, G, D = [7, 5], 2, 4, 2, 8
    n = sum(lens)
    ts = [_randn(n, H * Dh, G, seed=i, dtype=torch.float64) for i in range(4)]
    do = ts[3]

    def f(q, k, v):
        return float((ref.attention(q, k, v, do, lens, lens, H, H, True)[0]["o"] * do).sum())

    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, q_offsets=off, k_offsets=off, causal=True)
    dev = [t.float().to(DEV) for t in ts]
    o, lse = eq.eqlin_attention_forward(*dev[:3], **kw)
    grads = eq.eqlin_attention_backward(dev[3], *dev[:3], o, lse, **kw)
    for which in range(3):
        for at in ((0, 0, 0), (6, 3, 1), (11, 7, 0), (8, 5, 1)):
            d = [torch.zeros_like(t) for t in ts[:3]]
            d[which][at] = 1e-5
            up, down = f(*(t + e for t, e in zip(ts, d))), f(*(t - e for t, e in zip(ts, d)))
            # the inputs' rounding to fp32 moves the gradient by about 1e-6, the differences by 1e-9
            assert abs((up - down) / 2e-5 - grads[which][at].item()) < 2e-5


def test_streams_graphs_and_two_calls_at_once():
    """A captured call replayed on new inputs, and two calls in flight on two streams."""
    H, Dh, G = 4, 16, 4
    lens = [150, 49, 128, 1]
    n = sum(lens)
    off = ref.offsets(lens, DEV)
    kw = dict(heads=H, q_offsets=off, k_offsets=off, causal=True)
    make = lambda s: [_randn(n, H * Dh, G, seed=s + i, dtype=torch.bfloat16).to(DEV) for i in range(4)]   # noqa: E731
    w = _randn(H * Dh, seed=1, dtype=torch.float32).to(DEV)
    pos = torch.randint(0, 20, (n, 2), dtype=torch.int32).to(DEV)

    def step(q, k, v, do):
        q2 = eq.eqlin_rope(q, pos, heads=H, sections=(4, 4))
        o, lse = eq.eqlin_attention_forward(q2, k, v, **kw)
        y, r = eq.eqlin_add_rmsnorm(o, q, w)
        dr, dw = eq.eqlin_rmsnorm_backward(do, r, w)
        return (o, y, dr, dw) + eq.eqlin_attention_backward(dr, q2, k, v, o, lse, **kw)

    a, b = make(10), make(20)
    want_a, want_b = [t.clone() for t in step(*a)], [t.clone() for t in step(*b)]
    static = [t.clone() for t in a]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(*static)
    for x, want in ((a, want_a), (b, want_b), (a, want_a)):
        for s, t in zip(static, x):
            s.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            o1 = step(*a)
        with torch.cuda.stream(s2):
            o2 = step(*b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(o1, want_a))
        assert all(torch.equal(u, v) for u, v in zip(o2, want_b))


def test_calls_on_a_given_stream():
    """stream=: a torch Stream or its number; allocations inside belong to it, and work that is queued on the
    current stream neither delays nor disturbs the call."""
    H, Dh, G = 4, 16, 4
    lens = [1, 1, 2]
    k_lens = [3000, 500, 1200]                      # split keys: a workspace that the call gives up on return
    q = _randn(sum(lens), H * Dh, G, seed=1, dtype=torch.bfloat16).to(DEV)
    k, v = (_randn(sum(k_lens), H * Dh, G, seed=i, dtype=torch.bfloat16).to(DEV) for i in (2, 3))
    kw = dict(heads=H, q_offsets=ref.offsets(lens, DEV), k_offsets=ref.offsets(k_lens, DEV))
    x = _randn(300, 96, 4, seed=4, dtype=torch.bfloat16).to(DEV)
    pos = torch.ones(300, 1, dtype=torch.int32, device=DEV)
    want = eq.eqlin_attention_forward(q, k, v, **kw) + eq.eqlin_rmsnorm_backward(x, x)
    want += (eq.eqlin_rope(x, pos, 1, (48,)),)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        noise = torch.randn(2048, 2048, device=DEV)
        for _ in range(10):
            noise = (noise @ noise).clamp_(-1, 1)   # keeps the current stream busy, and its allocator
            got = eq.eqlin_attention_forward(q, k, v, stream=stream, **kw)
            got += eq.eqlin_rmsnorm_backward(x, x, stream=stream)
            got += (eq.eqlin_rope(x, pos, 1, (48,), stream=stream),)
            torch.full((1 << 20,), 3.0, device=DEV)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_stream_numbers_with_keyword_arguments_in_any_order():
    x = _randn(30, 16, 4, seed=1, dtype=torch.bfloat16).to(DEV)
    pos = torch.arange(30, dtype=torch.int32, device=DEV)[:, None].contiguous()
    want = eq.eqlin_rope(x, pos, 2, (4,)), eq.eqlin_attention_forward(x, x, x, 2)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side.cuda_stream, side, 0):
        y = eq.eqlin_rope(heads=2, sections=(4,), positions=pos, x=x, stream=stream)
        o, _ = eq.eqlin_attention_forward(heads=2, causal=False, v=x, k=x, q=x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(o, want[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_transformer_block(dtype):
    """norm -> joint projection -> rotary positions -> attention -> projection -> add and norm, forward
    and gradients, through the layers and the operators together, against float64."""
    import oracle
    C, G, H, lens = 32, 4, 4, [49, 30, 130]
    n, Dh, eps = sum(lens), C // H, 1e-6
    x = _randn(n, C, G, seed=1, dtype=dtype)
    w1, w2 = _randn(C, seed=2, dtype=dtype, std=0.2) + 1, _randn(C, seed=3, dtype=dtype, std=0.2) + 1
    wqkv = _randn(3 * C, C, G, seed=4, dtype=dtype, std=(C * G) ** -0.5)
    wo = _randn(C, C, G, seed=5, dtype=dtype, std=(C * G) ** -0.5)
    dz = _randn(n, C, G, seed=6, dtype=dtype)
    side = 7
    pos = torch.stack([torch.arange(n) // side, torch.arange(n) % side], 1).to(torch.int32)
    off = ref.offsets(lens, DEV)
    qkv_layer = eq.prepare(wqkv.to(DEV), None, io_dtype=dtype, backward=True)
    out_layer = eq.prepare(wo.to(DEV), None, io_dtype=dtype, backward=True)
    d = lambda t: t.to(DEV)   # noqa: E731
    rope = dict(heads=2 * H, sections=(Dh // 4, Dh // 4), base=100.0)
    att = dict(heads=H, q_offsets=off, k_offsets=off)
    # forward
    y, r = eq.eqlin_add_rmsnorm(d(x), None, d(w1), eps=eps)
    joint = qkv_layer.forward(y)
    qk, v = joint[:, :2 * C], joint[:, 2 * C:]
    eq.eqlin_rope(qk, d(pos), out=qk, **rope)
    o, lse = eq.eqlin_attention_forward(qk[:, :C], qk[:, C:], v, **att)
    a = out_layer.forward(o)
    z, r2 = eq.eqlin_add_rmsnorm(a, r, d(w2), eps=eps)
    # gradients
    dr2, dw2 = eq.eqlin_rmsnorm_backward(d(dz), r2, d(w2), eps=eps)
    do = out_layer.backward_dx(dr2)
    dwo, _ = out_layer.backward_dw(o, dr2, with_bias=False)
    dj = torch.empty_like(joint)
    eq.eqlin_attention_backward(do, qk[:, :C], qk[:, C:], v, o, lse, grads=(dj[:, :C], dj[:, C:2 * C], dj[:, 2 * C:]), **att)
    eq.eqlin_rope(dj[:, :2 * C], d(pos), out=dj[:, :2 * C], inverse=True, **rope)
    dy = qkv_layer.backward_dx(dj)
    dwqkv, _ = qkv_layer.backward_dw(y, dj, with_bias=False)
    dx, dw1 = eq.eqlin_rmsnorm_backward(dy, r, d(w1), dsum=dr2, eps=eps)
    torch.cuda.synchronize()
    # the same in float64, with autograd's gradients
    X, W1, W2, Q, O = (t.double().requires_grad_() for t in (x, w1, w2, wqkv, wo))
    shift = torch.tensor([[(g - h) % G for h in range(G)] for g in range(G)])

    def layer(t, w):
        return torch.einsum("oigh,nih->nog", w[:, :, shift], t)

    def norm(t, w):
        return t / torch.sqrt((t * t).mean((1, 2), keepdim=True) + eps) * w[None, :, None]

    angle = torch.cat([pos[:, i:i + 1].double() * torch.tensor([100.0 ** (-j / (Dh // 4)) for j in range(Dh // 4)],
                                                               dtype=torch.float64) for i in range(2)], 1)
    cos, sin = angle.cos()[:, None, :, None], angle.sin()[:, None, :, None]

    def turn(t):
        t = t.reshape(n, H, 2, Dh // 2, G)
        p, q = t[:, :, 0], t[:, :, 1]
        return torch.stack([p * cos - q * sin, q * cos + p * sin], 2).reshape(n, H, Dh * G)

    J = layer(norm(X, W1), Q)
    qq, kk, vv = turn(J[:, :C]), turn(J[:, C:2 * C]), J[:, 2 * C:].reshape(n, H, Dh * G)
    parts, at = [], 0
    for L in lens:
        s = torch.einsum("ihd,jhd->hij", qq[at:at + L], kk[at:at + L]) / math.sqrt(Dh * G)
        parts.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), vv[at:at + L]))
        at += L
    R2 = layer(torch.cat(parts).reshape(n, C, G), O) + X
    Z = norm(R2, W2)
    (Z * dz.double()).sum().backward()
    assert abs(float(torch.from_numpy(oracle.forward(x, wo, None)).sub(layer(x.double(), wo.double())).abs().max())) < 1e-9
    # normwise: each stage rounds its output (u) and its 16-bit operands (2 u); the longest way back
    # passes 12 stages, whose errors add at most linearly: 12 * 3 u = 0.14 in the worst case for
    # bf16; independent roundings add by root sum of squares, 6 u * sqrt(12) = 0.08 at three
    # times their expected size; fp32 stages: 1e-6 each
    tol = 6 * ref.unit(dtype) * math.sqrt(12) if dtype != torch.float32 else 12 * 2e-6
    for name, got, want in (("z", z, Z), ("dx", dx, X.grad), ("dw1", dw1, W1.grad), ("dw2", dw2, W2.grad),
                            ("dwqkv", dwqkv, Q.grad), ("dwo", dwo, O.grad)):
        err = float((got.double().cpu() - want.detach()).norm() / want.detach().norm())
        assert err <= tol, (name, err, tol)
    qkv_layer.close()
    out_layer.close()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("backward", [False, True])
def test_attention_wait_timeout_is_reported_and_the_gpu_stays_usable(D, backward, monkeypatch):
    """The load warp stops early (test hook, read on each call), so that the bounded waits of the other
    warps run out: the kernel returns, the status word tells, and the next call is right."""
    H, G, n = 2, 4, 700
    q, k, v, do = (_randn(n, H * D // G, G, seed=i, dtype=torch.bfloat16).to(DEV) for i in range(4))
    o, lse = eq.eqlin_attention_forward(q, k, v, heads=H)
    want = (o, lse) + eq.eqlin_attention_backward(do, q, k, v, o, lse, heads=H)
    assert eq.eqlin_attention_device_status() == eq.EQLIN_OK
    monkeypatch.setenv("EQLIN_WAIT_TIMEOUT_MS", "100")
    monkeypatch.setenv("EQLIN_TEST_STOP_AFTER", "3")
    if backward:
        eq.eqlin_attention_backward(do, q, k, v, o, lse, heads=H)
    else:
        eq.eqlin_attention_forward(q, k, v, heads=H)
    assert eq.eqlin_attention_device_status() == eq.EQLIN_ERR_TIMEOUT
    assert eq.eqlin_attention_device_status() == eq.EQLIN_OK         # reading the word clears it
    monkeypatch.delenv("EQLIN_TEST_STOP_AFTER")
    monkeypatch.delenv("EQLIN_WAIT_TIMEOUT_MS")
    got = eq.eqlin_attention_forward(q, k, v, heads=H)
    got += eq.eqlin_attention_backward(do, q, k, v, *got, heads=H)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert eq.eqlin_attention_device_status() == eq.EQLIN_OK


def test_device_status_follows_the_device():
    assert eq.eqlin_attention_device_status("cuda:0") == eq.EQLIN_OK
