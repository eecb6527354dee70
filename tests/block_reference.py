"""Float64 definitions of the transformer-block operators, and how far a kernel's outputs may be
from them.

Error bounds.  u = finfo(T).eps / 2 is the largest relative error of one rounding to the I/O type T.
Every bound is a sum of absolute values of the terms that were rounded, computed in float64 beside
the value itself:
  - an output rounded once from fp32: u |y|;
  - fp32 arithmetic: E = 2^-20 relative to the sum of the absolute values of the terms (sums of up to
    a few hundred products of 2^-24 each, approximate exponentials of 2^-22);
  - attention's fp32 products may each be three products of tf32 (11 significant bits): a = h + l with h
    rounded to nearest, |l| <= 2^-11 |a|; l, cut to 11 bits, loses less than 2^-10 |l| <= 2^-21 |a|.
    a b - (h h' + h l' + l h') is l l' (2^-22 |a b|) and the two cuts (2^-21 |a b| each): 2.5 * 2^-21 |a b|.  Their sums start from zero every
    32 terms, as the tensor cores' additions are cut and not rounded;
  - attention's 16-bit forward may take its weights from a polynomial for 2^x of relative error 2^-18.5 (a
    fit of degree 4 to 2^f on [-1/2, 1/2]): the normaliser and the weights each move by that, which in o
    adds up to twice as much per term and in lse, the normaliser's logarithm, to once as much;
  - attention weights and ds, rounded to T before their products: u per term, plus half of the
    smallest subnormal of T where T is fp16.
"""
from __future__ import annotations

import math

import torch

E = 2.0 ** -20


def unit(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny(dtype: torch.dtype) -> float:
    """Half of the smallest subnormal: the absolute error of a rounding near zero."""
    return {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}.get(dtype, 2.0 ** -150)


def within(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor, what: str) -> None:
    got, want, bound = got.double().cpu(), want.double().cpu(), bound.double().cpu()
    assert got.shape == want.shape, what
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: other values are finite"
    assert torch.equal(got[~fine].isnan(), want[~fine].isnan()), what
    off = (got - want).abs()[fine]
    over = off > bound[fine]
    if over.any():
        k = int((off / bound[fine].clamp_min(1e-300)).argmax())
        raise AssertionError(f"{what}: {int(over.sum())} of {over.numel()} values too far off; worst "
                             f"{got[fine][k]:.9g} for {want[fine][k]:.9g}, bound {bound[fine][k]:.3g}")


def offsets(lens, device=None) -> torch.Tensor:
    t = torch.zeros(len(lens) + 1, dtype=torch.int64)
    t[1:] = torch.tensor(list(lens), dtype=torch.int64).cumsum(0)
    return t.to(torch.int32).to(device) if device else t.to(torch.int32)


def attention(q, k, v, do, q_lens, k_lens, heads, kv_heads, causal, scale=None, chained=False, o_err=0.0):
    """{"o", "lse", "dq", "dk", "dv"} in float64 and {name: bound} for kernels of q's dtype, for
    q [Nq, H Dh, G], k and v [Nk, Hk Dh, G]; the gradients are those for o rounded to q's dtype.
    chained: the gradients were given the kernel's own o and lse.  Then o is off by up to its bound, which
    moves delta_i = do_i . o_i by up to sum_d |do_id| bound(o_id), and lse by up to its bound, which
    moves every weight by that much relative to itself.  o_err: what each element of the o given to them is off
    by beside its rounding."""
    T, u, t0 = q.dtype, unit(q.dtype), tiny(q.dtype)
    if T == torch.float32:
        p_round, ds_round = 0.0, 0.0          # fp32 keeps them unrounded
    else:
        p_round = ds_round = u
    M = E + 2.5 * 2.0 ** -21 if T == torch.float32 else E      # products
    X = 0.0 if T == torch.float32 else 2.0 ** -18.5            # the forward's weights
    H, Hk, G = heads, kv_heads, q.shape[2]
    D = q.shape[1] * G // H
    scale = 1 / math.sqrt(D) if scale is None else scale
    Q, K, V, dO = (t.double().reshape(len(t), t.shape[1] * G // D, D) for t in (q, k, v, do))
    out = {"o": torch.zeros_like(Q), "lse": torch.full((H, len(Q)), -math.inf, dtype=torch.float64),
           "dq": torch.zeros_like(Q), "dk": torch.zeros_like(K), "dv": torch.zeros_like(V)}
    bound = {n: torch.zeros_like(x) for n, x in out.items()}
    q0 = k0 = 0
    for a, b in zip(q_lens, k_lens):
        i, j = torch.arange(a), torch.arange(b)
        hidden = (j[None, :] > i[:, None] + (b - a)) if causal else torch.zeros(a, b, dtype=torch.bool)
        for h in range(H):
            g = h // (H // Hk)
            x, y, z, w = Q[q0:q0 + a, h], K[k0:k0 + b, g], V[k0:k0 + b, g], dO[q0:q0 + a, h]
            s = scale * (x @ y.T)
            s_err = M * scale * (x.abs() @ y.abs().T) + E * s.abs()
            s = s.masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(s, 1) if b else torch.full((a,), -math.inf, dtype=torch.float64)
            p = torch.exp(s - torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[:, None])
            lse_err = (p * s_err).sum(1) + E * (1 + lse.abs()) + X
            p_err = p * (s_err + torch.where(lse == -math.inf, torch.zeros_like(lse), lse_err)[:, None]
                         + E + p_round) + t0 * (p > 0)
            # a row whose weights underflow far below its largest keeps an absolute error only
            o = p @ z
            rows, keys = slice(q0, q0 + a), slice(k0, k0 + b)
            out["o"][rows, h], out["lse"][h, rows] = o, lse
            bound["o"][rows, h] = p_err @ z.abs() + (M + X) * (p @ z.abs()) + u * o.abs() + t0
            bound["lse"][h, rows] = lse_err
            ot = o.to(T).double()
            dp, delta = w @ z.T, (w * ot).sum(1)
            dp_err = M * (w.abs() @ z.abs().T)
            delta_err = E * (w.abs() * ot.abs()).sum(1) + o_err * w.abs().sum(1)
            ds = p * (dp - delta[:, None])
            p32 = p_err - p * p_round - t0 * (p > 0)             # ds is formed from unrounded weights
            if chained:
                delta_err = delta_err + (w.abs() * bound["o"][rows, h]).sum(1)
                off = p * torch.where(lse == -math.inf, torch.zeros_like(lse), lse_err)[:, None]
                p32, p_err = p32 + off, p_err + off
            ds_err = p32 * (dp - delta[:, None]).abs() + p * (dp_err + delta_err[:, None]) \
                + E * p * (dp.abs() + delta.abs()[:, None])
            ds_err = ds_err + ds_round * (ds.abs() + ds_err) + t0 * (p > 0)
            dq, dk, dv = scale * ds @ y, scale * ds.T @ x, p.T @ w
            out["dq"][rows, h] = dq
            out["dk"][keys, g] += dk
            out["dv"][keys, g] += dv
            bound["dq"][rows, h] = scale * (ds_err @ y.abs() + M * ds.abs() @ y.abs()) + u * dq.abs() + t0
            bound["dk"][keys, g] += scale * (ds_err.T @ x.abs() + M * ds.abs().T @ x.abs()) + t0
            bound["dv"][keys, g] += p_err.T @ w.abs() + M * (p.T @ w.abs()) + t0
        q0, k0 = q0 + a, k0 + b
    for n in ("dk", "dv"):
        bound[n] += u * (out[n].abs() + bound[n])
    shapes = {"o": q.shape, "dq": q.shape, "dk": k.shape, "dv": v.shape}
    return ({n: x.reshape(shapes.get(n, x.shape)) for n, x in out.items()},
            {n: x.reshape(shapes.get(n, x.shape)) for n, x in bound.items()})


def add_rmsnorm(x, residual, weight, eps):
    """(y, r, rstd) in float64."""
    r = x.double() + (0 if residual is None else residual.double())
    rstd = 1 / torch.sqrt((r * r).mean((1, 2), keepdim=True) + eps)
    w = torch.ones(x.shape[1], dtype=torch.float64) if weight is None else weight.double()
    return r * rstd * w[None, :, None], r, rstd


def rmsnorm_backward(dy, r, weight, dsum, eps):
    """(dx, dweight, bound of dx, bound of dweight) in float64 from the stored sum r."""
    u, T = unit(r.dtype), r.dtype
    _, r64, rstd = add_rmsnorm(r, None, weight, eps)
    w = (torch.ones(r.shape[1], dtype=torch.float64) if weight is None else weight.double())[None, :, None]
    dy64, un = dy.double(), r64 * rstd
    inner = (w * dy64 * un).mean((1, 2), keepdim=True)
    dx = rstd * (w * dy64 - un * inner)
    size = rstd * ((w * dy64).abs() + un.abs() * (w * dy64 * un).abs().mean((1, 2), keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    dweight = (dy64 * un).sum((0, 2))
    return dx, dweight, u * dx.abs() + E * size + tiny(T), E * (dy64 * un).abs().sum((0, 2)) + 1e-40


def rope(x, positions, heads, sections, base, inverse=False):
    """(y, bound) in float64: y by complex multiplication."""
    N, C, G = x.shape
    Dh = C // heads
    angle = torch.cat([positions[:, a:a + 1].double() * torch.tensor([base ** (-j / n) for j in range(n)],
                                                                     dtype=torch.float64)
                       for a, n in enumerate(sections)], 1)
    if inverse:
        angle = -angle
    v = x.double().reshape(N, heads, 2, Dh // 2, G)
    z = torch.complex(v[:, :, 0], v[:, :, 1]) * torch.polar(torch.ones_like(angle), angle)[:, None, :, None]
    y = torch.stack([z.real, z.imag], 2).reshape(N, C, G)
    size = (v[:, :, 0].abs() + v[:, :, 1].abs())[:, :, None].expand(-1, -1, 2, -1, -1).reshape(N, C, G)
    return y, unit(x.dtype) * y.abs() + E * size + tiny(x.dtype)
