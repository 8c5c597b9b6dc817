"""The streaming attention calls in 64 bits on the CPU, straight from their formulas, and the
error each call's arithmetic allows.  Plain loops over sequences and heads.

Error bounds (u = half a step of the tensors' type, relative: bf16 2^-8, fp16 2^-11):
  * scores: a product of d terms summed in fp32 by the tensor cores, at most d steps of
    2^-23 of sum |q k|; times scale this is the absolute error `dx` of an exponent, so every
    probability is off by about dx relative, and lse by dx;
  * probabilities are rounded to the tensors' type before they meet V: u relative, or in
    fp16 half its smallest step (2^-25) where that is more, with the row's sum >= 1;
  * sums in fp32 and the exponential add less than 2^-17 relative;
  * the result is rounded once: u relative to it, or in fp16 half its smallest step where that
    is more: below 2^-14 fp16 values are 2^-24 apart, so rounding moves one by up to 2^-25,
    which u times a value below 2^-14 does not cover.
"""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ARITH = 2.0 ** -17


def kept(mask, nq, nk):
    """[nq, nk] truth values of WindowMask `mask` for a sequence of nq queries and nk keys."""
    p = torch.arange(nq)[:, None] + (nk - nq)
    j = torch.arange(nk)[None, :]
    bp, bj = torch.floor_divide(p, mask.block), torch.floor_divide(j, mask.block)
    keep = torch.ones(nq, nk, dtype=torch.bool)
    if mask.window >= 0:
        keep = ((bp - bj).abs() <= mask.window) | (j < mask.sinks)
    return keep & (bj <= bp) if mask.causal else keep


def attention(q, k, v, mask, scale):
    """One sequence and head: q [nq, d], k and v [nk, d].  Returns o, lse (64 bits) and the
    bounds of both for results in q's type."""
    u, d = HALF_STEP[q.dtype], q.shape[1]
    q64, k64, v64 = q.double(), k.double(), v.double()
    keep = kept(mask, q.shape[0], k.shape[0])
    x = torch.where(keep, scale * q64 @ k64.T, torch.tensor(-math.inf, dtype=torch.float64))
    lse = torch.logsumexp(x, 1) if k.shape[0] else torch.full((q.shape[0],), -math.inf).double()
    p = torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None])
    p = torch.where(keep, p, torch.zeros_like(p))
    v0 = torch.where(keep.any(0)[:, None], v64, torch.zeros_like(v64)) if q.shape[0] else v64
    o = p @ v0
    dx = (torch.where(keep, scale * q64.abs() @ k64.abs().T, torch.zeros_like(x)).amax(1)
          if k.shape[0] else torch.zeros(q.shape[0]).double()) * d * 2.0 ** -23
    o_tol = (u + 2 * dx + ARITH)[:, None] * (p @ v0.abs()) + u * o.abs()
    if q.dtype == torch.float16:
        o_tol = o_tol + 2.0 ** -25 * (keep.double() @ v0.abs()) + 2.0 ** -25
    return o, lse, o_tol, dx + 2.0 ** -19 * (1 + lse.abs().nan_to_num(posinf=0.0))


def gradients(q, k, v, do, mask, scale):
    """One sequence and query head: dq, dk, dv in 64 bits with bounds for a call that is given
    o rounded to the tensors' type and lse in fp32."""
    u, d = HALF_STEP[q.dtype], q.shape[1]
    o, lse, o_tol, lse_tol = attention(q, k, v, mask, scale)
    q64, k64, v64, g64 = q.double(), k.double(), v.double(), do.double()
    keep = kept(mask, q.shape[0], k.shape[0])
    zero = torch.zeros((), dtype=torch.float64)
    x = scale * q64 @ k64.T
    p = torch.where(keep, torch.exp(x - torch.where(lse.isinf(), zero, lse)[:, None]), zero)
    dp = torch.where(keep, g64 @ v64.T, zero)
    delta = (g64 * o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    dq, dk, dv = scale * ds @ k64, scale * ds.T @ q64, p.T @ g64
    # P: its exponent's error and fp32 lse; dS: P's, dP's sum of d terms, delta from a rounded
    # o, then one rounding to the tensors' type (fp16: or half its smallest step)
    dx = (scale * q64.abs() @ k64.abs().T) * d * 2.0 ** -23 + lse_tol[:, None]
    p_rel = 2 * dx + ARITH
    dp_abs = (g64.abs() @ v64.abs().T) * d * 2.0 ** -23
    delta_abs = (g64.abs() * (u * o.abs() + o_tol)).sum(1, keepdim=True) + \
        2.0 ** -20 * (g64.abs() * o.abs()).sum(1, keepdim=True)
    tiny = 2.0 ** -25 if q.dtype == torch.float16 else 0.0
    ds_err = torch.where(keep, p * (dp_abs + delta_abs) + (p_rel + u + ARITH) * ds.abs() + tiny,
                         zero)
    p_err = torch.where(keep, p * (u + p_rel) + tiny, zero)
    return (dq, dk, dv,
            tiny + scale * ds_err @ k64.abs() + (u + ARITH) * dq.abs() + ARITH * scale * ds.abs() @ k64.abs(),
            tiny + scale * ds_err.T @ q64.abs() + (u + ARITH) * dk.abs() + ARITH * scale * ds.abs().T @ q64.abs(),
            tiny + p_err.T @ g64.abs() + (u + ARITH) * dv.abs() + ARITH * p.T @ g64.abs())


def angles(spec, theta, place):
    """[tokens, pairs] angles of the tokens' places in the grid, in 64 bits."""
    S = spec.grid_h * spec.grid_w
    axes = (place // S, place % S // spec.grid_w, place % spec.grid_w)
    return torch.cat([x.double()[:, None] *
                      theta ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
                      for x, n in zip(axes, spec.pairs)], 1)


def rotate(x, spec, theta, place, inverse=False):
    """x [tokens, d] turned at its places in 64 bits, and the bound of a rounded fp32 result:
    cos and sin off by half a step of fp32 each, three fp32 operations, one rounding."""
    u = HALF_STEP[x.dtype]
    a = angles(spec, theta, place)
    c, s = a.cos(), -a.sin() if inverse else a.sin()
    n = a.shape[1]
    i0 = 2 * torch.arange(n) if spec.interleaved else torch.arange(n)
    i1 = i0 + 1 if spec.interleaved else i0 + n
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    x0, x1 = x.double()[:, i0], x.double()[:, i1]
    y[:, i0], y[:, i1] = x0 * c - x1 * s, x1 * c + x0 * s
    size[:, i0] = size[:, i1] = x0.abs() + x1.abs()
    tol = u * y.abs() + 4 * 2.0 ** -24 * size
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half its smallest step
    return y, tol


def within(got, want, tol, what=""):
    got, want = got.double().cpu(), want.double()
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~same & ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values off, the worst by "
                           f"{((got - want).abs() / tol.clamp(min=1e-300))[bad].max():.3g} times "
                           f"the bound")
