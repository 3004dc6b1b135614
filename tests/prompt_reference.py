"""Plain 64-bit forms of the prompt side's operators and the error bounds the kernels are held to.

Bounds count roundings: to an element type at most eps / 2 relative (half the least subnormal near zero),
fp32 arithmetic 2^-24 relative an operation.
"""
from __future__ import annotations

import math

import torch

HALF_SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def within(got: torch.Tensor, want: torch.Tensor, bound: torch.Tensor, label: str = ""):
    """Every value of got within `bound` of want (fp64, same device); what is not finite in want is the same in got."""
    g = got.double()
    fine = want.isfinite()
    assert torch.equal(g.isfinite(), fine), f"{label}: non-finite values differ"
    assert torch.equal(g[~fine].nan_to_num(nan=7.0), want[~fine].nan_to_num(nan=7.0)), label
    over = ((g - want).abs() - bound)[fine]
    if over.numel():
        assert float(over.max()) <= 0, f"{label}: {int((over > 0).sum())} of {over.numel()} values past their bound, by up to {float(over.max()):.3g}"


def rope(x, positions, frequencies, interleaved, amplitude=1.0, inverse=False):
    """(rotated fp64, bound) of x [tokens, heads, head_dim]."""
    r = 2 * len(frequencies)
    f = torch.tensor(frequencies, dtype=torch.float64, device=x.device)
    angle = positions.double()[:, None] * f * (-1 if inverse else 1)
    cos, sin = (amplitude * angle.cos())[:, None], (amplitude * angle.sin())[:, None]
    y = x.double().clone()
    size = y.abs()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    # cos and sin are off by at most 2^-22 (the angle's fp32 rounding pi 2^-25, sincospi's few 2^-24,
    # the amplitude's), each product and the sum by 2^-24; the reference's own angle by position * f * 2^-52
    reach = abs(amplitude) * (a.abs() + b.abs()) * (2.0 ** -21 + (angle.abs() * 2.0 ** -51)[:, None])
    bound = torch.zeros_like(y)
    bound[..., first] = bound[..., second] = reach
    rotated = torch.zeros(y.shape[-1], dtype=torch.bool, device=x.device)
    rotated[:r] = True
    bound = torch.where(rotated, bound + half_step(x.dtype) * (y.abs() + bound) + HALF_SUBNORMAL[x.dtype], 0.0 * size)
    return y, bound


def rmsnorm(x, f, gamma, eps):
    """(h in x's type, y fp64) of the rows; statistics of the rounded h."""
    h = x if f is None else (x.double() + f.double()).float().to(x.dtype)  # the fp64 sum is exact
    y = h.double()
    return h, y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()


# fp32 sum of squares (chains of up to 64 + 12 additions), mean, root, two products: below 100 roundings
RMSNORM_RELATIVE = 100 * 2.0 ** -24


def attention(q, k, v, starts_q, starts_k, lengths_k=None, causal=True, scale=None):
    """fp64 (o, lse, bound of o, bound of lse) of packed sequences; indices are lists.  Rows outside every
    sequence: NaN with an infinite bound."""
    heads, kv, d = q.shape[1], k.shape[1], q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64, device=q.device)
    o_bound, lse_bound = torch.full_like(o, math.inf), torch.full_like(lse, math.inf)
    e = half_step(q.dtype)
    for s in range(len(starts_q) - 1):
        a, b, c = starts_q[s], starts_q[s + 1], starts_k[s]
        n = starts_k[s + 1] - c if lengths_k is None else lengths_k[s]
        qs = q[a:b].double().transpose(0, 1)                                            # [heads, lq, d]
        ks = k[c:c + n].double().repeat_interleave(heads // kv, 1).transpose(0, 1)     # [heads, lk, d]
        vs = v[c:c + n].double().repeat_interleave(heads // kv, 1).transpose(0, 1)
        seen = torch.ones(b - a, n, dtype=torch.bool, device=q.device)
        if causal:
            seen = seen.tril(n - (b - a))
        logits = (qs @ ks.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
        norm = torch.logsumexp(logits, 2) if n else torch.full(qs.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        p = (logits - norm[..., None].nan_to_num(neginf=0.0)).exp()
        p = p.masked_fill(~seen, 0.0)
        # what a query does not attend has no influence: non-finite values count for their own queries only
        fine = torch.where(vs.isfinite(), vs, 0.0)
        out = p @ fine
        for j in (~vs.isfinite()).any(0).any(1).nonzero().flatten().tolist() if n else []:
            bad = torch.where(vs[:, j].isfinite(), 0.0, vs[:, j])
            out = out + torch.where(seen[:, j][None, :, None], bad[:, None, :], 0.0)
        # a logit is off by at most 2 (d + 8) 2^-24 of the sum of its products' sizes, which moves every weight
        # by that relative amount, in numerator and denominator; P is rounded once (fp16: to 2^-25 where it is
        # subnormal, against a row sum of at least one), o once
        size = (qs.abs() @ ks.abs().transpose(1, 2) * scale).masked_fill(~seen, 0.0).amax(2) if n else torch.zeros_like(norm)
        shift = 2 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20
        weighed = p @ fine.abs()
        most = fine.abs().amax(1, keepdim=True) if n else torch.zeros_like(out[:, :1])
        spread = weighed * (e + 2 * shift[..., None]) + n * HALF_SUBNORMAL[q.dtype] * most
        o[a:b], lse[a:b] = out.transpose(0, 1), norm.transpose(0, 1)
        o_bound[a:b] = (spread + e * (out.abs() + spread)).transpose(0, 1) + HALF_SUBNORMAL[q.dtype]
        lse_bound[a:b] = (shift + 2.0 ** -21 * norm.abs().nan_to_num(posinf=0.0)).transpose(0, 1)
    return o, lse, o_bound, lse_bound
