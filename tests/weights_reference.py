"""Attention and attention weights from their definitions, in 64 bits, with the
bounds that the kernels' roundings allow.

Bounds.  A logit in log2 units is a sum of D products of 16-bit values (exact in
32 bits), each addition off by at most 2^-23 of the partial sums (the tensor
cores may truncate), then one product with the scale and one subtraction: off
by at most dz = D 2^-23 scale sum_i |q_i k_i| + 4 * 2^-24 |z| in natural units
(twice the largest |z| covers z and the reference or lse).  The same holds for
the lse.  2^x and log2 are off by 2^-22 relative (absolute).  So exp(z - lse)
is off by rel = 2 dz + 2^-20 relative, and sums of such terms by as much plus
2^-24 a term added one after another (counted by the caller).
"""
from __future__ import annotations

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative


def attend(q, k, v, scale, causal_from=None):
    """q [R, D], k/v [n, D] of one head (16-bit); row r sees keys <= causal_from + r
    (all, if None).  Returns p [R, n], out [R, D], lse [R], rel [R] (bound above)
    and pv [R, D] = sum p |v|."""
    q, k, v = q.double(), k.double(), v.double()
    R, n = q.shape[0], k.shape[0]
    mask = torch.zeros(R, n, dtype=torch.bool, device=q.device)
    if causal_from is not None:
        at = torch.arange(n, device=q.device)
        mask = at[None] > torch.arange(R, device=q.device)[:, None] + causal_from
    z = (q @ k.T * scale).masked_fill(mask, -torch.inf)
    size = (q.abs() @ k.abs().T * abs(scale)).masked_fill(mask, 0)
    big = z.masked_fill(mask, 0).abs().amax(1)
    rel = 2 * (q.shape[1] * 2.0 ** -23 * size.amax(1) + 8 * 2.0 ** -24 * big) + 2.0 ** -20
    p = torch.softmax(z, 1)
    v0 = v.masked_fill(~torch.isfinite(v), 0)
    return p, p @ v0, torch.logsumexp(z, 1), rel, p @ v0.abs()


def out_bound(out, pv, rel, n, vmax, dtype, p_half):
    """Bound of the rounded output: P enters P V rounded by p_half relative (and,
    in fp16, by 2^-25 where it is subnormal, against a sum of at least 1), p and l
    are off by rel each, the sums add 2^-23 a key, and the result is rounded
    once (2^-25 where it is a subnormal fp16)."""
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return (HALF[dtype] * out.abs() + (p_half + 2 * rel[:, None] + n * 2.0 ** -23) * pv +
            n * 2.0 ** -25 * vmax * (dtype == torch.float16) + sub + 1e-30) * (1 + HALF[dtype])
