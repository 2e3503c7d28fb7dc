"""Plain 64-bit forms of the dense attention calls and the bounds their tests use.

Bounds, derived from how the kernels compute (u = torch.finfo(t).eps / 2 of a 16-bit type t, the
half step of a rounding; A = softmax-weighted mean of |v| over the keys of a row):
- every weight is rounded once to the products' type and the output once to its own: (u_p + u_o) A;
- a logit is a sum of head_dim exact products in fp32, whose rounding is at most one step (2^-23)
  of the sum of magnitudes each time: delta = head_dim 2^-23 scale max_j sum_d |q_d k_jd|; the
  maximum, the multiplication by the scale and the exponential's argument round a few times more
  (4 steps of the largest logit, 2^-21 of it). Numerator and denominator each move by that factor;
- the sums over n keys run in fp32: n 2^-23 each, twice;
- the exponential and the division: 2^-21.
  |o - ref| <= (u_p + u_o + 2 (delta + 2^-21 max|logit|) + 2 n 2^-23 + 2^-21) A, and an absolute floor of
  half the smallest step of the output's type (its subnormals);
- lse: (delta + 2^-21 max|logit|) + n 2^-23 + 2^-20, plus its own rounding 2^-23 |lse|.
"""
from __future__ import annotations

import math

import torch


def attention(q, k, v, lo, hi, scale, valid=None):
    """q [n][d], k, v [t][d] in 64 bits, lo, hi [n]: rows i weigh keys [lo_i, hi_i) (and `valid` ones)."""
    x = (q @ k.T) * scale
    at = torch.arange(k.shape[0], device=q.device)
    hide = (at[None] < lo[:, None]) | (at[None] >= hi[:, None])
    if valid is not None:
        hide |= ~valid[None]
    mag = ((q.abs() @ k.abs().T) * scale).masked_fill(hide, 0).amax(-1) if k.shape[0] else torch.zeros_like(q[:, 0])
    x = x.masked_fill(hide, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None]).masked_fill(hide, 0)
    v = v.masked_fill(~(~hide).any(0)[:, None], 0)         # keys no row sees have no part, whatever they hold
    return p @ v, lse, p @ v.abs(), mag


def check(got, got_lse, want, lse, A, mag, n, dim, p_type, name=""):
    """got [rows][d] and got_lse [rows] of the kernel against the 64-bit row results."""
    u_o, u_p = torch.finfo(got.dtype).eps / 2, torch.finfo(p_type).eps / 2
    delta = dim * 2.0 ** -23 * mag + 2.0 ** -21 * mag
    rel = u_p + u_o + 2 * delta + 2 * n * 2.0 ** -23 + 2.0 ** -21
    floor = torch.finfo(got.dtype).smallest_normal * u_o * 2
    off = (got.double() - want).abs()
    bound = rel[:, None] * A + floor
    assert torch.isfinite(got).all(), f"{name}: not finite"
    worst = (off / bound).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: an output is {worst:.2f} times its bound off"
    if got_lse is not None:
        none = lse == -math.inf
        assert torch.equal(got_lse == -math.inf, none), f"{name}: empty rows"
        off = (got_lse.double() - lse)[~none].abs()
        bound = (delta + n * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -23 * lse.abs())[~none]
        worst = (off / bound).max().item() if off.numel() else 0.0
        assert worst <= 1.0, f"{name}: lse is {worst:.2f} times its bound off"
    return worst


def paged(batch, longest, heads, dim, page, dtype, seed, spare=2, scale=1.0):
    """Random pools and a shuffled table (unneeded entries -1) for `longest[b]` positions each."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in longest]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((batch, max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    k = (torch.randn(total, heads, page, dim, generator=g) * scale).to(dtype)
    v = torch.randn(total, heads, page, dim, generator=g).to(dtype)
    return k, v, table


def unpage(pool, table, b, n):
    """Positions 0 .. n - 1 of request b: [n][heads][dim] in 64 bits (pages outside the pool: zeros)."""
    page = pool.shape[2]
    at = torch.arange(n, device=pool.device)
    ids = table[b].long()[at // page] if n else at
    ok = (ids >= 0) & (ids < pool.shape[0])
    rows = pool.view(torch.uint8 if pool.element_size() == 1 else pool.dtype)[ids.clamp(0, pool.shape[0] - 1), :, at % page]
    rows = rows.view(pool.dtype).double() if pool.element_size() == 1 else rows.double()
    return rows.masked_fill(~ok[:, None, None], 0), ok
