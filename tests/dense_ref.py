"""The dense attention operators and their cache written out in 64 bits, one
sequence and one head at a time, and how far a kernel's results may be from
them.

Tolerances.  Let p_j be a row's softmax weights, S = sum_j p_j |v_j| / den (per
output element) and A = scale * max_j sum_d |q_d k_jd|.  A kernel makes these
roundings:
* a score is an f32 sum of hd exact products: at most hd additions of f32, each
  off by at most 2^-23 of the running magnitude (truncating adders included), so
  |dt| <= hd 2^-23 A; one or two f32 products for the scales add 2^-23 A.
  A weight is off by a factor e^{dt}, plus the exponential's own 2^-21;
* a weight is rounded to bf16 for the second product: 2^-8 relative;
* the sum over n keys adds n f32 terms (and the rescaling products): n 2^-23 of
  the sum of magnitudes; the same holds for the denominator;
* the output is rounded to bf16: 2^-8 relative.
* on an e4m3 cache the weights p_j vs_j are rounded to f16 instead, 2^-11
  relative, but not finer than 2^-25 of their reference, which is at most
  p_max vs_max: that adds 2^-25 p_max vs_max sum_j |code_j|.
* what lies below 2^-126 may be taken for 0 (a weight, the factor that a sink
  leaves, an output): 2^-126 (1 + sum_j |v_j|).
All of it scales with S except the last three: |o - exact| <= 2^-8 |exact| +
S (2^-8 + 2 (hd + 4) 2^-23 A + 2^-20 + 2 n 2^-23) (1 + 2^-7) (+ the f16 and the
smallest-number terms), the last factor for the products of the small terms.
"""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def quantise(x):
    """x [..., hd] (bf16) to (codes as float8, scales f32): the definition.  The
    quotients are taken in 64 bits and rounded to f32, which gives the correctly
    rounded f32 quotients (53 >= 2 * 24 + 2 bits)."""
    x = x.double()
    s = (x.abs().amax(-1).clamp_min(E4M3_MAX * 2.0 ** -126) / E4M3_MAX).float()
    bad = ~torch.isfinite(x).all(-1)
    y = torch.where(bad[..., None], torch.zeros_like(x), x / s.double()[..., None]).float()
    return y.to(torch.float8_e4m3fn), torch.where(bad, torch.full_like(s, math.nan), s)


def values(codes, scales):
    """A cache's values in 64 bits."""
    return codes.double() if scales is None else codes.double() * scales.double()[..., None]


def attend(q, k, v, visible, scale, sink, vs=None):
    """q [n, nh, hd], k, v [L, kvh, hd], visible [n, L]: (o, lse, tolerance of o,
    tolerance of lse), 64 bits.  v rows that a query does not see do not count,
    whatever they hold.  vs [L, kvh]: the scales of v on an e4m3 cache."""
    n, nh, hd = q.shape
    L, kvh = k.shape[:2]
    per = nh // kvh
    q, k, v = q.double(), k.double(), v.double()
    o = torch.zeros(n, nh, hd, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(o)
    lse = torch.full((n, nh), -math.inf, dtype=torch.float64, device=q.device)
    ltol = torch.zeros_like(lse)
    for h in range(nh):
        kh, vh = k[:, h // per], v[:, h // per]
        vh = torch.where(visible.any(0)[:, None], vh, 0.0)
        s = torch.where(visible, q[:, h] @ kh.T * scale, -math.inf)
        A = torch.where(visible, q[:, h].abs() @ kh.abs().T * scale, 0.0)
        A = A.amax(1) if L else torch.zeros(n, dtype=torch.float64, device=q.device)
        t = s if sink is None else torch.cat([s, sink[h].double().expand(n, 1)], 1)
        if t.shape[1] == 0:
            continue
        lse[:, h] = torch.logsumexp(t, 1)
        p = torch.exp(s - torch.where(lse[:, h] == -math.inf, 0.0, lse[:, h])[:, None])
        o[:, h] = p @ vh
        dt = (hd + 4) * 2.0 ** -23 * A + 2.0 ** -21
        rel = 2.0 ** -8 + 2 * dt + 2 * L * 2.0 ** -23
        tol[:, h] = 2.0 ** -8 * o[:, h].abs() + (p @ vh.abs()) * rel[:, None] * (1 + 2.0 ** -7)
        tol[:, h] += 2.0 ** -126 * (1 + visible.double() @ vh.abs())
        if vs is not None and L:
            x = torch.where(visible.any(0), vs[:, h // per].double(), 0.0)
            code = vh.abs() / x.clamp_min(2.0 ** -126)[:, None]
            tol[:, h] += 2.0 ** -25 * (p.amax(1) * x.max())[:, None] * (visible.double() @ code)
        ltol[:, h] = (dt + L * 2.0 ** -23) * (1 + 2.0 ** -7) + 2.0 ** -21 * (
            1 + torch.where(torch.isfinite(lse[:, h]), lse[:, h].abs(), 0.0))
    return o, lse, tol, ltol


def prompt_visible(n, m, window, device):
    """[n, m]: query i stands at i + m - n."""
    p = torch.arange(n, device=device)[:, None] + (m - n)
    j = torch.arange(m, device=device)
    return (j <= p) & ((j > p - window) if window else True)


def tree_visible(n, length, bits, window, device):
    """[n, length] for n drafted tokens, `bits` their mask words as Python
    integers (None: a chain)."""
    pre = length - n
    vis = torch.zeros(n, length, dtype=torch.bool)
    for t in range(n):
        seen = [u for u in range(n) if (u <= t if bits is None else bits[t] >> u & 1)]
        d = t if bits is None else len(seen) - 1
        lo = pre + d - window if window else -1
        vis[t, max(0, lo + 1):pre] = True
        for u in seen:
            vis[t, pre + u] = True
    return vis.to(device)


def close(got_o, got_lse, o, lse, tol, ltol):
    """Asserts both outputs within their tolerances (and equal where infinite)."""
    e = (got_o.double() - o).abs()
    assert bool((e <= tol).all()), ("o", float((e / tol.clamp_min(1e-300)).max()), float(e.max()))
    inf = torch.isinf(lse)
    assert bool((got_lse.double()[inf] == lse[inf]).all()), "lse of rows that see nothing"
    e = (got_lse.double() - lse).abs()[~inf]
    assert bool((e <= ltol[~inf]).all()), ("lse", float((e / ltol[~inf]).max()))
