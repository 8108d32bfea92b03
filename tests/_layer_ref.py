"""Plain 64-bit forms of conv_*, ssm_* and spec_verify, token by token, with the
error bounds that the GPU tests hold the kernels to.

Bounds, from the roundings that fp32 arithmetic makes (u = 2^-24 is half a step):
  * conv: W products and sums, each off by u of the sum of magnitudes M at most:
    (W + 2) u M before the activation, whose slope is below 1.1.
  * silu: e^-y by the SFU is off by 2 + 1.173 |y| steps of 2^-23, the quotient by
    2 more: (6 + 1.2 |y|) 2^-23 of the result.
  * softplus(v): v = dt + bias is off by u |v|; e^-|v| by 4 u + 1.5 |v| u, the
    logarithm by 8 u: (2 |v| + 16) u =: es, relative (the slope over the value is
    at most 1).
  * decay e^(s A): SFU 4 u, its argument |s A| (es + 2 u): ea = 4 u + |s A| (es + 2 u).
  * state: E <- a E + |a h| ea + |s x B| (es + 3 u) + 2 u |h|: the bound obeys the
    recurrence itself, so it covers any regrouping of the tokens whose decays are
    products of the same factors.
  * y: sum |C| E + (N + 2) u sum |C h| + 2 u |D x|, times silu(z) and its own bound.
  * the last rounding: u for fp32, 2^-8 (half a step) for bf16, relative.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def rounded(a, dtype):
    """A 64-bit array as a tensor type holds it."""
    return torch.from_numpy(np.asarray(a)).to(dtype).double().numpy()


def silu(y):
    with np.errstate(over="ignore"):
        return y / (1 + np.exp(-y))


def _bound_silu(y, err):
    return 1.1 * err + np.abs(silu(y)) * (6 + 1.2 * np.abs(y)) * 2.0 ** -23


def conv_tokens(x, weight, bias, seed, act):
    """x [T, C] after seed [W - 1, C]: (out, bound, inputs [W - 1 + T, C])."""
    W = weight.shape[1]
    row = np.concatenate([seed, x], 0)
    T = x.shape[0]
    b = np.zeros(x.shape[1]) if bias is None else bias
    y = np.zeros_like(x)
    mag = np.zeros_like(x)
    for t in range(T):
        win = row[t:t + W]
        y[t] = b + (win * weight.T).sum(0)
        mag[t] = np.abs(b) + np.abs(win * weight.T).sum(0)
    err = (W + 2) * U * mag
    return (silu(y), _bound_silu(y, err), row) if act else (y, err, row)


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def ssm_tokens(x, dt, A, B, C, seed, *, D=None, z=None, dt_bias=None, soft=False, seed_err=None):
    """x, dt, z [T, Dch], B, C [T, G, N] after seed [Dch, N]:
    (out, bound, states [T, Dch, N], their bounds)."""
    T, Dch = x.shape
    G = B.shape[1]
    group = np.arange(Dch) // (Dch // G)
    h = seed.copy()
    E = np.zeros_like(h) if seed_err is None else seed_err
    out, bound = np.zeros_like(x), np.zeros_like(x)
    hs, Es = np.zeros((T,) + h.shape), np.zeros((T,) + h.shape)
    N = h.shape[1]
    for t in range(T):
        if soft:
            v = dt[t] + (0 if dt_bias is None else dt_bias)
            s, es = softplus(v), (2 * np.abs(v) + 16) * U
        else:
            s, es = dt[t], np.zeros(Dch)
        s, es = s[:, None], es[:, None]
        a = np.exp(s * A)
        ea = 4 * U + np.abs(s * A) * (es + 2 * U)
        inp = s * x[t][:, None] * B[t][group]
        E = a * E + np.abs(a * h) * ea + np.abs(inp) * (es + 3 * U)
        h = a * h + inp
        E = E + 2 * U * np.abs(h)
        c = C[t][group]
        y = (c * h).sum(1)
        e = (np.abs(c) * E).sum(1) + (N + 2) * U * np.abs(c * h).sum(1)
        if D is not None:
            y = y + D * x[t]
            e = e + 2 * U * np.abs(D * x[t]) + U * np.abs(y)
        if z is not None:
            gz = silu(z[t])
            e = e * np.abs(gz) * 1.001 + np.abs(y) * (_bound_silu(z[t], 0) + U * np.abs(gz))
            y = y * gz
        out[t], bound[t], hs[t], Es[t] = y, e, h, E
    return out, bound, hs, Es


def assert_within(gpu, ref, bound, what=""):
    """|gpu - ref| <= bound plus the rounding of gpu's type."""
    g = f64(gpu)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    assert np.isfinite(g).all(), f"{what}: not finite"
    half = HALF[gpu.dtype]
    tol = bound * (1 + half) + np.abs(ref) * half + 1e-37
    bad = np.abs(g - ref) > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside the bound, the worst "
                           f"{float((np.abs(g - ref) / tol).max()):.3g} times it")


def verify(draft, target, u_accept, u_sample, probs=None, num_draft=None):
    """spec_verify by exact sums (math.fsum).  draft [B][T-1] ints, target [B, T, V]
    and probs [B, T-1, V] 64-bit arrays, all as held.  Returns (accepted, tokens)."""
    B, T, V = target.shape
    acc, toks = [], []
    for b in range(B):
        k = T - 1 if num_draft is None else min(max(int(num_draft[b]), 0), T - 1)
        n = 0
        while n < k:
            d = int(draft[b][n])
            if not 0 <= d < V:
                break
            q = 1.0 if probs is None else probs[b, n, d]
            if not u_accept[b, n] * q < target[b, n, d]:
                break
            n += 1

        def clean(w):
            return np.where((w > 0) & np.isfinite(w), w, 0.0)

        p = target[b, n]
        w = clean(p)
        if n < k:
            if probs is not None:
                with np.errstate(invalid="ignore"):
                    r = clean(p - probs[b, n])
            else:
                r = w.copy()
                if 0 <= int(draft[b][n]) < V:
                    r[int(draft[b][n])] = 0
            w = r if r.sum() > 0 else w
        tok = -1
        if w.sum() > 0:
            thr = float(u_sample[b]) * math.fsum(w)
            run = np.cumsum(w.astype(np.longdouble))
            over = np.nonzero((w > 0) & (run > thr))[0]
            tok = int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])
        acc.append(n + 1)
        toks.append([int(draft[b][i]) for i in range(n)] + [tok] + [-1] * (T - 1 - n))
    return np.array(acc), np.array(toks)
