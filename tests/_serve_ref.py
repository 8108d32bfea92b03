"""Plain 64-bit forms of kv_append, attn_decode and sample_tokens, row by row, with the
error bounds that the GPU tests hold the kernels to.

Bounds, from the roundings that the arithmetic makes (u = 2^-24 is half a step of fp32):
  * rotation: the angle is good to 2^-33 turns (7.4e-10 rad), cosine and sine to 2 u each,
    times rope_scale u more, two products and a sum 2 u: 6 u m (|x| + |y|) per component.
  * an e4m3 code: half a step, 2^-4 of the value or 2^-10 of the scale (the least step is
    2^-9), of the value that is off as above.  Values that are not rotated give the very
    codes.
  * scores, base 2: D products summed in fp32 by the tensor cores, each sum off by a step (2 u)
    of the magnitudes' sum A at most: D 2 u A, and 4 roundings of the result and of log2 of
    the values' scale: es = (2 D + 8) u A + 8 u |e|; the exponential's 2^-22 and es ln 2 are
    relative errors of a weight: ew.
  * weights: fp16 rounds by 2^-11, and below 2^-14 by 2^-25 of a unit that is at most the
    greatest weight; two bf16 terms leave 2^-16 (and 2^-24 at the least).  With S = sum w |V| /
    sum w and n tokens: (ew + 2^-11) S + n 2^-25 max |V|, twice ew for the weights' sum,
    and the products' sums n 2 u S.
  * lse: ew + n 2 u, absolute, and 4 u of itself.
  * the last rounding: u for fp32, 2^-8 (half a step) for bf16, relative.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
E_LO, E_HI = -64, 64
F8 = torch.float8_e4m3fn


def f64(t):
    """Any tensor, 8-bit ones included, in 64 bits."""
    return None if t is None else t.detach().cpu().float().double().numpy()


def to_e4m3(a):
    """Codes (bytes) of a 64-bit array whose values fit, to nearest even; NaN stays NaN."""
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).float().to(F8).view(torch.uint8).numpy()


def of_e4m3(c):
    return torch.from_numpy(np.array(c)).view(F8).float().double().numpy()


def scale_exponent(m):
    """Least e with m <= 448 2^e."""
    if not m > 0:
        return E_LO
    e = int(np.ceil(np.log2(m / 448)))
    while m <= 448 * 2.0 ** (e - 1):
        e -= 1
    while m > 448 * 2.0 ** e:
        e += 1
    return min(max(e, E_LO), E_HI)


def rotate(x, place, inv_freq, interleaved, m=1.0):
    """x [heads, D] of the token at `place`; the result and its bound."""
    y, b = x.copy(), np.zeros_like(x)
    if inv_freq is None:
        return y, b
    half = len(inv_freq)
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    # the angle less whole turns in extended precision: place f is exact in long doubles
    a = np.fmod(np.longdouble(place) * inv_freq.astype(np.longdouble), 2 * np.longdouble(np.pi) + np.longdouble(1.2246467991473532e-16) * 2)
    c, s = np.cos(a).astype(np.float64), np.sin(a).astype(np.float64)
    y[:, one] = m * (x[:, one] * c - x[:, two] * s)
    y[:, two] = m * (x[:, two] * c + x[:, one] * s)
    mag = abs(m) * (np.abs(x[:, one]) + np.abs(x[:, two]))
    b[:, one] = b[:, two] = (6 * U + 1e-9 + 2e-16 * abs(float(place))) * mag
    return y, b


def attend(q, keys, vals, scale, lo, hi, r=None, eight=True, ks=1.0):
    """One query row q [D] over keys, vals [n, D] at places lo .. hi - 1 (the caller cuts
    them): out [D], its bound before the last rounding, lse, its bound."""
    D, n = q.shape[0], hi - lo
    if n <= 0:
        return np.zeros(D), np.zeros(D), -np.inf, 0.0
    k, v = keys[lo:hi], vals[lo:hi]
    s = k @ q * scale
    A = np.abs(k) @ np.abs(q) * abs(scale) * 1.4427
    top = s.max()
    w = np.exp(s - top)
    total = w.sum()
    out = w @ v / total
    es = (2 * D + 8) * U * A.max() + 8 * U * (np.abs(s).max() * 1.4427 + 64)
    ew = es * 0.6932 + 2.0 ** -22
    S = w @ np.abs(v) / total
    wr = 2.0 ** -11 if eight else 2.0 ** -16
    big = np.abs(v).max(0) if not eight else np.abs(vals).max()
    bound = (2 * ew + wr + n * 2 * U) * S + n * 2.0 ** -25 * big
    lse = top + np.log(total)
    return out, bound, lse, ew + n * 2 * U + 4 * U * abs(lse)


def sample(x, u, temp=1.0, k=0, top_p=1.0, min_p=0.0):
    """One row of logits, 64 bits: (token, probabilities)."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    V = len(x)
    order = np.argsort(-x, kind="stable")
    if not x[order[0]] > -np.inf:
        return -1, np.zeros(V)
    top = x[order[0]]
    if not temp > 0:
        w = np.zeros(V)
        w[order[0]] = 1
    elif np.isinf(top):
        w = (x == top).astype(np.float64)
    else:
        w = np.exp((x - top) / temp)
    n = V if k <= 0 else min(k, V)
    run = np.cumsum(w[order[:n]].astype(np.longdouble))
    if not top_p > 0:
        n = 1
    elif top_p < 1:
        n = min(n, int((run < np.longdouble(top_p) * run[-1]).sum()) + 1)
    if min_p > 0:
        n = min(n, max(1, int((w[order] >= min_p).sum())))
    kept = np.zeros(V)
    kept[order[:n]] = w[order[:n]]
    run = np.cumsum(kept.astype(np.longdouble))
    hit = run > np.longdouble(max(u, 0.0) if u == u else 0.0) * run[-1]
    token = int(np.argmax(hit)) if hit.any() else int(np.nonzero(kept)[0][-1])
    return token, kept / float(run[-1])
