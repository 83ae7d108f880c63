"""Elementwise error bounds of the paged decode against its 64-bit definition, one query head at a time.

From the roundings that the kernel documents, in normalised weights w_t (they sum to 1), with a group's stored scale s and zero
z, a code n, and v = n s + z.  What is rounded independently a token (p, p s and p z to fp16) adds up as a root of squares: a sum
of independent errors, each within its b_t and without bias, leaves SIGMA sqrt(sum b_t^2) with a probability below
2 exp(-SIGMA^2 / 2) (Hoeffding).  What may have a bias (tensor-core sums, which truncate; float32 logits) adds up by size.

 * output: one rounding, eps / 2.
 * logits: float32 sums (d + 8 roundings of 2^-23 of sum |q k| scale) and the exponential (2^-20); products of a code, held as a
   subnormal of nominal size 2^-14, keep 2^-23 of that: 2^-13 of a step of the largest product of a group's 16 channels, 18 of
   these (the second 16 weigh a sixteenth).  A weight's relative error moves the output by w (v - o).
 * bf16 outputs: p (2^-11 of w (v - o)), p s (2^-11 of w n s), sums of four p z (four roundings of 2^-11 of sums of four), and
   2^-13 max(p s) for each of the 16 products of a cell, truncated like the logits'.
 * fp16 outputs: two fp16 parts of each (2^-22), products truncated to 2^-19 max(p s), 32 a cell.
 * fp16's smallest step, 2^-25 by half.  The largest p of a warp's part is 2^9 or more in units of 2^E, the power of two above the
   largest scale and zero of groups that lie within 2^8 of each other: 2^(E - 34) of the largest weight a token, for p (times v)
   and for p s (times a code) and the sums of p z; 2^(E - 30) for the latter of fp16 outputs.  Groups further apart have their
   scales and zeros brought to 2^6 (2^-31 of the group's largest, times a code) and p to 2^3.
 * float32 sums of a part of `cells` cells (three products a cell at most, 2^-23 each) and of the parts' records (2^-18 in all).
"""

from __future__ import annotations

import numpy as np

SIGMA = 6.0


def attend(q, k, v, scale):
    """(weights [n], output [d]) in 64 bits."""
    s = k @ q * scale
    w = np.exp(s - s.max())
    w /= w.sum()
    return w, w @ v


def bound(q, k, key, v, val, scale, out_bits, cells=2):
    """Largest error of each channel of the output (all float64; key, val: the oracle's codes, scale16 and zero16; out_bits: 8 of
    bf16, 11 of fp16; cells: of a warp's part, see above)."""
    n, d = v.shape
    w, o = attend(q, k, v, scale)
    W = w[:, None]
    s, z = (np.repeat(np.asarray(val[x], np.float64), 32, 1) for x in ("scale16", "zero16"))
    code = np.asarray(val["codes"], np.float64)
    lead = np.maximum(np.abs(np.asarray(val["scale16"], np.float64)), np.abs(np.asarray(val["zero16"], np.float64))).max(0)
    E = np.maximum(np.floor(np.log2(np.maximum(lead, 2.0 ** -24))) + 1, -2)
    own_E = np.repeat(E, 32)
    E = np.minimum(E.max(), own_E + 8)
    qmax = np.abs(q).reshape(-1, 32).max(1)
    logit = (d + 8) * 2.0 ** -23 * (np.abs(k) @ np.abs(q)) * abs(scale) + 2.0 ** -20
    logit = logit + 18 * 2.0 ** -13 * (np.asarray(key["scale16"], np.float64) @ qmax) * abs(scale)
    off = np.abs(v - o)
    tol = 2.0 ** -out_bits * np.abs(o) + (w * logit) @ off
    pad = -n % 16
    cell_top = np.pad(W * s, ((0, pad), (0, 0))).reshape(-1, 16, d).max(1).sum(0)  # sum over cells of max p s
    if out_bits == 8:
        own = 2.0 ** -11 * np.concatenate([W * off, W * code * s, 4 * W * np.abs(z)])
        tol = tol + SIGMA * np.sqrt((own ** 2).sum(0)) + 16 * 2.0 ** -13 * cell_top
    else:
        tol = tol + 2.0 ** -22 * (W * (off + 2 * code * s + 2 * np.abs(z))).sum(0) + 32 * 2.0 ** -19 * cell_top
        tol = tol + n * w.max() * 2.0 ** (E - 30)
    floor = w.max() * 2.0 ** (np.maximum(E, 6) - 34) * (15 * s + np.abs(z)).sum(0) + n * w.max() * 16 * 2.0 ** (E - 34)
    floor = floor + 16 * 2.0 ** (own_E - 31)
    spread = (W * (code * s + np.abs(z))).sum(0)
    return tol + floor + (3 * cells * 2.0 ** -23 + 2.0 ** -18) * (spread + np.abs(o)) + 2.0 ** -25
