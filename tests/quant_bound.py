"""How far the attention over the 4-bit cache may be from the formula, derived from
the arithmetic of its kernels, and the same attention in coarser forms, which the
bound has to tell from it.  quant_ref.attend() bounds the same outputs from above
more loosely.

Notation: U = 2^-24; z = scale <q, K_j>, in units of log2 (z2) where the kernels
hold it; A_j = scale sum_c |q_c K_jc|; s_j the largest scale of key j's V.

Logits.  q is fixed point, within 2^-30 of the largest magnitude of its group of 32
channels: F_j = scale 2^-30 sum_r top_r sum_{c in r} |K_jc|.  Sums of digits are
exact; a group's digits are joined with one rounding, its unit is a product of two
rounded factors (the scale in units of log2, and that times K's scale), four groups
are summed with four roundings, the two halves of up to 4 heads with one more:
        dz_j = 9 U A_j + F_j.
A weight is p = 2^(z + off), off = 13 - m rounded, of a reference m that is a float:
ln 2 U (|13 - m| + |z + off|) relative, and 2^-22 of the exponential.  m lies between
z2_j + size_j - 1 and the largest z2 + size, size the exponent of s_j (clamped at -80):
|m| <= M, |z2_j + off| <= 14 + smax + (max z2 - z2_j).
Raising m, and joining warps, workers and slices, multiplies by 2^(difference of two
floats): ln 2 U |difference| + 2^-22 + 2 U each.  What is multiplied by 2^-d has a share
of at most 2^-d of the sum to which it is added, so d 2^-d < 1 stands for it, and the
spread of sizes, by which a sum of weights can keep its share.  A sum is raised by steps
of at least one: all but three of its raises are of shares below 1/8 (together less than
one more), or come with sizes.  A worker's reference is stored less 13: U (13 + M).
        ref = 2 ln 2 U (13 + M) + (7 + span) (ln 2 U (1 + span) + 2^-22 + 2 U).
Sums.  Weights are added by 4 to a lane and block, blocks to a warp (workers of 4 warps
at least), 16 warps and then the workers: 6 sigma of as many roundings, and 16 U.
        sums = U (16 + 6 sqrt(4 B + 16 + W)), B = n / 128 + 1 blocks, W = min(592, B) workers.
Outputs.  w = p s: U; held as a pair of halves: 2^-22, and 2^-37 of the largest p s
absolutely (a half's 2^-25, lifted by 2^13 over a reference of at most twice that).  With
|code - 8| <= 7 and s = max |V| / 7 the n keys give n 2^-37 max(p max|V|).  Products of 16
keys are summed by instructions that may cut, up to four in a row: 16 U.
"""
import math

import numpy as np

U = 2.0 ** -24
LN2 = math.log(2)


def fixed_point(q, bits=30, per_group=True):
    """q [..][128] to `bits` bits and a sign below the power of two above the largest magnitude, of each group of 32 or of all."""
    g = q.reshape(-1, 4, 32)
    top = np.abs(g).max(-1, keepdims=True)
    if not per_group:
        top = top.max(1, keepdims=True)
    unit = 2.0 ** (np.floor(np.log2(np.where(top > 0, top, 1.0))) + 1 - bits)
    return (np.rint(g / unit) * unit).reshape(q.shape)


def v_sizes(V):
    """Exponent of each key's largest scale of V, as the kernel clamps it."""
    s = np.abs(V).max(1) / 7
    return np.maximum(np.floor(np.log2(np.where(s > 0, s, 2.0 ** -126))) + 1, -80.0)


def attend(q, K, V, scale=None):
    """q [G][128], K, V [n][128] in 64 bits, n > 0 -> out [G][128], lse [G], weights [G][n], and the bounds of their
    errors: absolute, absolute, relative."""
    n = len(K)
    scale = 1 / math.sqrt(128) if scale is None else scale
    z = scale * (q @ K.T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    out, lse = p @ V, (np.log(total) + top)[:, 0]

    A = scale * (np.abs(q) @ np.abs(K).T)
    tops = np.repeat(np.maximum(np.abs(q).reshape(-1, 4, 32).max(-1), 2.0 ** -97), 32, 1)
    dz = 9 * U * A + scale * 2.0 ** -30 * (tops @ np.abs(K).T)
    z2, size = z / LN2, v_sizes(V)
    smax, span = np.abs(size).max(), size.max() - size.min()
    M = np.abs(z2).max(1, keepdims=True) + smax
    ep = dz + LN2 * U * (14 + smax + z2.max(1, keepdims=True) - z2) + 2.0 ** -22
    ref = 2 * LN2 * U * (13 + M) + (7 + span) * (LN2 * U * (1 + span) + 2.0 ** -22 + 2 * U)
    B = n / 128 + 1
    sums = U * (16 + 6 * math.sqrt(4 * B + 16 + min(592, B)))
    el = (p * ep).sum(1, keepdims=True) + ref + sums
    held = n * 2.0 ** -37 * (p * np.abs(V).max(1)).max(1, keepdims=True)
    e_out = (p * ep) @ np.abs(V) + (p @ np.abs(V)) * (ref + sums + 2.0 ** -22 + 18 * U + el) + held + 1e-37
    e_lse = el[:, 0] + U * (4 * np.abs(lse) + 2 * (13 + smax + math.log2(n) + M[:, 0] + np.abs(lse) / LN2))
    e_w = dz + e_lse[:, None] + LN2 * U * np.abs(z - lse[:, None]) / LN2 + 2.0 ** -22
    return out, lse, p, e_out, e_lse, e_w


def coarse(q, K, V, form, scale=None):
    """out [G][128], lse [G] with one part in fewer bits."""
    scale = 1 / math.sqrt(128) if scale is None else scale
    if form == "q 15 bits":
        q = fixed_point(q, 15)
    elif form == "q 22 bits of all":
        q = fixed_point(q, 22, per_group=False)
    elif form == "q 30 bits of all":
        q = fixed_point(q, 30, per_group=False)
    z = scale * (q @ K.T)
    if form == "logits as halves":
        z = z.astype(np.float16).astype(np.float64)
    top = z.max(1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(1, keepdims=True)
    if form == "weights as halves":          # times each group's scale, lifted as the kernel lifts them
        s = np.abs(V).reshape(-1, 4, 32).max(-1) / 7
        ps = p[:, :, None] * s[None]
        lift = 2.0 ** (13 - np.ceil(np.log2(ps.max((1, 2), keepdims=True))))
        ps = (ps * lift).astype(np.float16).astype(np.float64) / lift
        code = np.where(np.repeat(s, 32, 1) > 0, V / np.repeat(np.where(s > 0, s, 1.0), 32, 1), 0.0)
        return np.einsum("gjr,jrc->grc", ps, code.reshape(-1, 4, 32)).reshape(len(q), 128) / total, (np.log(total) + top)[:, 0]
    return (p / total) @ V, (np.log(total) + top)[:, 0]
