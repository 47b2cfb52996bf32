"""The 4-bit KV cache in 64 bits, from the documented block format: what the
tests hold the kernels against.  Plain numpy, one row and one pair at a time."""
import math

import numpy as np
import torch

D, KEYS, BLOCK = 128, 32, 4608
U = 2.0 ** -24                      # half a step of fp32, relative


def k_nibble(c):
    r, x = divmod(c, 32)
    return 32 * (x // 8) + 8 * r + x % 8


def v_nibble(c, j):
    r, x = divmod(c, 32)
    i, g = divmod(x, 8)
    return 16 * (g ^ 4 if j & 2 else g) + 4 * r + i


K_NIB = np.array([k_nibble(c) for c in range(D)])
V_NIB = np.array([[v_nibble(c, j) for c in range(D)] for j in range(KEYS)])
GROUP = np.arange(D) // 32


def bf16_value(bits):
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def decode(blocks):
    """One pair's blocks [m][4608] u8 -> codes K, V [32 m][128], scales K, V [32 m][4] in 64 bits."""
    m = blocks.shape[0]
    out = []
    for code0, nib in ((0, np.broadcast_to(K_NIB, (KEYS, D))), (2048, V_NIB)):
        b = blocks[:, code0:code0 + 2048].reshape(m, KEYS, 64)
        byte = np.take_along_axis(b, np.broadcast_to(nib // 2, (m, KEYS, D)), 2)
        out.append(((byte >> (4 * (nib % 2)).astype(np.uint8)) & 15).reshape(-1, D).astype(np.int64))
    for s0 in (4096, 4352):
        out.append(bf16_value(np.ascontiguousarray(blocks[:, s0:s0 + 256]).view(np.uint16)).reshape(-1, 4))
    return out


def values(blocks):
    """K, V [32 m][128] of one pair's blocks."""
    kc, vc, ks, vs = decode(blocks)
    return (kc - 8) * ks[:, GROUP], (vc - 8) * vs[:, GROUP]


def stored(x):
    """What rows x [n][128] (fp32 or bf16 values in fp32) are stored as: codes, scale bits (bf16), values."""
    g = np.asarray(x, np.float32).reshape(-1, 4, 32)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(g).max(-1)
        top = np.where(np.isfinite(top), top, np.float32(np.nan))
        s32 = top / np.float32(7)
        scale = torch.from_numpy(s32).to(torch.bfloat16)
        s = scale.double().numpy()[..., None]
        k = np.where(s > 0, np.rint(g.astype(np.float64) / s), 0.0)
    return (np.clip(k, -7, 7) + 8).reshape(-1, D), s[..., 0], (np.clip(k, -7, 7) * s).reshape(-1, D)


def pack(K, V):
    """Rows [n][128] -> blocks [ceil(n / 32)][4608]; rows behind n are 0xff bytes (NaN scales)."""
    n = len(K)
    m = max(1, -(-n // KEYS))
    nibs = np.full((m * KEYS, 2, D), 15, np.uint8)
    scales = np.full((m * KEYS, 2, 4), 0xffff, np.uint16)
    for which, x in ((0, K), (1, V)):
        code, s, _ = stored(x)
        at = np.broadcast_to(K_NIB, (n, D)) if which == 0 else V_NIB[np.arange(n) % KEYS]
        np.put_along_axis(nibs[:n, which], at, code.astype(np.uint8), 1)
        scales[:n, which] = torch.from_numpy(s).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    byte = nibs[..., 0::2] | (nibs[..., 1::2] << 4)
    parts = [byte[:, 0].reshape(m, -1), byte[:, 1].reshape(m, -1)]
    parts += [np.ascontiguousarray(scales[:, w]).view(np.uint8).reshape(m, -1) for w in (0, 1)]
    return np.concatenate(parts, 1)


def attend(q, K, V, scale=None):
    """q [G][128], K, V [n][128] in 64 bits -> out [G][128], lse [G], weights [G][n], and the bound of the
    kernel's errors: of out [G][128], of lse [G], of each weight relative [G].

    Bounds.  A logit is a sum of 128 products of exact codes with q (fp32 q as a pair of halves, off by 2^-22
    relative at most), summed in fp32 by instructions that may cut instead of round (2 U a step, 136 steps), scaled
    by a few rounded factors: |dz| <= (2 * 136 U + 2^-21) S, S = scale sum |q||k|; z itself is rounded to fp32 in
    log2 units (2 U |z|, also of the maximum).  A weight's relative error is then e = 2 (dz) + 2^-21 (the two
    exponentials).  Sums over n keys: steps of 16 keys that may cut (2 U each), else rounding, six sigma.
    A product p s of a weight and a group's scale is held as a pair of halves lifted by 2^13 over a reference at most
    2 max(p s), so it is off by at most 2^-25 of that unit, 2^-37 max(p s), beside the 2^-22 relative that e covers;
    with |code - 8| <= 7 the n keys give at most 7 n 2^-37 max(p s).  s of a key is its largest |V| / 7 (pack() makes the
    largest code of a group +-7)."""
    n = len(K)
    scale = 1 / math.sqrt(D) if scale is None else scale
    if n == 0:
        z = np.zeros(len(q))
        return np.zeros((len(q), D)), z - np.inf, np.zeros((len(q), 0)), np.zeros((len(q), D)), z, z
    z = scale * (q @ K.T)
    top = z.max(1, keepdims=True)
    e = np.exp(z - top)
    total = e.sum(1, keepdims=True)
    p = e / total
    S = (scale * (np.abs(q) @ np.abs(K).T)).max(1)
    dz = (272 * U + 2.0 ** -21) * S + 4 * U * np.abs(z).max(1)
    sums = U * (n / 8 + 6 * math.sqrt(n))
    rel = 2 * dz + 2.0 ** -20 + sums
    out = p @ V
    held = n * 2.0 ** -37 * (p * np.abs(V).max(1)).max(1, keepdims=True)
    return out, (np.log(total) + top)[:, 0], p, (p @ np.abs(V)) * rel[:, None] + held + 1e-37, rel + 2 * U * np.abs(top[:, 0]), rel


def evict(acc, n, budget, sink, recent):
    """Kept slots of a pair of n keys, ascending."""
    if n <= budget:
        return np.arange(n)
    mid = np.arange(sink, n - recent)
    a = np.asarray(acc, np.float64)[mid]
    a = np.where(np.isnan(a), -np.inf, a)
    nan = np.isnan(np.asarray(acc)[mid])
    order = np.lexsort((mid, nan, -a))            # heaviest first, NaN behind -inf, then the lower slot
    return np.sort(np.concatenate([np.arange(sink), mid[order[:budget - sink - recent]], np.arange(n - recent, n)]))
