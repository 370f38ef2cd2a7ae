"""The 4-bit paged cache: quantisation, pages, and attention over them.

A page holds 16 slots of one kv head: 16 rows of D/2 code bytes (even column in
the low nibble), then 16 rows of D/16 scale bytes.  Sixteen consecutive
columns share a scale byte b, the half-precision number with bits
min(b, 0xE2) << 7; codes are E2M1 (sign bit, then the index of the magnitude
among 0, 0.5, 1, 1.5, 2, 3, 4, 6).

Quantisation works on exact fp64 values (every boundary and product involved is
exact in fp64): scale = nearest representable to max|x| / 6, ties to the even
byte, at most 10240; code = nearest magnitude to |x| / scale, ties to the even
code.  NaN counts as 0; infinities saturate.
"""

from __future__ import annotations

import numpy as np

from .attention import bf16_to_f64

PAGE = 16
GROUP = 16
MAX_SCALE = 0xE2
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def scale_values() -> np.ndarray:
    """Values of scale bytes 0..0xE2."""
    bits = (np.arange(MAX_SCALE + 1, dtype=np.uint16) << 7).astype(np.uint16)
    return bits.view(np.float16).astype(np.float64)


def _nearest(y, grid):
    """Index of the nearest grid value to y >= 0, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, y, side="left")
    hi = np.searchsorted(mid, y, side="right")
    return np.where(lo == hi, lo, lo + (lo & 1))


def quantise_rows(x_bits):
    """bf16 bits [..., D] -> (codes uint8 [..., D/2], scales uint8 [..., D/16])."""
    x = bf16_to_f64(x_bits)
    sign = (np.asarray(x_bits) >> 15).astype(np.uint8)
    nan = np.isnan(x)
    mag = np.where(nan, 0.0, np.abs(x))
    sign = np.where(nan, 0, sign).astype(np.uint8)
    g = mag.reshape(*mag.shape[:-1], -1, GROUP)
    grid = scale_values()
    byte = _nearest(np.minimum(g.max(-1), 1e30) / 6.0, grid)
    s = grid[byte][..., None]
    y = np.where(s > 0, np.minimum(g, 1e30) / np.where(s > 0, s, 1.0), 0.0)
    code = _nearest(y, MAGNITUDES).astype(np.uint8).reshape(mag.shape) + 8 * sign
    pair = code.reshape(*code.shape[:-1], -1, 2)
    return (pair[..., 0] | (pair[..., 1] << 4)).astype(np.uint8), byte.astype(np.uint8)


def dequantise_rows(codes, scales):
    """fp64 [..., D] values of code and scale rows."""
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = scale_values()[np.minimum(scales, MAX_SCALE)]
    return v * np.repeat(s, GROUP, axis=-1)


def split_pages(pool):
    """(codes [...][16][D/2], scales [...][16][D/16]) views of pages [...][9 D]."""
    D = pool.shape[-1] // 9
    return (pool[..., :8 * D].reshape(*pool.shape[:-1], PAGE, D // 2),
            pool[..., 8 * D:].reshape(*pool.shape[:-1], PAGE, D // GROUP))


def write_rows(pool, x_bits, slots):
    """Copy of pool uint8 [num_blocks][Hkv][9 D] with rows x_bits
    [T][Hkv][D] stored at slots (those outside the pool skipped)."""
    out = pool.copy()
    codes, scales = split_pages(out)
    c, s = quantise_rows(x_bits)
    for t, slot in enumerate(slots):
        if 0 <= slot < out.shape[0] * PAGE:
            codes[slot // PAGE, :, slot % PAGE] = c[t]
            scales[slot // PAGE, :, slot % PAGE] = s[t]
    return out


def read_rows(pool, slots):
    """fp64 [T][Hkv][D] values at slots (zeros outside the pool)."""
    codes, scales = split_pages(pool)
    D = pool.shape[-1] // 9
    out = np.zeros((len(slots), pool.shape[1], D))
    for t, slot in enumerate(slots):
        if 0 <= slot < pool.shape[0] * PAGE:
            out[t] = dequantise_rows(codes[slot // PAGE, :, slot % PAGE], scales[slot // PAGE, :, slot % PAGE])
    return out


def commit_path(k_pool, v_pool, block_table, prefix_len, accept_len, path, err, tail_base=None):
    """The bf16 commit's moves on 4-bit pools [num_blocks][Hkv][9 D]."""
    outs = [k_pool.copy(), v_pool.copy()]
    B = len(prefix_len)
    new_len = np.array(prefix_len, dtype=np.int32).copy()
    moved = np.zeros(B, dtype=np.int32)
    for b in range(B):
        if err[b] != 0:
            continue
        P = int(prefix_len[b])
        T = P if tail_base is None else int(tail_base[b])
        A = int(accept_len[b])
        new_len[b] = P + A + 1
        src = [T + int(path[b, k]) - 1 for k in range(A + 1)]
        moved[b] = sum(s != P + k for k, s in enumerate(src))
        for before, after in zip((k_pool, v_pool), outs):
            for view_b, view_a in zip(split_pages(before), split_pages(after)):
                for k, s in enumerate(src):
                    d = P + k
                    view_a[block_table[b, d // PAGE], :, d % PAGE] = \
                        view_b[block_table[b, s // PAGE], :, s % PAGE]
    return outs[0], outs[1], new_len, moved


def visible(mask, b, i, n, N_max):
    """Boolean [n]: the tree nodes that node i sees (mask None: 0..i)."""
    if mask is None:
        return np.arange(n) <= i
    words = np.asarray(mask[b, i]).view(np.uint32)
    return np.array([(int(words[j // 32]) >> (j % 32)) & 1 for j in range(n)], dtype=bool)


def tree_attention_q4(q_bits, k_pool, v_pool, block_table, prefix_len, n_nodes, mask, err, scale):
    """fp64 attention over 4-bit pools.  Returns (out, lse, weight, total,
    score): weight [B][N_max][Hq][D] = sum p |v|, total [B][N_max][Hq][D] = sum
    |v| over the visible keys and score [B][N_max][Hq] = max over the visible
    keys of sum |q| |k| |scale|, which scale the rounding bounds."""
    B, N_max, Hq, D = q_bits.shape
    Hkv = k_pool.shape[1]
    g = Hq // Hkv
    q = bf16_to_f64(q_bits)
    out = np.zeros(q.shape)
    weight, total = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    score = np.zeros(q.shape[:3])
    for b in range(B):
        if err is not None and err[b] != 0:
            continue
        P, n = int(prefix_len[b]), int(n_nodes[b]) if n_nodes is not None else N_max
        slots = [int(block_table[b, t // PAGE]) * PAGE + t % PAGE for t in range(P + n)]
        k, v = read_rows(k_pool, slots), read_rows(v_pool, slots)
        for i in range(n):
            seen = np.concatenate([np.ones(P, dtype=bool), visible(mask, b, i, n, N_max)])
            if not seen.any():
                continue
            for h in range(Hq):
                kk, vv = k[seen, h // g], v[seen, h // g]
                with np.errstate(all="ignore"):
                    x = kk @ q[b, i, h] * scale
                    m = x.max()
                    p = np.exp(x - m)
                    lse[b, i, h] = m + np.log(p.sum())
                    p = p / p.sum()
                    out[b, i, h] = p @ vv
                    weight[b, i, h] = p @ np.abs(vv)
                    total[b, i, h] = np.abs(vv).sum(0)
                    score[b, i, h] = (np.abs(kk) @ np.abs(q[b, i, h])).max() * abs(scale)
    return out, lse, weight, total, score
