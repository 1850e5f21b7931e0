"""Float64 restatement of attention over the 4-bit paged key/value cache and of what feeds it.

Written from the formulas (``kv4_cache`` and the calls next to it in
``include/qmoe.h``), with plain loops over requests and heads; test
infrastructure only.
"""
from __future__ import annotations

import numpy as np

#: bit position of value i of a 32-bit word of codes
BITS = np.array([4 * (i // 2) + 16 * (i % 2) for i in range(8)], dtype=np.uint32)


def bf16_round(x: np.ndarray) -> np.ndarray:
    """Values rounded to bf16 (nearest even), as float64.  Rounds the fp32 value of x."""
    u = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def quantise(x: np.ndarray):
    """Codes uint8 and the (s, z) fp16 pair of each row (last axis) of x; fp32 steps as the format defines them."""
    x = np.where(np.isnan(x), 0.0, x).astype(np.float32)
    x = np.clip(x, np.float32(-32768), np.float32(32768))
    z = x.min(-1, keepdims=True).astype(np.float16)
    zf = z.astype(np.float32)
    s = ((x.max(-1, keepdims=True) - zf) / np.float32(15)).astype(np.float16)
    sf = s.astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        u = np.where(sf > 0, np.clip(np.rint((x - zf) / sf), 0, 15), 0)
    return u.astype(np.uint8), s[..., 0], z[..., 0]


def dequantise(u, s, z):
    return u.astype(np.float64) * s.astype(np.float64)[..., None] + z.astype(np.float64)[..., None]


def pack_page(uk, sk, zk, uv, sv, zv) -> np.ndarray:
    """Bytes of one kv head of one page from its codes [P, D] and pairs [P]."""
    def words(u):
        w = u.reshape(u.shape[0], -1, 8).astype(np.uint32)
        return (w << BITS).sum(-1, dtype=np.uint32)
    parts = [words(uk).tobytes(), words(uv).tobytes(), np.stack([sk, zk], -1).tobytes(), np.stack([sv, zv], -1).tobytes()]
    return np.frombuffer(b"".join(parts), dtype=np.uint8)


def unpack_head(raw: np.ndarray, P: int, D: int):
    """float64 keys and values [P, D] of one kv head of one page."""
    def side(i):
        w = raw[i * P * D // 2:(i + 1) * P * D // 2].copy().view(np.uint32).reshape(P, D // 8, 1)
        u = ((w >> BITS) & 15).reshape(P, D)
        sz = raw[P * D + 4 * P * i:P * D + 4 * P * (i + 1)].copy().view(np.float16).reshape(P, 2)
        return dequantise(u, sz[:, 0], sz[:, 1])
    return side(0), side(1)


def unpack(pages: np.ndarray, row, length: int, P: int, hkv: int, D: int):
    """float64 keys and values [hkv, length, D] of a request from its block-table row."""
    nb = -(-length // P)
    k, v = np.zeros((hkv, nb * P, D)), np.zeros((hkv, nb * P, D))
    for i in range(nb):
        pg = pages[row[i]].reshape(hkv, P * (D + 8))
        for h in range(hkv):
            k[h, i * P:(i + 1) * P], v[h, i * P:(i + 1) * P] = unpack_head(pg[h], P, D)
    return k[:, :length], v[:, :length]


def norm_rope(x, w, eps, cos_sin, pos, interleaved):
    """x float64 [T, H, D] -> normed (w None: not) and rotated (cos_sin None: not), not rounded."""
    x = x.copy()
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    if cos_sin is not None:
        half = cos_sin.shape[1] // 2
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos_sin[pos][:, None, :half], cos_sin[pos][:, None, half:]
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def visible(kv_len, q_len, n, causal, window):
    """(first, last + 1) of the tokens that query n of a request sees."""
    pos = kv_len - q_len + n if causal else kv_len - 1
    return max(0, pos - window + 1) if window else 0, max(0, min(kv_len, pos + 1))


def attention(q, q_start, k, v, scale, causal=True, window=0):
    """q float64 [n, hq, D]; k, v: lists of float64 [hkv, len, D].  (out, spread): spread[i, h] is
    max |v| times scale * sum |q| |k| (the largest over the visible tokens), and the second output's
    second column max |v|, for error bounds."""
    out, spread = np.zeros_like(q), np.zeros(q.shape[:2] + (2,))
    hq = q.shape[1]
    for b in range(len(k)):
        hkv, length, _ = k[b].shape
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            lo, hi = visible(length, n, i, causal, window)
            if hi <= lo:
                continue
            for h in range(hq):
                kk, vv = k[b][h // (hq // hkv)][lo:hi], v[b][h // (hq // hkv)][lo:hi]
                r = q[q_start[b] + i, h]
                s = kk @ r * scale
                p = np.exp(s - s.max())
                out[q_start[b] + i, h] = (p / p.sum()) @ vv
                vmax = np.abs(vv).max()
                spread[q_start[b] + i, h] = vmax * scale * (np.abs(kk) @ np.abs(r)).max(), vmax
    return out, spread


def block_tables(cached, new, free_pages, n_free, P, table, n_tokens):
    """Plain loops over requests and tokens; returns (table, q_start, kv_len, slots, positions, free pages left)."""
    table = table.copy()
    slots, positions = np.full(n_tokens, -1, np.int32), np.zeros(n_tokens, np.int32)
    q_start, t, taken = [0], 0, 0
    for b in range(len(cached)):
        have, want = -(-cached[b] // P), -(-(cached[b] + new[b]) // P)
        for i in range(have, want):
            at = n_free - 1 - taken
            taken += 1
            if i < table.shape[1]:
                table[b, i] = free_pages[at] if at >= 0 else -1
        for i in range(new[b]):
            if t < n_tokens:
                pos = cached[b] + i
                page = table[b, pos // P] if pos // P < table.shape[1] else -1
                slots[t] = page * P + pos % P if page >= 0 else -1
                positions[t] = pos
            t += 1
        q_start.append(min(t, n_tokens))
    return table, np.array(q_start, np.int32), (cached + new).astype(np.int32), slots, positions, max(0, n_free - taken)
