"""Float64 restatement of what stands around a decoder layer's attention and experts: the norm of whole rows with the
residual's addition, the scored choice of experts, and attention over chosen blocks of the 4-bit cache.

Written from the formulas of the calls in ``include/qmoe.h``, with plain loops; test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import kv4 as K


def add_norm(x, residual, weight, eps):
    """(x + residual, its norm times weight), float64."""
    h = x if residual is None else x + residual
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, y if weight is None else y * weight


def scales(y, group):
    """max |y| / 448 over each row (group 0) or each `group` values of it."""
    cut = [slice(i, i + group) for i in range(0, y.shape[1], group)] if group else [slice(None)]
    return np.stack([np.abs(y[:, c]).max(-1) for c in cut], -1) / 448


def e4m3(code):
    """Values of e4m3 bytes: sign, 4 exponent bits (bias 7, 0 subnormal), 3 fraction bits, no infinity."""
    code = np.asarray(code).astype(np.int64)
    e, f = (code >> 3) & 15, code & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(float) - 10))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def route(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, best=1, renorm=False, scale=1.0):
    """(ids [T, k], gates [T, k] float64), by comparing one value after another."""
    ids, gates = np.zeros((len(logits), k), np.int64), np.zeros((len(logits), k))
    for t, row in enumerate(np.asarray(logits, dtype=np.float64)):
        row = np.minimum(np.where(np.isnan(row), -np.inf, row), np.finfo(np.float32).max)
        with np.errstate(over="ignore", invalid="ignore"):
            if sigmoid:
                s = 1 / (1 + np.exp(-row))
            elif row.max() > -np.inf:
                s = np.exp(row - row.max())
                s /= s.sum()
            else:
                s = np.zeros_like(row)
            c = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        c = np.where(np.isnan(c), -np.inf, c)
        order = row if bias is None else c
        size = len(row) // groups
        allowed = list(range(len(row)))
        if groups > 1:
            by = order if best == 1 else c
            with np.errstate(invalid="ignore"):
                value = [sum(sorted(by[g * size:(g + 1) * size])[-best:]) for g in range(groups)]
            value = [-np.inf if np.isnan(v) else v for v in value]
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
            allowed = [e for e in allowed if e // size in kept]
        chosen = sorted(allowed, key=lambda e: (-order[e], e))[:k]
        w = s[chosen]
        if renorm and sigmoid and row[chosen].max() < 0:
            # ratios, whatever the scores' magnitude
            top = row[chosen].max()
            w = np.exp(row[chosen] - top) / (1 + np.exp(row[chosen])) if top > -np.inf else np.zeros(k)
        if renorm and w.sum() > 0:
            w = w / w.sum()
        ids[t], gates[t] = chosen, w * scale
    return ids, gates


def bounds(keys):
    """(hi codes, lo codes, step) of the keys [tokens, head_dim] of a block (their fp32 values)."""
    k = keys.astype(np.float32).astype(np.float64)
    hi, lo = k.max(0), k.min(0)
    big = max(np.abs(hi).max(), np.abs(lo).max())
    if big == 0:
        return np.zeros(k.shape[1], np.int8), np.zeros(k.shape[1], np.int8), 0.0
    step = 2.0 ** math.frexp(big)[1]
    while big <= 127 * step / 2:
        step /= 2
    return np.ceil(hi / step).astype(np.int8), np.floor(lo / step).astype(np.int8), step


def whole_query(q):
    """(sum of positive parts, sum of negative parts) over the heads of q [G, head_dim], as whole numbers."""
    bits = 15 - math.ceil(math.log2(q.shape[0]))
    big = 3.3895313892515355e38
    q = np.clip(np.where(np.isnan(q), 0, q), -big, big)
    top = np.abs(q).max()
    up = bits - math.frexp(top)[1] if top > 0 else 0
    whole = np.clip(np.rint(np.ldexp(q, up)), 1 - 2 ** bits, 2 ** bits - 1).astype(np.int64)
    return np.maximum(whole, 0).sum(0), np.minimum(whole, 0).sum(0)


def select(q, q_start, kv_len, table, codes, steps, P, top, first, last, sel, max_kv):
    """sel [n, hkv, top] filled in as kv4_select_blocks does; q float64 [n, hq, head_dim], codes [pages, hkv, 2, head_dim]."""
    sel = sel.copy()
    hkv = codes.shape[1]
    G = q.shape[1] // hkv
    for b in range(len(kv_len)):
        for t in range(q_start[b], q_start[b + 1]):
            pos = kv_len[b] - (q_start[b + 1] - t)
            seen = pos // P + 1 if pos >= 0 and 0 <= kv_len[b] <= max_kv else 0
            for h in range(hkv):
                up, down = whole_query(q[t, h * G:(h + 1) * G])
                value = []
                for j in range(seen):
                    page = table[b, j] if j < table.shape[1] else -1
                    if not 0 <= page < len(codes):
                        value.append(-np.inf)
                        continue
                    dot = int(codes[page, h, 0].astype(np.int64) @ up + codes[page, h, 1].astype(np.int64) @ down)
                    value.append(float(np.float32(dot) * np.float32(steps[page, h])))
                forced = sorted(set(range(min(first, seen))) | set(range(max(0, seen - last), seen))) if seen > top else list(range(seen))
                rest = [j for j in range(seen) if j not in forced]
                rest = sorted(rest, key=lambda j: (-value[j], j))[:top - len(forced)] if seen > top else []
                pick = sorted(forced + rest)
                sel[t, h] = pick + [-1] * (top - len(pick))
    return sel


def attention_blocks(q, q_start, kv_len, table, pages, P, hkv, sel, scale):
    """(out, spread) as oracle.kv4.attention gives them, each query over its list's blocks; q float64 [n, hq, head_dim]."""
    out, spread = np.zeros_like(q), np.zeros(q.shape[:2] + (2,))
    n, hq, D = q.shape
    G, top = hq // hkv, sel.shape[2]
    for b in range(len(kv_len)):
        for t in range(q_start[b], q_start[b + 1]):
            pos = kv_len[b] - (q_start[b + 1] - t)
            if pos < 0:
                continue
            seen = pos // P + 1
            for h in range(hkv):
                k, v = [], []
                for blk in sel[t, h, :min(top, seen)]:
                    if not 0 <= blk < seen or blk >= table.shape[1] or not 0 <= table[b, blk] < len(pages):
                        continue
                    kk, vv = K.unpack_head(pages[table[b, blk]].reshape(hkv, -1)[h], P, D)
                    m = min(P, pos + 1 - blk * P)
                    k.append(kk[:m])
                    v.append(vv[:m])
                if not k:
                    continue
                k, v = np.concatenate(k), np.concatenate(v)
                for i in range(h * G, (h + 1) * G):
                    s = k @ q[t, i] * scale
                    p = np.exp(s - s.max())
                    out[t, i] = (p / p.sum()) @ v
                    big = np.abs(v).max()
                    spread[t, i] = big * scale * (np.abs(k) @ np.abs(q[t, i])).max(), big
    return out, spread
