"""Plain NumPy float64 definitions of the operators around a drafted step (TEST
INFRASTRUCTURE ONLY): rotary positions and head norms, attention of a tree of
drafted tokens, accumulated attention weight, eviction and packing.

Like the rest of the package these take bf16 bit patterns and share no code
with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import bf16_bits_to_f64, gather_kv, slot_of


# ----------------------------------------------------------------------------
# Rotation and norms
# ----------------------------------------------------------------------------
def rope(x, positions, inv_freq, interleaved: bool, factor: float):
    """Rotate the first ``2 * len(inv_freq)`` dims of float64 rows [T, H, D]: pair
    ``i`` of a token at position ``p`` turns by ``p * inv_freq[i]``."""
    y = np.array(x, np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = np.asarray(positions, np.float64) * float(inv_freq[i])
        c, s = np.cos(ang)[:, None] * factor, np.sin(ang)[:, None] * factor
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    return y


def head_norm(x, weight, eps: float):
    """``x * w / sqrt(mean(x^2) + eps)`` over the last dim, float64."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


# ----------------------------------------------------------------------------
# Tree attention and accumulated weight
# ----------------------------------------------------------------------------
def _visible(mask_row, c: int, n: int):
    """Key indices a drafted token sees: the cached ones and its mask's bits."""
    bits = [j for j in range(n) if (int(mask_row[j // 64]) >> (j % 64)) & 1]
    return np.concatenate([np.arange(c), c + np.asarray(bits, np.int64)]).astype(np.int64)


def tree_attention(q, cu, mask, k_pool, v_pool, tables, lens, scale: float):
    """Row ``i`` of sequence ``s`` attends to the sequence's ``c = lens[s] - n``
    cached tokens and to those of its ``n`` new tokens whose bit is set in
    ``mask[row]`` (int64 words, bit ``j`` = new token ``j``).  No visible token:
    zeros and ``-inf``.  Returns float64 ``out`` [T, Hq, D], ``lse`` [T, Hq]."""
    t, hq, d = q.shape
    hkv = k_pool.shape[1]
    qf = bf16_bits_to_f64(q)
    out = np.zeros((t, hq, d))
    lse = np.full((t, hq), -np.inf)
    for s in range(len(lens)):
        r0, r1 = int(cu[s]), int(cu[s + 1])
        n, L = r1 - r0, int(lens[s])
        kb, vb = gather_kv(k_pool, v_pool, tables[s], L)
        K, V = bf16_bits_to_f64(kb), bf16_bits_to_f64(vb)
        for i in range(n):
            see = _visible(mask[r0 + i], L - n, n)
            if not len(see):
                continue
            for h in range(hq):
                g = h // (hq // hkv)
                x = scale * (K[g][see] @ qf[r0 + i, h])
                w = np.exp(x - x.max())
                out[r0 + i, h] = w @ V[g][see] / w.sum()
                lse[r0 + i, h] = x.max() + np.log(w.sum())
    return out, lse


def attention_mass(q, lse, cu, k_pool, tables, lens, scale: float):
    """Per sequence, float64 [Hkv, L]: for every cached token the sum over the
    sequence's query rows ``i`` (at position ``c + i``, seeing keys up to it) and
    the q heads of its KV head of ``exp(scale * q.k - lse)``."""
    hq = q.shape[1]
    hkv = k_pool.shape[1]
    qf = bf16_bits_to_f64(q)
    res = []
    for s in range(len(lens)):
        r0, r1 = int(cu[s]), int(cu[s + 1])
        n, L = r1 - r0, int(lens[s])
        K = bf16_bits_to_f64(gather_kv(k_pool, k_pool, tables[s], L)[0])
        m = np.zeros((hkv, L))
        for i in range(n):
            top = L - n + i + 1
            for h in range(hq):
                if lse[r0 + i, h] == -np.inf:
                    continue
                x = scale * (K[h // (hq // hkv)][:top] @ qf[r0 + i, h])
                m[h // (hq // hkv), :top] += np.exp(x - float(lse[r0 + i, h]))
        res.append(m)
    return res


# ----------------------------------------------------------------------------
# Eviction and packing
# ----------------------------------------------------------------------------
def evict_choice(mass, length: int, budget: int, sink: int, recent: int):
    """Indices kept, ascending: ``min(length, budget)`` tokens -- the first
    ``sink``, the last ``recent``, then the heaviest others (the lowest index
    first among equals; NaN counts as less than -inf)."""
    keep = min(int(length), max(int(budget), 0))
    sink = min(keep, sink)
    recent = min(keep - sink, recent)
    forced = list(range(sink)) + list(range(length - recent, length))
    value = lambda t: (1, 0.0) if np.isnan(mass[t]) else (0, -float(mass[t]))  # noqa: E731
    others = sorted(range(sink, length - recent), key=lambda t: (value(t), t))
    return np.array(sorted(forced + others[:keep - len(forced)]), np.int64)


def compact(pool, table, base: int, kept, new_table=None):
    """Copy of ``pool`` where, for KV head ``g`` of one sequence, row ``base + i`` of
    ``new_table`` (default: ``table``) holds what row ``base + kept[g][i]`` of
    ``table`` held."""
    res = np.array(pool)
    bs = pool.shape[2]
    new_table = table if new_table is None else new_table
    for g in range(pool.shape[1]):
        for i, t in enumerate(kept[g]):
            src, dst = slot_of(table, base + int(t), bs), slot_of(new_table, base + i, bs)
            res[dst // bs, g, dst % bs] = pool[src // bs, g, src % bs]
    return res
