"""The 8-bit block-scaled cache, written out from its definition.

TEST INFRASTRUCTURE: see the package docstring for who may import this.

Format (include/mtkv.h, "8-bit block-scaled cache"; it has no counterpart in
the pages): pools uint8 [n_phys][block_size][n_kv_heads][head_dim] of e4m3
codes, float32 scales [n_phys][n_kv_heads], value = code * scale.
  * e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; exponent field 0 is
    f * 2^-9; 0x7f and 0xff are NaN; no infinities; largest value 448.
  * store: scale = least power of two 2^e, e >= -126, with amax <= 448 * 2^e
    over the finite new values of a (block, head), not below the scale of kept
    rows; codes nearest, ties to the even code; infinities saturate.
  * attention as in `oracle.attention`, in float64 on the decoded values.

The nearest code is found by comparing with all 127 magnitudes, not by bit
arithmetic.
"""
from __future__ import annotations

import math

import numpy as np


def code_values() -> np.ndarray:
    """float64 value of each of the 256 codes."""
    v = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        a = math.ldexp(f, -9) if e == 0 else math.ldexp(8 + f, e - 10)
        if c & 127 == 127:
            a = math.nan
        v[c] = -a if c & 128 else a
    return v


_VALUES = code_values()
_MAGS = _VALUES[:127]  # ascending: codes 0 .. 126


def encode(x) -> np.ndarray:
    """Nearest code of each value, ties to the even code; saturates at 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_MAGS, np.where(np.isnan(a), 0.0, a))   # first magnitude >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _MAGS[lo], _MAGS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(hi % 2 == 0, hi, lo)))
    c = np.where(np.isnan(a), 127, c)
    return (c + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def pow2_scale(amax: float) -> float:
    """Least 2^e, e >= -126, with amax <= 448 * 2^e; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def store(pool, scales, new, table, ctx, q_start, block_size) -> None:
    """Store rows of one of K / V in place. new: float array [n_tokens][H][D]."""
    n_phys, bs = pool.shape[0], block_size
    new = np.asarray(new, dtype=np.float64)
    for s in range(len(ctx)):
        q0, n = int(q_start[s]), int(q_start[s + 1] - q_start[s])
        if n <= 0:
            continue
        p0 = int(ctx[s]) - n
        for b in range(p0 // bs, (p0 + n - 1) // bs + 1):
            phys = int(table[s][b])
            if phys < 0 or phys >= n_phys:
                continue
            a, z = max(p0 - b * bs, 0), min(p0 + n - b * bs, bs)
            x = new[q0 + b * bs + a - p0: q0 + b * bs + z - p0]          # [rows][H][D]
            for h in range(pool.shape[2]):
                v = x[:, h]
                fin = np.abs(v[np.isfinite(v)])
                need = pow2_scale(float(fin.max()) if fin.size else 0.0)
                old = float(scales[phys, h]) if a > 0 else 0.0
                if not (0.0 < old < math.inf):
                    old = 0.0
                now = max(old, need)
                if a > 0 and now != old:
                    kept = _VALUES[pool[phys, :a, h]] * (old / now)
                    pool[phys, :a, h] = encode(kept)
                if now > 0:
                    pool[phys, a:z, h] = encode(v / now)
                else:
                    pool[phys, a:z, h] = encode(np.where(np.isfinite(v), 0.0 * np.where(np.isfinite(v), v, 0), v))
                scales[phys, h] = now


def values(pool, scales) -> np.ndarray:
    """Decoded values, float64 [n_phys][bs][H][D]."""
    return _VALUES[pool] * np.asarray(scales, dtype=np.float64)[:, None, :, None]


def load(pool, scales, table, ctx, q_start, block_size, pos0=None) -> np.ndarray:
    """Rows of one of K / V in float32 (before the rounding to the output type);
    rows of no sequence are NaN."""
    bs, n = block_size, int(q_start[-1])
    out = np.full((n,) + pool.shape[2:], np.nan, dtype=np.float32)
    for s in range(len(ctx)):
        rows = int(q_start[s + 1] - q_start[s])
        p0 = int(pos0[s]) if pos0 is not None else int(ctx[s]) - rows
        for j in range(rows):
            p = p0 + j
            phys = int(table[s][p // bs]) if 0 <= p < int(ctx[s]) else -1
            r = int(q_start[s]) + j
            if phys < 0 or phys >= pool.shape[0]:
                out[r] = 0.0
            else:
                out[r] = (_VALUES[pool[phys, p % bs]].astype(np.float32)
                          * np.asarray(scales[phys], dtype=np.float32)[:, None])
    return out


def attention(q, k_pool, v_pool, k_scales, v_scales, table, ctx, block_size, scale,
              q_start=None, spans=None, kv_map=None, rows=None):
    """Attention of every query row (or of those in `rows`), float64.

    q [n_tokens][Hq][D]. Without q_start there is one query per sequence, at
    the last position; with it sequence s owns rows q_start[s] .. and its n
    queries are its last n positions, each seeing positions up to its own.
    Returns (out, lse), rows not asked for being NaN."""
    q = np.asarray(q, dtype=np.float64)
    n_tok, hq, d = q.shape
    h_kv, bs = k_pool.shape[2], block_size
    out, lse = np.full(q.shape, np.nan), np.full((n_tok, hq), np.nan)
    starts = np.arange(len(ctx) + 1) if q_start is None else np.asarray(q_start)
    for s in range(len(ctx)):
        c, n = int(ctx[s]), int(starts[s + 1] - starts[s])
        pos = np.array([p for p in range(c) if 0 <= int(table[s][p // bs]) < k_pool.shape[0]],
                       dtype=np.int64)
        phys = np.array([int(table[s][p // bs]) for p in pos], dtype=np.int64)
        k = _VALUES[k_pool[phys, pos % bs]] * np.asarray(k_scales, np.float64)[phys][:, :, None]
        v = _VALUES[v_pool[phys, pos % bs]] * np.asarray(v_scales, np.float64)[phys][:, :, None]
        for j in range(n):
            r = int(starts[s]) + j
            if rows is not None and r not in rows:
                continue
            ok = pos <= c - n + j
            if spans is not None:
                ok = ok & (pos >= spans[r][0]) & (pos < spans[r][1])
            elif kv_map is not None:
                inside = np.zeros(len(pos), dtype=bool)
                for a, ln in kv_map[r]:
                    inside |= (pos >= a) & (pos < int(a) + int(ln))
                ok = ok & inside
            for h in range(hq):
                g = h // (hq // h_kv)
                if not ok.any():
                    out[r, h], lse[r, h] = 0.0, -math.inf
                    continue
                t = scale * (k[ok, g] @ q[r, h])
                m = t.max()
                e = np.exp(t - m)
                out[r, h] = (e @ v[ok, g]) / e.sum()
                lse[r, h] = m + math.log(e.sum())
    return out, lse
