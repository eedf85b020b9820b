"""Plain CPU oracle for the K/V cache in 8 bits: attention over it, the insert
into it, and the batch's index arrays.

TEST INFRASTRUCTURE ONLY.  Only the test-suite may import this module.  It
shares no code with the CUDA library and imports nothing from it.

The cache holds K and V as e4m3 codes with one scale for each (page, KV head),
value = code * scale.  Everything here is float64 arithmetic (numpy) or plain
Python integers, straight from the definitions:

* attention: softmax(scale * q . k) v over the keys j <= p of a row's selected
  blocks, plus the log of the softmax's sum;
* insert: RMSNorm and rotary embedding (oracle/qk_rope_insert.py), then the
  page's scale (the least power of two that holds the largest finite new value
  in +-448, or the old scale where the page goes on and that is enough) and the
  values before their rounding to codes;
* advance: pages taken from the head of a ring of free pages and given back at
  its tail, in the order of (sequence, block).
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import fp8_cache as F
from . import qk_rope_insert as R

BLOCK = 128
E4M3_MAX = 448.0


def values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """codes uint8 [pages][Hkv][128][D], scale [pages][Hkv] -> float64 values."""
    return F.decode_bits(codes) * np.asarray(scale, dtype=np.float64)[:, :, None, None]


def attention(q, k, v, seq, pos, sel, page_table, softmax_scale: Optional[float] = None):
    """q [T][Hq][D]; k, v: values [pages][Hkv][128][D]; seq, pos [T]; sel [T][Hkv][topk].
    Returns (out [T][Hq][D], lse [T][Hq], mean_abs [T][Hq][D]): mean_abs is the softmax's mean of |v|,
    the size that errors of the probabilities act on."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    c = 1.0 / math.sqrt(D) if softmax_scale is None else softmax_scale
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    for t in range(T):
        for g in range(Hkv):
            ks, vs = [], []
            for b in sel[t][g]:
                if b < 0:
                    continue
                n = min(BLOCK, int(pos[t]) - int(b) * BLOCK + 1)
                page = int(page_table[int(seq[t])][int(b)])
                ks.append(k[page, g, :n])
                vs.append(v[page, g, :n])
            if not ks:
                continue
            kk, vv = np.concatenate(ks), np.concatenate(vs)
            h = slice(g * G, (g + 1) * G)
            x = c * (q[t, h] @ kk.T)
            m = x.max(axis=1, keepdims=True)
            p = np.exp(x - m)
            s = p.sum(axis=1, keepdims=True)
            out[t, h] = p @ vv / s
            mag[t, h] = p @ np.abs(vv) / s
            lse[t, h] = (m + np.log(s))[:, 0]
    return out, lse, mag


def block_scale(a: float) -> float:
    """The least power of two s, 2^-126 at least, with 448 s >= a."""
    s = 2.0 ** -126
    while E4M3_MAX * s < a:
        s *= 2.0
    return s


def insert(q, k_new, v_new, q_w, k_w, seq, pos, page_table, k_codes, v_codes, k_scale, v_scale, rotary_dim=64,
           theta=10000.0, eps=1e-6):
    """Returns (q_out, k, v): q_out float64; k, v each (target, scale, kind): the whole cache as the float64 values that
    its codes should round to, in units of the page's new scale; the new scales; and, for each cache row, kind 0 =
    untouched, 1 = an older row rounded again, 2 = new."""
    pos = np.asarray(pos)
    q_out = R.rope_partial(R.rms_norm_heads(q, q_w, eps), pos, rotary_dim, theta)
    results = []
    for x, codes, scale in ((R.rope_partial(R.rms_norm_heads(k_new, k_w, eps), pos, rotary_dim, theta), k_codes, k_scale),
                            (R._f64(v_new), v_codes, v_scale)):
        target = F.decode_bits(codes).copy()
        new_scale = np.asarray(scale, dtype=np.float64).copy()
        kind = np.zeros(target.shape[:3], dtype=np.int64)
        rows = {}
        for t in range(len(pos)):
            rows.setdefault(int(page_table[int(seq[t])][int(pos[t]) // BLOCK]), []).append(t)
        for page, ts in rows.items():
            first = min(int(pos[t]) % BLOCK for t in ts)
            for g in range(target.shape[1]):
                y = np.stack([x[t, g] for t in ts])
                a = float(np.max(np.where(np.isfinite(y), np.abs(y), 0.0)))
                old = float(new_scale[page, g])
                held = old if 0 < old < np.inf else 0.0
                grown = first == 0 or held == 0.0 or a > E4M3_MAX * held
                s = block_scale(a) if grown else old
                if grown and first > 0:
                    target[page, g, :first] *= held / s
                    kind[page, g, :first] = 1
                for t, row in zip(ts, y):
                    target[page, g, int(pos[t]) % BLOCK] = row / s
                    kind[page, g, int(pos[t]) % BLOCK] = 2
                new_scale[page, g] = s
        results.append((target, new_scale, kind))
    return q_out, results[0], results[1]


def advance(delta: Sequence[int], ctx: Sequence[int], table: List[List[int]], ring: List[int], pool: Sequence[int],
            max_rows: int) -> Tuple:
    """Returns (ctx, table, ring, pool, q_start, slot_map) after the step; the inputs are not changed."""
    table, ring, ctx = [list(r) for r in table], list(ring), list(ctx)
    width, P, (head, count) = len(table[0]), len(ring), pool[:2]
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    after = [c + d for c, d in zip(ctx, delta)]
    rows = sum(max(0, d) for d in delta)
    need = sum(max(0, blocks(a) - blocks(c)) for a, c in zip(after, ctx)) if min(after) >= 0 else 0
    back = sum(max(0, blocks(c) - blocks(a)) for a, c in zip(after, ctx))
    bad = (not 0 <= head < P or not 0 <= count <= P or min(ctx) < 0 or min(after) < 0 or max(after + ctx) > width * BLOCK
           or rows > max_rows or count + back > P)
    if bad or need > count:
        return ctx, table, ring, [head, count, -1 if bad else need - count, 0], [0] * (len(ctx) + 1), [-1] * max_rows
    taken = freed = 0
    q_start, slots = [0], []
    gone = []
    for s, (c, a) in enumerate(zip(ctx, after)):
        for b in range(blocks(c), blocks(a)):
            table[s][b] = ring[(head + taken) % P]
            taken += 1
        for b in range(blocks(a), blocks(c)):
            gone.append(table[s][b])
        q_start.append(q_start[-1] + max(0, a - c))
        slots += [table[s][p // BLOCK] * BLOCK + p % BLOCK for p in range(c, a)]
    for page in gone:
        ring[(head + count + freed) % P] = page
        freed += 1
    return after, table, ring, [(head + need) % P, count - need + back, 0, rows], q_start, slots + [-1] * (max_rows - rows)
