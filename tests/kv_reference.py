"""Plain references for the paged KV cache's tests: numpy in 64 bits, one loop
per thing that the definition loops over.  TEST INFRASTRUCTURE ONLY."""
import math

import numpy as np

from oracle import nvfp4_oracle as O

E4M3 = O.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)  # 0x7F and 0xFF are NaN

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a rounding, relative to the value


def block_table(cached, new, page, free, used, table, max_tokens):
    """(slots, lens, starts, first, used, table) by serving the requests one after another."""
    table = np.array(table, np.int64)
    slots = np.full(max_tokens, -1, np.int64)
    lens, starts, first = [], [], []
    used = max(int(used), 0)
    wanted, at = used, 0  # free pages asked for and tokens placed so far, served or not
    taken = used
    for r, (c, n) in enumerate(zip(map(int, cached), map(int, new))):
        starts.append(min(at, max_tokens))
        begin, at = at, at + max(n, 0)
        held, total = -(-c // page), -(-(c + n) // page)
        if c < 0 or n < 0 or total > table.shape[1] or at > max_tokens:
            lens.append(c)
            first.append(-1)
            continue
        need = total - held
        if need and wanted + need > len(free):
            wanted += need
            lens.append(c)
            first.append(-1)
            continue
        first.append(min(wanted, len(free)))
        lens.append(c + n)
        table[r, held:total] = free[wanted:wanted + need]
        wanted += need
        if need:
            taken = wanted
        for i in range(n):
            slot = table[r, (c + i) // page] * page + (c + i) % page
            slots[begin + i] = slot if table[r, (c + i) // page] >= 0 and slot < 2 ** 31 else -1
    starts.append(min(at, max_tokens))
    return slots, np.array(lens), np.array(starts), np.array(first), taken, table


def rope(x, positions, inv_freq, axes, adjacent):
    """x [tokens, heads, dim] float64 -> (turned, bound on the 32-bit arithmetic's error)."""
    x = np.asarray(x, np.float64)
    pairs = len(inv_freq)
    angle = positions.astype(np.float64)[axes].T * inv_freq.astype(np.float64)
    cos, sin = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    a = x[..., 0:2 * pairs:2] if adjacent else x[..., :pairs]
    b = x[..., 1:2 * pairs:2] if adjacent else x[..., pairs:2 * pairs]
    y, slack = x.copy(), np.zeros_like(x)
    size = np.abs(a) + np.abs(b)
    for to, v in ((0, a * cos - b * sin), (1, b * cos + a * sin)):
        at = slice(to, 2 * pairs, 2) if adjacent else slice(to * pairs, (to + 1) * pairs)
        y[..., at] = v
        # sine and cosine: 2 steps of their own and pi 2^-25 from their argument's rounding, 4 in all at 2^-24;
        # a product and the sum: one each
        slack[..., at] = 6 * 2.0 ** -24 * size
    return y, slack


def attention(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale, window, num_pages):
    """(out, lse, reach, sharp): float64 results; sum_j p_j |v_j| for each output, and for each row how far a
    score may be off by 32-bit sums, relative to e^score."""
    n, heads, dim = q.shape
    kv_heads, page = k_cache.shape[1], k_cache.shape[2]
    group = heads // kv_heads
    out, reach = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse, sharp = np.full((n, heads), -math.inf), np.zeros((n, heads))
    q = q.astype(np.float64)
    for r in range(n):
        length = min(max(int(lens[r]), 0), table.shape[1] * page)
        low = max(0, length - window) if window else 0
        at = np.arange(low, length)
        ids = table[r][at // page]
        at, ids = at[(ids >= 0) & (ids < num_pages)], ids[(ids >= 0) & (ids < num_pages)]
        if not len(at):
            continue
        for h in range(kv_heads):
            k = E4M3[k_cache[ids, h, at % page]] / float(k_scale)
            v = E4M3[v_cache[ids, h, at % page]] / float(v_scale)
            rows = slice(h * group, (h + 1) * group)
            s = q[r, rows] @ k.T * scale
            top = s.max(-1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(-1, keepdims=True)
            out[r, rows] = p @ v / total
            reach[r, rows] = p @ np.abs(v) / total
            lse[r, rows] = (top + np.log(total))[:, 0]
            sharp[r, rows] = ((dim + 8) * 2.0 ** -24 * (np.abs(q[r, rows]) @ np.abs(k).T).max(-1) * scale)
    return out, lse, reach, sharp


def attention_bounds(out, lse, reach, sharp, lens, dtype):
    """How far the kernel may be from the reference.

    A score is off by at most `sharp` (sums of dim + 8 roundings), and by 2^-22 relative to its exponential for
    the exponent's argument and the exponential itself, so each probability by e = sharp + 2^-22.  A probability
    meets v as fp16, 2^-11 off (two parts of it, fp16 and float32 outputs: 2^-22).  The sums over tokens run in
    32 bits: one rounding a tile of 32 tokens, 32 in a tile's product, and some thirty where partial results are
    joined.  Numerator and denominator each, and the output's own rounding."""
    sums = np.maximum(np.asarray(lens, np.float64), 0)[:, None] / 16 + 64
    e = sharp + 2.0 ** -22 + sums * 2.0 ** -24
    p = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    b_out = HALF_STEP[dtype] * 1.01 * np.abs(out) + (2 * e + p)[..., None] * reach + 2.0 ** -25 * (dtype == "f16")
    with np.errstate(invalid="ignore"):
        b_lse = e + 2.0 ** -22 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 12)
    return b_out, b_lse
