"""Plain 64-bit numpy implementations the operator tests compare with.

Written from the definitions in ``include/yoco_kv.h`` alone, request by
request; they share no code with the library or with the C oracle.
"""
from __future__ import annotations

import math

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------- page tables

def build_block_tables(table, seq_lens, qsl, num_tokens, num_blocks, bs, free=None, num_free=0):
    """(table, slots, num_free_after, error bits) for well-formed or odd lengths."""
    table = np.array(table, copy=True)
    R, width = table.shape
    slots = np.full(num_tokens, -1, dtype=np.int64)
    bits = 0
    cap = 0 if free is None else len(free)
    avail = min(max(num_free, 0), cap)
    if free is not None and avail != num_free:
        bits |= 0x8
    demand = taken = 0
    for r in range(R):
        q0, q1, seq = int(qsl[r]), int(qsl[r + 1]), int(seq_lens[r])
        if q0 < 0 or q1 < q0 or q1 > num_tokens:
            bits |= 0x8
            continue
        q = q1 - q0
        if q == 0:
            continue
        need = -(-seq // bs) if seq > 0 else 0
        if seq < q or need > width:
            bits |= 0x2
            continue
        held = -(-(seq - q) // bs) if free is not None else need
        before, demand = demand, demand + need - held
        if need > held and demand > avail:
            bits |= 0x80
            continue
        taken = max(taken, demand if need > held else 0)
        for n, lp in enumerate(range(held, need)):
            page = int(free[avail - 1 - before - n])
            table[r, lp] = page if 0 <= page < num_blocks else -1
        for j in range(q):
            p = seq - q + j
            page = int(table[r, p // bs])
            if 0 <= page < num_blocks:
                slots[q0 + j] = page * bs + p % bs
            else:
                bits |= 0x1
    return table, slots, avail - taken, bits


# ---------------------------------------------------------- the 4-bit format

def e2m1_encode(x):
    """[..., D] float -> (codes [..., D], scale bytes [..., D / 32]), the append's rule."""
    x = np.asarray(x, dtype=np.float64)
    big = float.fromhex("0x1.fep127")  # largest finite bf16
    x = np.where(np.isnan(x), np.copysign(big, x), np.clip(x, -big, big))
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(g).max(-1)
    b = np.ones(top.shape, dtype=np.int64)
    while True:  # the smallest byte whose scale covers the block
        more = (top > 6.0 * np.ldexp(1.0, b - 127)) & (b < 251)
        if not more.any():
            break
        b[more] += 1
    a = np.abs(np.ldexp(g, (127 - b)[..., None]))
    d = np.abs(a[..., None] - LEVELS)
    d[..., 1::2] += 1e-12 * (d[..., 1::2] > 0)  # ties go to the even code (values are far coarser)
    code = d.argmin(-1) + 8 * np.signbit(g)
    return code.reshape(x.shape).astype(np.uint8), b.astype(np.uint8)


def e2m1_pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def e2m1_values(packed, b):
    """Packed codes [..., D / 2] and scale bytes [..., D / 32] -> float64 [..., D]."""
    code = np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    mag = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    g = mag.reshape(*mag.shape[:-1], -1, 32)
    return np.ldexp(g, (b.astype(np.int64) - 127)[..., None]).reshape(mag.shape)


# ---------------------------------------------------------------- attention

def cross_attn_e2m1(q, k_cache, v_cache, scales, table, seq_lens, cqsl, scale, max_rows):
    """(out, tolerance) [rows, H_q, D]; rows without keys are zero.

    The tolerance counts, element by element, what the documented arithmetic
    may lose: half a bf16 step of the output (2^-8), half an f16 step of every
    weight (2^-11 of sum p |v|), and the fp32 sums of the scores (each product
    or sum 2^-24 of the magnitudes summed, D + 64 of them, then exp).

    f16 has an absolute step below 2^-14, half of it 2^-25, which a relative
    step does not count. The weights are held as 2^3 p or more (relative to a
    reference at most the largest score), so each is off by up to 2^-28 as
    well: 2^-28 of sum |v|. Times its token's scale over the largest scale
    times 2^7 it may fall below 2^-14 once more: off by 2^-25 in units of
    2^(top - 127 - 10), that is 2^-35 of the largest scale, for each of the
    keys with codes up to 6.
    """
    rows = min(int(cqsl[-1]), max_rows)
    H_q, D = q.shape[1:]
    H = k_cache.shape[1]
    G, bs = H_q // H, k_cache.shape[2]
    out, tol = np.zeros((rows, H_q, D)), np.zeros((rows, H_q, D))
    for r in range(len(seq_lens)):
        c0, c1, seq = int(cqsl[r]), int(cqsl[r + 1]), int(seq_lens[r])
        n = min(seq, table.shape[1] * bs)
        if c1 <= c0 or n <= 0:
            continue
        pages = table[r, : -(-n // bs)]
        for h in range(H):
            k = e2m1_values(k_cache[pages, h], scales[pages, h, 0]).reshape(-1, D)
            v = e2m1_values(v_cache[pages, h], scales[pages, h, 1]).reshape(-1, D)
            for row in range(c0, min(c1, rows)):
                keys = min(seq - (c1 - c0) + (row - c0) + 1, n)
                if keys <= 0:
                    continue
                qq = q[row, h * G:(h + 1) * G].astype(np.float64)
                s = qq @ k[:keys].T * scale
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ v[:keys]
                mags = (np.abs(qq) @ np.abs(k[:keys]).T * scale).max(-1, keepdims=True)
                ds = (D + 64) * 2.0 ** -24 * mags + np.abs(s).max(-1, keepdims=True) * 2.0 ** -22 + 2.0 ** -20
                at = slice(h * G, (h + 1) * G)
                out[row, at] = o
                tol[row, at] = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.2 * ds) * (p @ np.abs(v[:keys]))
                top = np.ldexp(1.0, int(scales[pages, h, 1].reshape(-1, D // 32)[:keys].max()) - 127)
                tol[row, at] += 2.0 ** -28 * np.abs(v[:keys]).sum(0) + 2.0 ** -35 * 6 * keys * top + 1e-30
    return out, tol


# ---------------------------------------------------------------- retention

def retention(q, k, v, log_decay, state, where, qsl, seq_lens, scale):
    """Token by token in 64 bits: (out [T, H, D], states after [R, H, D, D])."""
    T, H, D = q.shape
    G = H // k.shape[1]
    g = np.broadcast_to(np.asarray(log_decay, np.float64), (T, H))
    out = np.zeros((T, H, D))
    after = []
    for r in range(len(seq_lens)):
        a, b = int(qsl[r]), int(qsl[r + 1])
        s = np.array(state[where[r]], dtype=np.float64)
        if int(seq_lens[r]) <= b - a:
            s = np.zeros_like(s)
        for t in range(a, b):
            kk, vv = (np.repeat(x[t].astype(np.float64), G, 0) for x in (k, v))
            s = np.exp(g[t])[:, None, None] * s + kk[:, :, None] * vv[:, None, :]
            out[t] = scale * np.einsum("hk,hkv->hv", q[t].astype(np.float64), s)
        after.append(s)
    return out, after


def log2_steps(n):
    return max(1, math.ceil(math.log2(max(n, 2))))
