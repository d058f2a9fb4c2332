"""Plain fp64 restatement of the 8-bit key/value cache (test infrastructure only): page
tables from request lengths, quantising rows into e4m3 codes with block scales, and the
verification attention over them. Shares nothing with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

PAGE = 128
LEAST = 2.0 ** -100

# value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff NaN
E4M3 = np.array([math.nan if c & 127 == 127 else
                 (-1.0) ** (c >> 7) * (math.ldexp(c & 7, -9) if c >> 3 & 15 == 0
                                       else math.ldexp(8 + (c & 7), (c >> 3 & 15) - 10)) for c in range(256)])


def encode(v):
    """e4m3 codes of fp64 values: round to nearest even, saturating; NaN -> 0x7f."""
    v = np.asarray(v, np.float64)
    grid = E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    a = np.minimum(np.abs(v), 448.0)
    code = np.searchsorted(mid, a)                   # values at a midpoint so far go to the lower code
    tie = (code < 126) & (a == mid[np.minimum(code, 125)]) & (code % 2 == 1)
    code = (code + tie) | (np.signbit(v) * 128)
    return np.where(np.isnan(v), 0x7f, code).astype(np.uint8)


def least_scale(a):
    """The least power of two s >= 2^-100 with a <= 448 s."""
    if a <= 448 * LEAST:
        return LEAST
    m, e = math.frexp(a / 448)                       # exact ties: a = 448 * 2^k gives m = 0.5
    return math.ldexp(1.0, e - 1 if m == 0.5 else e)


def write_block(rows, row, codes, scale):
    """Quantise rows [n][dh] into places row.. of one block's codes [sb][dh], in place;
    returns the block's new scale. Quotients are fp32 numbers before they become codes."""
    a = np.abs(rows[np.isfinite(rows)])
    need = least_scale(float(a.max()) if a.size else 0.0)
    new = need if row == 0 else max(scale, need)
    if row and new > scale:
        codes[:row] = encode(E4M3[codes[:row]].astype(np.float32) * (np.float32(scale) / np.float32(new)))
    codes[row:row + len(rows)] = encode(rows.astype(np.float32) / np.float32(new))
    return new


def append(rows, slots, codes, scale, sb):
    """Rows [T][Hkv][dh] to slots; codes [pages][Hkv][tokens][dh], scale [pages][Hkv][blocks], in place."""
    tokens, pool = codes.shape[2], codes.shape[0] * codes.shape[2]
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0 or s >= pool:
            t += 1
            continue
        page, off = divmod(s, tokens)
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (off + n) % sb and off + n < tokens:
            n += 1
        blk, row = off // sb, off % sb
        for h in range(codes.shape[1]):
            scale[page, h, blk] = write_block(rows[t:t + n, h], row, codes[page, h, blk * sb:(blk + 1) * sb], scale[page, h, blk])
        t += n


def commit(cand, prefix, best, n_out, Dmax, codes, scale, sb, table=None):
    """The accepted candidates' rows [B][NT][Hkv][dh] behind each prefix; returns (new_len, ok)."""
    tokens = codes.shape[2]
    new, ok = prefix.copy(), np.ones(len(prefix), bool)
    for b in range(len(prefix)):
        a = int(n_out[b]) - 1 if best[b] >= 0 else 0
        P = int(prefix[b])
        NB = cand.shape[1] // Dmax
        room = tokens if table is None else table.shape[1] * PAGE
        if best[b] >= NB or a > Dmax or P < 0 or (a > 0 and P + a > room):
            ok[b] = False
            continue
        if a <= 0:
            continue
        pos = np.arange(P, P + a)
        page = np.full(a, b) if table is None else table[b, pos // PAGE]
        if (page < 0).any() or (page >= len(codes)).any():
            ok[b] = False
            continue
        first = best[b] * Dmax
        append(cand[b, first:first + a], page * tokens + pos % tokens, codes, scale, sb)
        new[b] = P + a
    return new, ok


def page_tables(cur, add, held, table, stack, n_free, cap):
    """Tables of exactly ceil((cur + add) / 128) pages; stack: int array whose first n_free
    entries are free. Updates held, table and stack in place; returns (n_free, row_start,
    slot_map, served, error)."""
    B, pps = table.shape
    err, n = False, int(n_free)
    if n < 0 or n > len(stack):
        err, n = True, min(max(n, 0), len(stack))
    want = [-(-(int(c) + int(a)) // PAGE) for c, a in zip(cur, add)]
    ok = [cur[b] >= 0 and add[b] >= 0 and want[b] <= pps and 0 <= held[b] <= pps for b in range(B)]
    err |= not all(ok)
    for b in range(B):
        if ok[b]:
            for j in range(want[b], held[b]):
                if n < len(stack):
                    stack[n] = table[b, j]
                    n += 1
                else:
                    err = True
                table[b, j] = -1
            held[b] = min(held[b], want[b])
    served, stuck = np.zeros(B, np.int32), False
    for b in range(B):
        lack = want[b] - held[b] if ok[b] else 0
        if lack > 0 and (stuck or lack > n):
            stuck = True
        elif ok[b]:
            served[b] = 1
            for _ in range(lack):
                n -= 1
                table[b, held[b]] = stack[n]
                held[b] += 1
    start = np.concatenate([[0], np.cumsum(np.maximum(add, 0))]).astype(np.int32)
    slots = np.full(cap, -1, np.int32)
    err |= start[-1] > cap
    for b in range(B):
        if served[b]:
            for i in range(int(add[b])):
                if start[b] + i < cap:
                    p = int(cur[b]) + i
                    slots[start[b] + i] = table[b, p // PAGE] * PAGE + p % PAGE
    return n, start, slots, served, err


def values(codes, scale, sb, prefix, table=None):
    """The cached rows [Hkv][prefix][dh] of each sequence, as fp64 (a list over sequences)."""
    out = []
    for b, P in enumerate(prefix):
        pages = [b] if table is None else table[b, :-(-int(P) // PAGE)]
        parts = [E4M3[codes[p]] * np.repeat(scale[p].astype(np.float64), sb, 1)[:, :codes.shape[2], None] for p in pages]
        out.append(np.concatenate(parts, 1)[:, :P] if parts else np.zeros((codes.shape[1], 0, codes.shape[3])))
    return out


def attention(q, k, v, k_cand, v_cand, blk_len, Dmax, slots=None, scale=None, probs=None):
    """Verification attention of the present tokens over cached rows k, v (from values()), all
    fp64. Returns {(b, t): (out [Hq][dh], spread [Hq][dh])}, where spread is
    sum_j p_j |v_j|, the size that relative errors of the probabilities act on. A dict `probs`
    receives {(b, t): [(p [G][keys], v [keys][dh]) for each kv head]}."""
    B, NT, Hq, dh = q.shape
    Hkv = k_cand.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(dh) if scale is None else scale
    res = {}
    for b in range(B):
        for t in range(NT):
            blk, d = divmod(t, Dmax)
            if d >= blk_len[b, blk] or (slots is not None and (b, t) not in slots):
                continue
            own = slice(blk * Dmax, t + 1)
            out, size = np.empty((Hq, dh)), np.empty((Hq, dh))
            for h in range(Hkv):
                kk = np.concatenate([k[b][h], k_cand[b, own, h]])
                vv = np.concatenate([v[b][h], v_cand[b, own, h]])
                z = q[b, t, h * G:(h + 1) * G] @ kk.T * scale
                e = np.exp(z - z.max(1, keepdims=True))
                p = e / e.sum(1, keepdims=True)
                out[h * G:(h + 1) * G] = p @ vv
                size[h * G:(h + 1) * G] = p @ np.abs(vv)
                if probs is not None:
                    probs.setdefault((b, t), []).append((p, vv))
            res[b, t] = (out, size)
    return res
