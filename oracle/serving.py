"""fp64 / integer oracle of the calls around decode over an 8-bit latent cache: the step
plan, rotary positions, the quantising cache write and decode_q8.  Plain numpy loops from
the definitions in include/sfa.h; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np

D_QK, D_V = 576, 512
MIN_EXP, MAX_EXP = -100, 120


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3 (1 sign, 4 exponent bits of bias 7, 3 mantissa bits; no
    infinities, 0x7f and 0xff are NaN)."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            x = math.nan
        v[code] = -x if code & 128 else x
    return v


E4M3 = e4m3_values()
_POS = E4M3[:127]          # non-negative finite values, ascending with their code


def to_e4m3(x) -> np.ndarray:
    """Codes of x rounded to nearest, ties to the even code; beyond 448 saturates, an
    infinity or NaN gives NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = np.abs(_POS[hi] - a), np.abs(a - _POS[lo])
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isfinite(x), code, 127).astype(np.uint8)
    return code | np.where(np.signbit(x), 128, 0).astype(np.uint8)


def bf16_values(bits) -> np.ndarray:
    return (np.asarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def scale_exponent(row) -> int:
    """Least k with amax / 2^k <= 448 over the row's finite values, in [MIN_EXP, MAX_EXP]."""
    fin = np.abs(row[np.isfinite(row)])
    amax = float(fin.max()) if fin.size else 0.0
    k = MIN_EXP
    while k < MAX_EXP and amax > 448.0 * 2.0 ** k:
        k += 1
    return k


def kv_write_q8(codes, scales, slots, rows, group):
    """codes uint8 [num_slots, 576], scales float64 [num_slots / group], rows float64 [T, 576]:
    the cache after the write, as new arrays."""
    codes, scales = codes.copy(), scales.copy()
    members = {}
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0]:
            members.setdefault(int(s) // group, []).append(t)
    for g, ts in members.items():
        mine = {int(slots[t]) for t in ts}
        before = 0.0 if g * group in mine else float(scales[g])
        if not (before > 0.0 and math.isfinite(before)):
            before = 0.0
        after = max([before] + [2.0 ** scale_exponent(rows[t]) for t in ts])
        if 0.0 < before < after:
            for s in range(g * group, (g + 1) * group):
                codes[s] = to_e4m3(E4M3[codes[s]] * (before / after))
        for t in ts:
            codes[int(slots[t])] = to_e4m3(rows[t] / after)
        scales[g] = after
    return codes, scales


def decode_q8(q, codes, scales, group, block_table, seq_lens, topk_idx, scale, Q=1, n_splits=1, interleave=0,
              bt_per_token=False):
    """Shard partials (out [n, T, h, 512], lse [n, T, h]) in fp64 and, for bounds, sum_j w_j |v_j|
    and max_j(w_j c_j) * sum_j |e_j|, both [n, T, h, 512] (w the softmax weights, v = c e with c
    a row's scale and e its e4m3 values).  q float64
    [T, h, 576], codes uint8 [num_blocks, block_size, 576], scales float64 [num_blocks, groups]."""
    T, h, _ = q.shape
    bs = codes.shape[1]
    out = np.zeros((n_splits, T, h, D_V))
    lse = np.full((n_splits, T, h), -np.inf)
    wabs, wmax = np.zeros_like(out), np.zeros_like(out)
    for t in range(T):
        b = t // Q
        S = int(seq_lens[b])
        L = S - (Q - 1 - t % Q)
        c = -(-S // n_splits) if S > 0 else 0
        for r in range(n_splits):
            rows, sc = [], []
            for p in topk_idx[t]:
                p = int(p)
                if not 0 <= p < L:
                    continue
                if n_splits > 1 and ((p // interleave) % n_splits if interleave > 0 else p // c) != r:
                    continue
                blk = int(block_table[t if bt_per_token else b][p // bs])
                rows.append(codes[blk, p % bs])
                sc.append(scales[blk, (p % bs) // group])
            if not rows:
                continue
            e4, c4 = E4M3[np.array(rows)], np.array(sc)
            k = e4 * c4[:, None]
            s = scale * (q[t] @ k.T)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(axis=1, keepdims=True)
            w = e / z
            v = k[:, :D_V]
            out[r, t] = w @ v
            lse[r, t] = (m + np.log(z))[:, 0]
            wabs[r, t] = w @ np.abs(v)
            wmax[r, t] = (w * c4).max(axis=1)[:, None] * np.abs(e4[:, :D_V]).sum(axis=0)[None, :]
    return out, lse, wabs, wmax


def step_plan(cached, new, table, free, taken, bs, num_tokens):
    """(table, seq_lens, token_start, positions, slots, taken), lists and arrays of ints."""
    table = np.array(table, dtype=np.int64).copy()
    positions, slots = np.full(num_tokens, -1, np.int64), np.full(num_tokens, -1, np.int64)
    seq, start, i, head = [], [0], 0, int(taken)
    for b, (c, n) in enumerate(zip(cached, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        for k in range(min(-(-c // bs), table.shape[1]), min(-(-(c + n) // bs), table.shape[1])):
            table[b, k] = free[head] if head < len(free) else -1
            head += 1
        for p in range(c, c + n):
            if i < num_tokens:
                positions[i] = p
                blk = table[b, p // bs] if p // bs < table.shape[1] else -1
                slots[i] = blk * bs + p % bs if blk >= 0 else -1
            i += 1
        seq.append(c + n)
        start.append(i)
    return table, np.array(seq), np.array(start), positions, slots, min(head, max(len(free), int(taken)))


def rope(x, positions, inv_freq, interleaved=True, mscale=1.0, inverse=False):
    """x float64 [T, n, width] rotated; rows of negative positions come back as they are."""
    y = np.array(x, dtype=np.float64)
    rot = 2 * len(inv_freq)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for i, f in enumerate(inv_freq):
            a = float(p) * float(f)
            c, s = math.cos(a) * mscale, math.sin(a) * mscale * (-1.0 if inverse else 1.0)
            j0, j1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            u, v = x[t, :, j0], x[t, :, j1]
            y[t, :, j0], y[t, :, j1] = u * c - v * s, u * s + v * c
    return y
