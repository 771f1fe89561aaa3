"""fp64 / integer oracle of a step that verifies drafted trees and of the blocks that requests
hold.  Plain numpy loops from the definitions in include/sfa.h; shares no code with the library."""
from __future__ import annotations

import numpy as np

D_QK, D_V = 576, 512


def tree_plan(parents, start, cached, max_nodes):
    """(mask, positions): lists of ints, the mask of a token as one whole number."""
    mask, pos = [0] * len(parents), [-1] * len(parents)
    for b in range(len(cached)):
        for i in range(min(start[b + 1] - start[b], max_nodes)):
            j, depth = i, -1
            while j >= 0:
                mask[start[b] + i] |= 1 << j
                depth += 1
                up = parents[start[b] + j]
                j = up if -1 <= up < j else -1
            pos[start[b] + i] = max(cached[b], 0) + depth
    return mask, pos


def mask_words(mask, words):
    """[T, words] int64 of whole numbers."""
    out = np.zeros((len(mask), words), np.uint64)
    for t, m in enumerate(mask):
        for w in range(words):
            out[t, w] = (m >> (64 * w)) & (2 ** 64 - 1)
    return out.view(np.int64)


def decode_tree(q, kv, table, cached, start, mask, scale, max_nodes):
    """out [T, h, 512], lse [T, h], and for bounds sum_p w_p |v_p| [T, h, 512] and max_p scale *
    sum |q k_p| [T, h], in fp64; NaN in rows of padding tokens.  q, kv float64, mask whole numbers."""
    T, h, _ = q.shape
    bs = kv.shape[1]
    out, lse = np.full((T, h, D_V), np.nan), np.full((T, h), np.nan)
    wabs, smax = np.zeros((T, h, D_V)), np.zeros((T, h))
    for b in range(len(cached)):
        c, n = max(int(cached[b]), 0), min(int(start[b + 1] - start[b]), max_nodes)
        for i in range(n):
            t = int(start[b]) + i
            seen = list(range(c)) + [c + j for j in range(n) if mask[t] >> j & 1]
            rows = [(int(table[b, p // bs]), p % bs) for p in seen]
            rows = [r for r in rows if 0 <= r[0] < kv.shape[0]]
            if not rows:
                out[t], lse[t] = 0.0, -np.inf
                continue
            k = kv[[r[0] for r in rows], [r[1] for r in rows]]
            s = scale * (q[t] @ k.T)
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(axis=1, keepdims=True)
            w, v = e / z, k[:, :D_V]
            out[t], lse[t] = w @ v, (m + np.log(z))[:, 0]
            wabs[t] = w @ np.abs(v)
            smax[t] = abs(scale) * (np.abs(q[t]) @ np.abs(k).T).max(axis=1)
    return out, lse, wabs, smax


def tree_accept(tokens, targets, parents, start, cached, max_nodes):
    """(path, accepted, next_tokens, seq_lens)."""
    B = len(cached)
    path = np.full((B, max_nodes), -1, np.int64)
    acc, nxt, lens = [], [], []
    for b in range(B):
        a, n = start[b], min(start[b + 1] - start[b], max_nodes)
        cur, k, want = (0 if n else -1), 0, -1
        while cur >= 0:
            path[b, k] = cur
            k += 1
            want = targets[a + cur]
            found = [j for j in range(cur + 1, n) if parents[a + j] == cur and tokens[a + j] == want]
            cur = found[0] if found else -1
        acc.append(k)
        nxt.append(want)
        lens.append(max(cached[b], 0) + k)
    return path, np.array(acc), np.array(nxt), np.array(lens)


def kv_commit(kv, table, cached, path, accepted):
    """kv [num_blocks, block_size, cols] (any values) with the accepted rows in place, a new array."""
    kv, bs = kv.copy(), kv.shape[1]
    for b in range(len(cached)):
        c = max(int(cached[b]), 0)
        place = lambda p: (int(table[b, p // bs]), p % bs)  # noqa: E731
        old = [kv[place(c + int(x))].copy() for x in path[b, :accepted[b]]]
        for k, row in enumerate(old):
            kv[place(c + k)] = row
    return kv


def blocks_fork(table, lens, src, dst, shares, free, taken, bs):
    """(table, lens, shares, copies, taken)."""
    table, lens, shares = np.array(table), np.array(lens), np.array(shares)
    copies, head = [], int(taken)
    for a, d in zip(src, dst):
        if a < 0 or d < 0 or a >= len(table) or d >= len(table) or a == d:
            copies.append([-1] * 3)
            continue
        full, rows = divmod(int(lens[a]), bs)
        table[d, :full] = table[a, :full]
        for x in table[a, :full]:
            shares[x] += 1
        c = [-1] * 3
        if rows:
            new = int(free[head]) if head < len(free) else -1
            head += 1
            table[d, full] = new
            if new >= 0:
                c = [int(table[a, full]), new, rows]
        copies.append(c)
        lens[d] = lens[a]
    return table, lens, shares, np.array(copies).reshape(-1, 3), min(head, max(len(free), int(taken)))


def blocks_free(table, held, keep, shares, free, taken, bs):
    """(shares, free, taken)."""
    shares, free, order, times = np.array(shares), np.array(free), [], {}
    for r in range(len(table)):
        for j in range(-(-max(int(keep[r]), 0) // bs), -(-max(int(held[r]), 0) // bs)):
            if j < table.shape[1] and 0 <= table[r, j] < len(shares):
                x = int(table[r, j])
                if x not in times:
                    order.append(x)
                times[x] = times.get(x, 0) + 1
    gone = [x for x in order if times[x] > shares[x]]
    for x in order:
        shares[x] = max(shares[x] - times[x], 0)
    for k, x in enumerate(gone):
        if taken - len(gone) + k >= 0:
            free[taken - len(gone) + k] = x
    return shares, free, max(taken - len(gone), 0)


def blocks_compact(table, lens, shares, free, taken, bs, max_moves):
    """(table, shares, free, copies)."""
    table, old, shares, free = np.array(table), np.array(shares), np.array(shares), np.array(free)
    places = [(r, j) for r in range(len(table)) for j in range(min(-(-max(int(lens[r]), 0) // bs), table.shape[1]))]
    held = {int(table[p]) for p in places if 0 <= table[p] < len(shares)}
    rest = {int(x) for x in free[taken:] if 0 <= x < len(shares)} - held
    move = {}
    for lo, hi in zip(sorted(rest), sorted(held, reverse=True)):
        if lo < hi and len(move) < max_moves:
            move[hi] = lo
    for p in places:
        table[p] = move.get(int(table[p]), table[p])
    for hi, lo in move.items():
        shares[lo], shares[hi] = old[hi], 0
    now = sorted((rest - set(move.values())) | set(move))
    free[taken:] = -1
    free[taken:taken + len(now)] = now
    copies = np.full((max_moves, 3), -1)
    for k, (hi, lo) in enumerate(move.items()):
        copies[k] = hi, lo, bs
    return table, shares, free, copies


def copy_blocks(kv, copies):
    """kv [..., num_blocks, block_size, cols] after the copies, a new array."""
    kv = kv.copy()
    for a, d, n in copies:
        if a >= 0:
            kv[..., d, :n, :] = kv[..., a, :n, :]
    return kv
