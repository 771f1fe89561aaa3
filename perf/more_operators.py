"""Cases of speculative steps with a tree of drafted tokens and of the cache's blocks: the
tree's masks and positions, its attention over the paged latent cache, the accepted path and
the move of its rows; forking, freeing and compacting the blocks that requests hold.

Each case names its operator in "op" and carries the sizes.  With `own` false `run` computes
the operator's plain form with elementary torch operations; with `own` true it calls the
package.  `exact` gives the result from the definition in 64 bits (whole numbers by loops).
"""
import math

import torch

own = False

D_QK, D_V = 576, 512          # a latent row: 512 latent + 64 rope columns; V = the first 512


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request, 4 heads, a short context and a handful of drafts: the latency of a call
        dict(name="tree_one", op="decode", B=1, h=4, nodes=6, min_nodes=6, S=200, min_S=200, block_size=64, dtype="fp32"),
        # a verify step of few heads a GPU (the dense workload's 16), ragged long contexts
        dict(name="tree_h16", op="decode", B=64, h=16, nodes=8, min_nodes=2, S=16384, min_S=1000, block_size=64,
             dtype="fp32"),
        # a verify step of all 128 heads, trees of 16: bound by the products
        dict(name="tree_h128", op="decode", B=16, h=128, nodes=16, min_nodes=16, S=8192, min_S=8192, block_size=64,
             dtype="bf16"),
        # two long contexts, odd tree sizes, small blocks
        dict(name="tree_long", op="decode", B=2, h=64, nodes=25, min_nodes=21, S=131072, min_S=100000, block_size=16,
             dtype="bf16"),
        # what a verify step does around its attention, 64 requests with small trees: masks and
        # positions, the drafts' rows into the cache, the accepted path, its rows into place
        dict(name="step_small", op="step", B=64, nodes=8, min_nodes=4, S=1000, block_size=64, hit=0.6),
        # the same of 256 requests with wide trees
        dict(name="step_wide", op="step", B=256, nodes=61, min_nodes=30, S=500, block_size=64, hit=0.8),
        # eight samples forked from one prompt of a single-layer cache, then freed
        dict(name="fork_samples", op="fork", R=1, forks=8, S=1500, min_S=1500, block_size=64, layers=1, dtype="bf16"),
        # beams of many requests over the 8-bit caches of several layers
        dict(name="fork_beams", op="fork", R=128, forks=4, S=6000, min_S=40, block_size=64, layers=6, dtype="e4m3"),
        # a verify step's rejected drafts and finished requests of a running batch
        dict(name="free_step", op="free", R=64, S=8192, block_size=64, finished=0.1, trim=61),
        # a large batch is cancelled, long contexts in small blocks
        dict(name="free_batch", op="free", R=700, S=16384, block_size=16, finished=0.9, trim=61),
        # a small pool, whole
        dict(name="compact_small", op="compact", R=16, S=1000, block_size=64, blocks=512, max_moves=64, layers=1, dtype="bf16"),
        # a fragmented pool of two layers
        dict(name="compact_large", op="compact", R=300, S=2000, block_size=64, blocks=10000, max_moves=4000, layers=2,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "step", "fork", "free", "compact"])
    if op == "decode":
        h = rng.choice([1, 3, 8, 16, 27, 32, 64, 72, 128])
        nodes = _log(rng, 1, 130)
        S = _log(rng, 1, 100000)
        B = max(1, min(_log(rng, 1, 100), 300000000 // (nodes * h * S), 600000 // S))
        low = rng.choice([0, 1])
        return dict(op=op, B=B, h=h, nodes=nodes, min_nodes=rng.choice([nodes, 1, 0]), S=S,
                    min_S=S if low else max(0, S // 16 - 1), block_size=rng.choice([7, 16, 24, 64, 128]),
                    dtype=rng.choice(["fp32", "bf16"]))
    if op == "step":
        B = _log(rng, 1, 400)
        nodes = max(1, min(_log(rng, 1, 130), 16000 // B))
        return dict(op=op, B=B, nodes=nodes, min_nodes=rng.choice([0, 1, nodes]), S=_log(rng, 1, 600),
                    block_size=rng.choice([7, 16, 64, 128]), hit=rng.choice([0.3, 0.6, 0.9]))
    if op == "fork":
        R = _log(rng, 1, 128)
        S = _log(rng, 4, 6000)
        return dict(op=op, R=R, forks=_log(rng, 1, 4 + 128 // R // 4), S=S, min_S=rng.choice([0, S]),
                    block_size=rng.choice([16, 64, 128]), layers=rng.choice([1, 2, 6]), dtype=rng.choice(["bf16", "e4m3"]))
    if op == "free":
        R = _log(rng, 1, 2000)
        return dict(op=op, R=R, S=_log(rng, 16, max(20, min(16384, 10000000 // R))), block_size=rng.choice([16, 24, 64]),
                    finished=rng.choice([0.1, 0.5, 0.9]), trim=_log(rng, 1, 200))
    blocks = _log(rng, 20, 9000)
    bs = rng.choice([16, 64])
    R = _log(rng, 1, 300)
    return dict(op=op, R=R, S=max(1, _log(rng, bs, 2 * bs * blocks // R + bs)), block_size=bs, blocks=blocks,
                max_moves=_log(rng, 1, blocks), layers=rng.choice([1, 2]), dtype=rng.choice(["bf16", "e4m3"]))


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _int(g, lo, hi, shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _spread(g, lo, hi, n):
    """n whole numbers evenly over [lo, hi], in random order: their sum is the case's own."""
    x = [lo + (hi - lo) * (2 * i + 1) // (2 * n) for i in range(n)]
    return _i32(x)[torch.randperm(n, generator=g, device="cuda")]


def _cdiv(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _latent_rows(g, n):
    """Latent rows as they meet a cache: normed latents of about 1, a token's size varying,
    rope columns larger."""
    x = torch.randn((n, D_QK), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))
    x[:, D_V:] *= 2.0
    return x.to(torch.bfloat16)


def _fill(g, blocks, bs):
    kv = torch.empty((blocks, bs, D_QK), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 18) // bs)
    for b0 in range(0, blocks, step):
        nb = min(step, blocks - b0)
        kv[b0:b0 + nb] = _latent_rows(g, nb * bs).view(nb, bs, D_QK)
    return kv


def _paged(g, lens, block_size, most, total):
    """A block table over `total` shuffled physical blocks for sequences of these lengths, at
    most `most`: (table [R, max_blocks] with -1 in unused entries, the blocks that nobody holds)."""
    nblk = _cdiv(lens.long(), block_size)
    width = -(-most // block_size) + 2
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    start = torch.cumsum(nblk, 0) - nblk
    at = (start[:, None] + col[None, :]).clamp(max=total - 1)
    table = torch.where(col[None, :] < nblk[:, None], ids[at], torch.full_like(ids[at], -1))
    return table.contiguous(), ids[int(nblk.sum()):].contiguous()


def _trees(g, n):
    """Parents of drafted trees with n nodes each (n a list): node 0 is the root (the token that
    the step before chose); later nodes hang on one of the nodes before them, by preference a late
    one, as trees that grow level by level do."""
    T = sum(n)
    r = torch.rand((T,), generator=g, device="cuda").cpu().tolist()
    out = []
    for k in n:
        for i in range(k):
            out.append(-1 if i == 0 else min(i - 1, int(i * r[len(out)] ** 0.7)))
    return out


def prepare(case, seed):
    g = _gen(seed)
    op, bs = case["op"], case["block_size"]
    if op in ("decode", "step"):
        B = case["B"]
        lens = _spread(g, case.get("min_S", 0), case["S"], B)
        n = _spread(g, case["min_nodes"], case["nodes"], B)
        total = int(_cdiv(lens.long() + case["nodes"], bs).sum()) + 3
        table, _ = _paged(g, lens + n, bs, case["S"] + case["nodes"], total)
        kv = _fill(g, total, bs)
        nodes, cached = n.tolist(), lens.tolist()
        T = sum(nodes) + 2                                 # two rows of padding behind the last tree
        start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(n.long(), 0)]).int()
        parents = _trees(g, nodes) + [-1, -1]
        if op == "decode":
            dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
            mask = torch.zeros((T, -(-case["nodes"] // 64)), dtype=torch.int64)
            t = 0
            for k in nodes:
                for i in range(k):
                    if i:
                        mask[t + i] = mask[t + parents[t + i]]
                    mask[t + i, i // 64] |= (1 << (i % 64)) - (1 << 64 if i % 64 == 63 else 0)
                t += k
            q = torch.randn((T, case["h"], D_QK), generator=g, device="cuda").to(torch.bfloat16)
            return dict(op=op, case=case, q=q, kv=kv, table=table, lens=lens, start=start, mask=mask.cuda(),
                        nodes=nodes, cached=cached, scale=1.0 / math.sqrt(192.0),
                        out=torch.zeros((T, case["h"], D_V), dtype=dt, device="cuda"),
                        lse=torch.zeros((T, case["h"]), device="cuda"))
        # the drafts' rows and slots; targets that often are the token of a child
        p = torch.cat([torch.arange(c, c + k) for c, k in zip(cached, nodes)] or [torch.zeros(0)]).long().cuda()
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), n.long())
        slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        slots[:T - 2] = (table[b, p // bs].long() * bs + p % bs).int()
        tokens = _int(g, 0, 100000, (T,))
        targets = _int(g, 0, 100000, (T,))
        hit = torch.rand((T,), generator=g, device="cuda").cpu().tolist()
        tl, gl, t = tokens.tolist(), targets.tolist(), 0
        for k in nodes:
            for i in range(1, k):
                if hit[t + i] < case["hit"]:
                    gl[t + parents[t + i]] = tl[t + i]
            t += k
        return dict(op=op, case=case, kv=kv, table=table, lens=lens, start=start, parents=_i32(parents), slots=slots,
                    tokens=tokens, targets=_i32(gl), rows=_latent_rows(g, T), batch=b)
    L = case.get("layers", 1)
    if op == "free":
        R = case["R"]
        held = _spread(g, 1, case["S"], R)
        gone = torch.rand((R,), generator=g, device="cuda") < case["finished"]
        keep = torch.where(gone, torch.zeros_like(held), (held - _int(g, 0, case["trim"], (R,))).clamp(min=0))
        total = int(_cdiv(held.long(), bs).sum()) + 100
        table, rest = _paged(g, held, bs, case["S"], total)
        free = torch.cat([torch.full((total - rest.numel(),), -1, dtype=torch.int32, device="cuda"), rest])
        return dict(op=op, case=case, table=table, held=held, keep=keep, free=free.contiguous(),
                    taken=_i32([total - rest.numel()]), shares=torch.zeros(total, dtype=torch.int32, device="cuda"))
    if op == "fork":
        R, f = case["R"], case["forks"]
        lens = _spread(g, case["min_S"], case["S"], R)
        total = int(_cdiv(lens.long(), bs).sum()) + R * f + 5
        table, rest = _paged(g, lens, bs, case["S"], total)
        # rows R.. of the table are the forks'
        table = torch.cat([table, torch.full((R * f, table.shape[1]), -1, dtype=torch.int32, device="cuda")])
        lens = torch.cat([lens, torch.zeros(R * f, dtype=torch.int32, device="cuda")])
        src = torch.arange(R, device="cuda", dtype=torch.int32).repeat_interleave(f)
        dst = torch.arange(R, R + R * f, device="cuda", dtype=torch.int32)
        s = dict(op=op, case=case, src=src, dst=dst, free=rest, taken=_i32([3]),
                 held=torch.cat([torch.zeros(R, dtype=torch.int32, device="cuda"), lens[:R].repeat_interleave(f)]),
                 keep=torch.zeros(R + R * f, dtype=torch.int32, device="cuda"))
    else:
        R, nb = case["R"], case["blocks"]
        lens = _spread(g, 1, case["S"], R)
        # as many whole requests as 3/4 of the pool holds
        room = torch.cumsum(_cdiv(lens.long(), bs), 0) <= 3 * nb // 4
        lens = torch.where(room, lens, torch.zeros_like(lens))
        total = nb
        table, _ = _paged(g, lens, bs, case["S"], total)
        shared = torch.zeros(total, dtype=torch.int32, device="cuda")
        if R > 1 and int(lens[0]) >= bs and int(lens[R - 1]) >= bs:
            k = min(int(lens[0]), int(lens[R - 1])) // bs // 2 + 1   # the last request has the first's beginning
            table[R - 1, :k] = table[0, :k]
            shared[table[0, :k].long()] = 1
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        used[table[table >= 0].long()] = True
        rest = torch.nonzero(~used).flatten()
        rest = rest[torch.randperm(rest.numel(), generator=g, device="cuda")].to(torch.int32)
        free = torch.cat([torch.full((total - rest.numel(),), -1, dtype=torch.int32, device="cuda"), rest])
        s = dict(op=op, case=case, free=free.contiguous(), taken=_i32([total - rest.numel()]), shares=shared)
    s.update(table=table.contiguous(), lens=lens, layers=L, total=total)
    s.setdefault("shares", torch.zeros(total, dtype=torch.int32, device="cuda"))
    if case["dtype"] == "bf16":
        s["kv"] = torch.stack([_fill(g, total, bs) for _ in range(L)]) if L > 1 else _fill(g, total, bs)[None]
    else:
        s["kv"] = torch.empty((L, total, bs, D_QK), dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(L):
            s["kv"][i] = _fill(g, total, bs).to(torch.float8_e4m3fn)
        s["scales"] = torch.exp2(_int(g, -6, 3, (L, total, bs // 16)).float())
    return s


# ------------------------------------------------------------------------------- runs
def run(s):
    return {"decode": _decode, "step": _step, "fork": _fork, "free": _free, "compact": _compact}[s["op"]](s)


def _decode(s):
    """(out, lse) of every node; the padding rows behind the last tree stay as they were."""
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        return sfa.decode_tree(s["q"], s["kv"], s["table"], s["lens"], s["start"], s["mask"], s["scale"], out=s["out"],
                               lse=s["lse"])
    bs, h, t = s["case"]["block_size"], s["case"]["h"], 0
    for b, (c, n) in enumerate(zip(s["cached"], s["nodes"])):
        if n == 0:
            continue
        p = torch.arange(c + n, device="cuda")
        k = s["kv"].view(-1, D_QK)[s["table"][b, p // bs].long() * bs + p % bs].float()
        j = torch.arange(n, device="cuda")
        seen = (s["mask"][t:t + n][:, j // 64] >> (j % 64)[None, :]) & 1
        seen = torch.cat([torch.ones((n, c), dtype=torch.bool, device="cuda"), seen.bool()], 1)
        x = torch.matmul(s["q"][t:t + n].float().view(n * h, D_QK), k.t()).view(n, h, c + n) * s["scale"]
        x.masked_fill_(~seen[:, None, :], -math.inf)
        m = x.amax(-1, keepdim=True)
        x = torch.exp(x - m)
        z = x.sum(-1, keepdim=True)
        s["out"][t:t + n] = (torch.matmul(x.view(n * h, c + n), k[:, :D_V]).view(n, h, D_V) / z).to(s["out"].dtype)
        s["lse"][t:t + n] = (m + torch.log(z))[..., 0]
        t += n
    return s["out"], s["lse"]


def _step(s):
    """(mask, positions, path, accepted, next tokens, new lengths, cache)."""
    most, bs = s["case"]["nodes"], s["case"]["block_size"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        mask, pos = sfa.tree_plan(s["parents"], s["start"], s["lens"], most)
        sfa.kv_write(s["kv"], s["slots"], s["rows"])
        path, accepted, after, lens = sfa.tree_accept(s["tokens"], s["targets"], s["parents"], s["start"], s["lens"], most)
        sfa.kv_commit(s["kv"], s["table"], s["lens"], path, accepted)
        return mask, pos, path, accepted, after, lens, s["kv"]
    start, par, b = s["start"].long(), s["parents"].long(), s["batch"]
    B, T, N = start.numel() - 1, par.numel(), s["batch"].numel()
    W = -(-most // 64)
    first = start[b]
    par = par[:N]
    # masks and depths: every node's chain of parents, a step at a time
    mask = torch.zeros((T, W), dtype=torch.int64, device="cuda")
    depth = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    at = torch.arange(N, device="cuda") - first
    word = torch.arange(W, device="cuda")[None, :]
    for _ in range(most):
        real = at >= 0
        bit = torch.ones_like(at) << (at.clamp(min=0) % 64)
        mask[:N] |= torch.where(real[:, None] & (word == (at // 64)[:, None]), bit[:, None], torch.zeros_like(bit[:, None]))
        depth[:N] += real
        at = torch.where(real, par[first + at.clamp(min=0)], at)
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[:N] = (s["lens"].long()[b] + depth[:N]).int()
    kv = s["kv"].view(-1, D_QK)
    kv[s["slots"][:N].long()] = s["rows"][:N]
    # the path: from node 0 to the lowest child that is the target, as long as there is one
    tok, tgt = s["tokens"][:N], s["targets"][:N]
    local = torch.arange(N, device="cuda") - first
    n = start[1:] - start[:-1]
    cur = torch.where(n > 0, torch.zeros_like(n), torch.full_like(n, -1))
    path = torch.full((B, most), -1, dtype=torch.int64, device="cuda")
    accepted = torch.zeros_like(n)
    after = torch.full_like(n, -1)
    lim = max(N - 1, 0)
    for i in range(most):
        live = cur >= 0
        path[:, i] = cur
        accepted += live
        if N == 0:
            break
        want = tgt[(start[:-1] + cur.clamp(min=0)).clamp(max=lim)].long()
        after = torch.where(live, want, after)
        good = (par == cur[b]) & (tok.long() == want[b]) & live[b]
        nxt = torch.full_like(n, 1 << 30).scatter_reduce(0, b, torch.where(good, local, torch.full_like(local, 1 << 30)), "amin")
        cur = torch.where(nxt < (1 << 30), nxt, torch.full_like(nxt, -1))
    # the accepted rows move up
    c = s["lens"].long()[:, None]
    k = torch.arange(most, device="cuda")[None, :]
    moves = path >= 0
    where = lambda p: torch.gather(s["table"].long(), 1, (p // bs).clamp(max=s["table"].shape[1] - 1)) * bs + p % bs  # noqa: E731
    source = torch.where(moves, where(c + path.clamp(min=0)), torch.zeros_like(path))
    # rows that are not accepted go to a row of their own behind the cache
    both = torch.cat([kv, kv.new_zeros((1, D_QK))])
    both[torch.where(moves, where(c + k), torch.full_like(path, kv.shape[0])).flatten()] = kv[source.flatten()]
    kv.copy_(both[:-1])
    return mask, pos, path.int(), accepted.int(), after.int(), (s["lens"].long() + accepted).int(), s["kv"]


def _copy_plain(s, copies):
    """Rows [0, n) of block dst = those of block src, in every layer, and their scales."""
    bs = s["case"]["block_size"]
    c = copies.long()
    real = c[:, 0] >= 0
    a, d = c[:, 0].clamp(min=0), torch.where(real, c[:, 1], torch.full_like(c[:, 1], s["total"]))
    r = torch.arange(bs, device="cuda")
    for i in range(s["layers"]):
        kv = s["kv"][i].view(torch.uint8 if s["kv"].dtype == torch.float8_e4m3fn else torch.int16)
        keep = (r[None, :] < c[:, 2:3])[:, :, None]
        new = torch.where(keep, kv[a], kv[d.clamp(max=s["total"] - 1)])
        both = torch.cat([kv, kv[:1]])
        both[d] = new
        kv.copy_(both[:-1])
        if "scales" in s:
            sc = s["scales"][i]
            g = torch.arange(sc.shape[1], device="cuda")
            keep = g[None, :] * (bs // sc.shape[1]) < c[:, 2:3]
            both = torch.cat([sc, sc[:1]])
            both[d] = torch.where(keep, sc[a], sc[d.clamp(max=s["total"] - 1)])
            sc.copy_(both[:-1])


def _cache(s):
    if "scales" in s:
        return s["kv"], s["scales"]
    return (s["kv"],)


def _copy_own(s, copies):
    import deepseek_sparse_mla_sfa_gb300 as sfa
    if "scales" in s:
        sfa.kv_copy_blocks_q8(s["kv"], s["scales"], copies)
    else:
        sfa.kv_copy_blocks(s["kv"], copies)


def _free_plain(table, held, keep, shares, free, taken, bs):
    """taken after the blocks behind the kept positions are given back; shares and free in place."""
    held, keep = _cdiv(held.long().clamp(min=0), bs), _cdiv(keep.long().clamp(min=0), bs)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    named = ((col >= keep[:, None]) & (col < held[:, None])).flatten()
    nb = shares.numel()
    x = torch.where(named, table.flatten().long(), torch.full((table.numel(),), nb, device="cuda"))
    count = torch.zeros(nb + 1, dtype=torch.int64, device="cuda").scatter_add_(0, x, torch.ones_like(x))[:nb]
    left = shares.long() - count
    gone = (left < 0) & (count > 0)
    # a block goes where it is named first
    e = torch.arange(x.numel(), device="cuda")
    first = torch.full((nb + 1,), x.numel(), device="cuda").scatter_reduce(0, x, e, "amin")
    push = named & (first[x] == e) & torch.cat([gone, gone.new_zeros(1)])[x]
    rank = torch.cumsum(push.long(), 0) - 1
    new = taken.long() - push.sum()
    both = torch.cat([free, free.new_zeros(1)])
    both[torch.where(push, new + rank, torch.full_like(rank, free.numel()))] = torch.where(push, x, torch.zeros_like(x)).int()
    free.copy_(both[:-1])
    shares.copy_(left.clamp(min=0).int())
    return new.int()


def _fork(s):
    """Forks and frees them again: (copies, taken between, table, lens, shares, free list, taken after, cache)."""
    bs = s["case"]["block_size"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        copies, taken = sfa.blocks_fork(s["table"], s["lens"], s["src"], s["dst"], s["shares"], s["free"], s["taken"], bs)
        _copy_own(s, copies)
        back = sfa.blocks_free(s["table"], s["held"], s["keep"], s["shares"], s["free"], taken, bs)
        return (copies, taken, s["table"], s["lens"], s["shares"], s["free"], back, *_cache(s))
    src, dst = s["src"].long(), s["dst"].long()
    n = s["lens"][src].long()
    full, rows = torch.div(n, bs, rounding_mode="floor"), n % bs
    part = rows > 0
    at = s["taken"].long() + torch.cumsum(part.long(), 0) - part.long()
    fresh = s["free"][at.clamp(max=s["free"].numel() - 1)]
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    old = s["table"][src]
    row = torch.where(col < full[:, None], old, s["table"][dst])
    row = torch.where((col == full[:, None]) & part[:, None], fresh[:, None], row)
    s["table"][dst] = row
    s["lens"][dst] = n.int()
    shared = torch.where(col < full[:, None], old.long(), torch.full_like(old.long(), s["total"])).flatten()
    more = torch.zeros(s["total"] + 1, dtype=torch.int64, device="cuda").scatter_add_(0, shared, torch.ones_like(shared))
    s["shares"] += more[:-1].int()
    last = torch.gather(old, 1, full[:, None].clamp(max=old.shape[1] - 1))[:, 0]
    copies = torch.where(part[:, None], torch.stack([last, fresh, rows.int()], 1), torch.full((src.numel(), 3), -1, device="cuda").int())
    taken = (s["taken"].long() + part.sum()).int()
    _copy_plain(s, copies)
    back = _free_plain(s["table"], s["held"], s["keep"], s["shares"], s["free"], taken, bs)
    return (copies, taken, s["table"], s["lens"], s["shares"], s["free"], back, *_cache(s))


def _free(s):
    """(shares, free list, taken)."""
    bs = s["case"]["block_size"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        back = sfa.blocks_free(s["table"], s["held"], s["keep"], s["shares"], s["free"], s["taken"], bs)
    else:
        back = _free_plain(s["table"], s["held"], s["keep"], s["shares"], s["free"], s["taken"], bs)
    return s["shares"], s["free"], back


def _compact(s):
    """(table, shares, free list, copies, cache) with the highest held blocks in the lowest free ones."""
    bs, most = s["case"]["block_size"], s["case"]["max_moves"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        table, shares, free, copies = sfa.blocks_compact(s["table"], s["lens"], s["shares"], s["free"], s["taken"], bs, most)
        _copy_own(s, copies)
        return (table, shares, free, copies, *_cache(s))
    nb, F = s["total"], s["free"].numel()
    ids = torch.arange(nb, device="cuda")
    entry = torch.arange(F, device="cuda") >= s["taken"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    mine = col < _cdiv(s["lens"].long(), bs)[:, None]
    put = lambda ok, x: torch.zeros(nb + 1, dtype=torch.bool, device="cuda").index_fill(  # noqa: E731
        0, torch.where(ok, x.long(), torch.full_like(x.long(), nb)).flatten(), True)[:nb]
    isfree, held = put(entry, s["free"]), put(mine, s["table"])
    low = torch.sort(torch.where(isfree, ids, torch.full_like(ids, nb))).values[:most]
    high = torch.sort(torch.where(held, ids, torch.full_like(ids, -1)), descending=True).values[:most]
    real = low < high
    to = torch.cat([ids, ids.new_full((1,), -1)])
    to[torch.where(real, high, torch.full_like(high, nb))] = torch.where(real, low, torch.full_like(low, -1))
    table = torch.where(mine, to[s["table"].long().clamp(min=0)].int(), s["table"])
    moved = to[:nb] != ids
    shares = torch.where(moved, torch.zeros_like(s["shares"]), s["shares"])
    wide = torch.cat([shares, shares.new_zeros(1)])
    wide[torch.where(real, low, torch.full_like(low, nb))] = s["shares"][high.clamp(min=0)]
    shares = wide[:nb].contiguous()
    now = torch.cat([isfree | moved, isfree.new_zeros(1)])
    now[torch.where(real, low, torch.full_like(low, nb))] = False
    order = torch.sort(torch.where(now[:nb], ids, torch.full_like(ids, nb))).values
    free = torch.where(entry, order[(torch.arange(F, device="cuda") - s["taken"].long()).clamp(min=0, max=nb - 1)].int(), s["free"])
    copies = torch.where(real[:, None], torch.stack([high, low, torch.full_like(low, bs)], 1), torch.full((low.numel(), 3), -1, device="cuda")).int()
    if copies.shape[0] < most:
        copies = torch.cat([copies, copies.new_full((most - copies.shape[0], 3), -1)])
    _copy_plain(s, copies)
    return (table, shares, free, copies, *_cache(s))


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    """What `run` returns, from the definitions: attention in 64 bits, whole numbers by loops."""
    s = prepare(case, seed)
    bs = case["block_size"]
    if case["op"] == "decode":
        if sum(n * (c + n) for n, c in zip(s["nodes"], s["cached"])) * case["h"] > 2_000_000_000:
            return None
        h = case["h"]
        out, lse = s["out"].double(), s["lse"].double()
        words = s["mask"].cpu().tolist()
        t = 0
        for b, (c, n) in enumerate(zip(s["cached"], s["nodes"])):
            row = s["table"][b].long()
            slots = (row[:, None] * bs + torch.arange(bs, device="cuda")[None, :]).flatten()[:c + n]
            k = s["kv"].view(-1, D_QK)[slots].double()
            for i in range(n):
                use = list(range(c)) if c < 2 else None
                anc = [j for j in range(n) if words[t + i][j // 64] >> (j % 64) & 1]
                mine = torch.cat([k[:c], k[c:][anc]]) if use is None else k[use + [c + j for j in anc]]
                z = (s["q"][t + i].double() @ mine.t()) * s["scale"]
                lse[t + i] = torch.logsumexp(z, 1)
                out[t + i] = torch.softmax(z, 1) @ mine[:, :D_V]
            t += n
        return out, lse
    tab = s["table"].cpu().tolist()
    if case["op"] == "step":
        B, most = case["B"], case["nodes"]
        st, par, lens = s["start"].tolist(), s["parents"].tolist(), s["lens"].tolist()
        tok, tgt = s["tokens"].tolist(), s["targets"].tolist()
        T, W = len(par), -(-most // 64)
        mask, pos = [[0] * W for _ in range(T)], [-1] * T
        path, acc, after = [[-1] * most for _ in range(B)], [0] * B, [-1] * B
        kv = s["kv"].clone().view(-1, D_QK)
        for b in range(B):
            a, n, c = st[b], st[b + 1] - st[b], lens[b]
            slot = lambda p: tab[b][p // bs] * bs + p % bs  # noqa: E731
            for i in range(n):
                j, d = i, 0
                while j >= 0:
                    mask[a + i][j // 64] |= 1 << (j % 64)
                    j, d = par[a + j], d + 1
                pos[a + i] = c + d - 1
                kv[slot(c + i)] = s["rows"][a + i]
            cur = 0 if n else None
            while cur is not None:
                path[b][acc[b]] = cur
                acc[b] += 1
                after[b] = tgt[a + cur]
                cur = next((j for j in range(n) if par[a + j] == cur and tok[a + j] == after[b]), None)
            rows = [kv[slot(c + j)].clone() for j in path[b][:acc[b]]]
            for i, r in enumerate(rows):
                kv[slot(c + i)] = r
        sign = [[w - (1 << 64) if w >> 63 else w for w in m] for m in mask]
        cpu = lambda x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
        return (cpu(sign).view(T, W), cpu(pos), cpu(path), cpu(acc), cpu(after), cpu([x + y for x, y in zip(lens, acc)]),
                kv.view(s["kv"].shape))
    share, free, taken = s["shares"].tolist(), s["free"].tolist(), int(s["taken"][0])

    def give_back(held, keep, taken):
        out = []
        seen = {}
        for r in range(len(tab)):
            for j in range(-(-keep[r] // bs), -(-held[r] // bs)):
                x = tab[r][j]
                seen.setdefault(x, 0)
                seen[x] += 1
        for x, m in seen.items():                          # in the order of first mention
            if m > share[x]:
                out.append(x)
            share[x] = max(share[x] - m, 0)
        free[taken - len(out):taken] = out
        return taken - len(out)

    i64 = lambda x: torch.tensor(x, dtype=torch.int64)  # noqa: E731
    if case["op"] == "free":
        back = give_back(s["held"].tolist(), s["keep"].tolist(), taken)
        return i64(share), i64(free), i64([back])

    def copied(copies):
        kv = s["kv"].clone().view(torch.uint8)
        sc = s["scales"].clone() if "scales" in s else None
        for a, d, n in copies:
            if a < 0:
                continue
            kv[:, d, :n] = kv[:, a, :n]
            if sc is not None:
                k = -(-n // (bs // sc.shape[2]))
                sc[:, d, :k] = sc[:, a, :k]
        kv = kv.view(s["kv"].dtype)
        return (kv,) if sc is None else (kv, sc)

    lens = s["lens"].tolist()
    if case["op"] == "fork":
        copies, at = [], taken
        for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
            full, rows = divmod(lens[a], bs)
            tab[d][:full] = tab[a][:full]
            for x in tab[a][:full]:
                share[x] += 1
            copies.append([-1, -1, -1])
            if rows:
                copies[-1] = [tab[a][full], free[at], rows]
                tab[d][full] = free[at]
                at += 1
            lens[d] = lens[a]
        back = give_back(s["held"].tolist(), s["keep"].tolist(), at)
        return (i64(copies), i64([at]), i64(tab), i64(lens), i64(share), i64(free), i64([back]), *copied(copies))
    mine = {tab[r][j] for r in range(len(tab)) for j in range(-(-lens[r] // bs))}
    rest = sorted(free[taken:])
    move = {}
    for lo, hi in zip(rest, sorted(mine, reverse=True)):
        if lo < hi and len(move) < case["max_moves"]:
            move[hi] = lo
    for r in range(len(tab)):
        for j in range(-(-lens[r] // bs)):
            tab[r][j] = move.get(tab[r][j], tab[r][j])
    for hi, lo in move.items():
        share[lo], share[hi] = share[hi], 0
    free[taken:] = sorted((set(rest) - set(move.values())) | set(move))
    copies = [[hi, lo, bs] for hi, lo in move.items()]
    copies += [[-1, -1, -1]] * (case["max_moves"] - len(copies))
    return (i64(tab), i64(share), i64(free), i64(copies), *copied(copies))


# ------------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations of a pass on average: each input read once, each output written once."""
    op, bs = case["op"], case["block_size"]
    if op == "decode":
        n, S = (case["nodes"] + case["min_nodes"]) / 2, (case["S"] + case["min_S"]) / 2
        out = 4 if case["dtype"] == "fp32" else 2
        row = case["h"] * (D_QK * 2 + D_V * out + 4) + 8 * -(-case["nodes"] // 64)
        return {"bytes": case["B"] * ((S + n) * (D_QK * 2 + 4 / bs) + n * row),
                "flops": case["B"] * 2.0 * n * case["h"] * (S + n) * (D_QK + D_V)}
    if op == "step":
        n = (case["nodes"] + case["min_nodes"]) / 2
        moved = min(n, 2.0)                                # rows of a path that change places
        return {"bytes": case["B"] * (n * (2 * D_QK * 2 + 24 + 8 * -(-case["nodes"] // 64)) + moved * 2 * D_QK * 2
                                      + 4 * case["nodes"] + 20), "flops": 0}
    size = 2 if case.get("dtype") == "bf16" else 1
    if op == "fork":
        N, S = case["R"] * case["forks"], (case["S"] + case["min_S"]) / 2
        return {"bytes": N * (case["layers"] * (min(S, bs) / 2) * D_QK * size * 2 + S / bs * 24 + 40), "flops": 0}
    if op == "free":
        given = case["R"] * (case["finished"] * case["S"] / 2 + (1 - case["finished"]) * case["trim"] / 2) / bs
        return {"bytes": given * 16 + case["R"] * 8 + 8, "flops": 0}
    held = min(0.75 * case["blocks"], case["R"] * (case["S"] / bs / 2 + 0.5))
    moves = min(case["max_moves"], held * (1 - held / case["blocks"]))
    return {"bytes": moves * (case["layers"] * bs * D_QK * size * 2 + 12) + held * 8 + case["blocks"] * 16, "flops": 0}
