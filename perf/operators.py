"""Cases of the serving step around sparse MLA decode: block tables and slot maps from
request lengths, rotary positions, the write of an 8-bit latent cache and the attention
that reads it.

Each case names its operator in "op" and carries the sizes.  With `own` false `run`
computes the operator's plain form with elementary torch operations; with `own` true it
calls the package.  `exact` gives the result from the definition in 64 bits.
"""
import math

import torch

own = False

D_QK, D_V = 576, 512          # a latent row: 512 latent + 64 rope columns; V = the first 512
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 120  # exponents of the cache's power-of-two scales


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 running requests, one new token each: the smallest plan,
        # where latency counts
        dict(name="plan_decode", op="plan", B=64, max_new=1, min_new=1, max_cached=8192, block_size=64, pad=0),
        # a mixed step: 512 requests, prompt chunks beside single tokens, padded for a graph
        dict(name="plan_mixed", op="plan", B=512, max_new=300, min_new=0, max_cached=40000, block_size=64, pad=1000),
        # the queries of one decode step (128 heads) at far positions, neighbouring pairs, YaRN
        dict(name="rope_q_decode", op="rope", T=64, n=128, rot=64, d_in=192, in_off=128, d_out=576, out_off=512,
             pos_max=131072, interleaved=True, scaling="yarn", inverse=False, dtype="bf16"),
        # the queries of a prompt chunk (64 heads), halves
        dict(name="rope_q_prompt", op="rope", T=4096, n=64, rot=64, d_in=192, in_off=128, d_out=576, out_off=512,
             pos_max=65536, interleaved=False, scaling="linear", inverse=False, dtype="bf16"),
        # the gradient of a rotation (its transpose) in fp32, half of each head, odd sizes
        dict(name="rope_grad", op="rope", T=777, n=16, rot=48, d_in=96, in_off=0, d_out=96, out_off=0,
             pos_max=5000, interleaved=True, scaling="none", inverse=True, dtype="fp32"),
        # the new rows of one decode step of 64 requests: each joins a partly filled group
        dict(name="write_decode", op="write", B=64, new=1, S=4000, block_size=64, group=64, min_S=100),
        # a prompt chunk: many rows of few requests, whole groups and ragged ends
        dict(name="write_prompt", op="write", B=5, new=1777, S=2000, block_size=64, group=16, min_S=0),
        # one request, 4 heads, a short list: the latency of a call
        dict(name="decode_one", op="decode", B=1, Q=1, h=4, S=256, k=64, n_splits=1, block_size=64, group=64, kind="uniform"),
        # the benchmark's sparse decode step: 128 heads, 2048 of 32768 positions
        dict(name="decode_h128", op="decode", B=64, Q=1, h=128, S=32768, k=2048, n_splits=1, block_size=64, group=64,
             kind="uniform"),
        # the benchmark's step with a speculated token: causal lists, 64 heads, ragged lengths
        dict(name="decode_mtp", op="decode", B=128, Q=2, h=64, S=16384, k=2048, n_splits=1, block_size=64, group=16,
             kind="causal"),
        # every position of each request by few heads, four shards merged
        dict(name="decode_dense", op="decode", B=32, Q=1, h=16, S=8192, k=8192, n_splits=4, block_size=64, group=64,
             kind="dense"),
        # a few long requests, an odd head count and list length, eight shards merged
        dict(name="decode_long", op="decode", B=5, Q=1, h=100, S=131072, k=1537, n_splits=8, block_size=64, group=32,
             kind="uniform"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "write", "decode", "decode"])
    if op == "plan":
        B = _log(rng, 1, 700)
        most = max(1, min(_log(rng, 1, 2000), 100000 // B))
        return dict(op=op, B=B, max_new=most, min_new=rng.choice([0, min(1, most)]), max_cached=_log(rng, 16, 40000),
                    block_size=rng.choice([16, 24, 64, 128]), pad=rng.choice([0, rng.randrange(1, 2000)]))
    if op == "rope":
        n = _log(rng, 1, 128)
        T = _log(rng, 1, max(2, 4096 * 64 // n // 2))
        rot = 2 * rng.randrange(4, 65)
        off, rest = rng.choice([0, 32, 128]), rng.choice([0, 16, 24])
        return dict(op=op, T=min(T, 8192), n=n, rot=rot, d_in=off + rot + rest, in_off=off, d_out=rot + rest, out_off=0,
                    pos_max=_log(rng, 64, 1000000), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), inverse=rng.random() < 0.3,
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "write":
        B = _log(rng, 1, 128)
        new = max(1, min(_log(rng, 1, 2000), 8000 // B))
        bs = rng.choice([16, 64, 128])
        return dict(op=op, B=B, new=new, S=new + _log(rng, 16, 1000), block_size=bs,
                    group=rng.choice([g for g in (1, 8, 16, 64) if bs % g == 0]), min_S=0)
    bs = rng.choice([16, 64, 128])
    kind = rng.choice(["uniform", "causal", "dense"])
    S = _log(rng, 64, 16384)
    k = S if kind == "dense" else _log(rng, 1, min(S, 4096))
    Q = rng.choice([1, 1, 2, 3]) if kind == "causal" else 1
    B = max(1, min(_log(rng, 1, 128), 200000 // (k * Q), 1000000 // S))
    return dict(op=op, B=B, Q=Q, h=rng.choice([1, 3, 8, 16, 27, 32, 64, 72, 128]), S=S, k=k,
                n_splits=rng.choice([1, 1, 2, 5]), block_size=bs,
                group=rng.choice([g for g in (1, 16, 32, 64, 128) if bs % g == 0]), kind=kind)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)


def _int(g, lo, hi, shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _cdiv(a, b):
    return torch.div(a + (b - 1), b, rounding_mode="floor")


def _inv_freq(rot, scaling):
    """Angle a position (radians), 64 bits: theta_i = 10000^(-2i/rot), scaled for contexts
    40 times the trained 4096: all of them divided ("linear"), or by the wavelength's share
    of the trained length as YaRN does."""
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / 40.0
    if scaling == "yarn":
        turns = 4096.0 * f / (2.0 * math.pi)
        ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f / 40.0 * (1.0 - ramp) + f * ramp
    return f


def _quantise(x, scale):
    """e4m3 values of x / scale."""
    return (x / scale).to(torch.float8_e4m3fn)


def _pow2_scale(amax):
    """The least power of two s with amax / s <= 448, its exponent in [MIN_EXP, MAX_EXP]."""
    m, e = torch.frexp(amax.double() / E4M3_MAX)      # m in [0.5, 1), amax / 448 = m 2^e
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax == 0, torch.full_like(e, MIN_EXP), e).clamp(MIN_EXP, MAX_EXP)
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e).float()


def _latent_rows(g, n):
    """Latent rows as they meet a cache: normed latents of about 1, a token's size varying,
    rope columns larger."""
    x = torch.randn((n, D_QK), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((n, 1), generator=g, device="cuda"))
    x[:, D_V:] *= 2.0
    return x.to(torch.bfloat16)


def _paged(g, lens, most, block_size, spare):
    """A block table over shuffled physical blocks of a pool, for sequences of these lengths
    (at most `most`): (table [B, max_blocks] with -1 in unused entries, number of blocks)."""
    nblk = _cdiv(lens.long(), block_size)
    width = -(-most // block_size) + 2
    total = lens.numel() * (width - 2) + spare
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    start = torch.cumsum(nblk, 0) - nblk
    at = (start[:, None] + col[None, :]).clamp(max=total - 1)
    table = torch.where(col[None, :] < nblk[:, None], ids[at], torch.full_like(ids[at], -1))
    return table.contiguous(), total


def _room(case):
    """Tokens that a planned step has room for."""
    B, most = case["B"], case["max_new"]
    return B * most if most <= 16 else B + B * most // 4


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "plan":
        B, bs = case["B"], case["block_size"]
        cached = _int(g, 0, case["max_cached"], (B,))
        new = _int(g, case["min_new"], case["max_new"], (B,))
        if case["max_new"] > 16:                       # two of three requests decode one token
            new = torch.where(torch.rand((B,), generator=g, device="cuda") < 0.66, new.clamp(max=1), new)
        # as many tokens as the step has room for
        room = _room(case)
        new = torch.minimum(new.long(), (room - (torch.cumsum(new.long(), 0) - new)).clamp(min=0)).int()
        table, total = _paged(g, cached, case["max_cached"] + case["max_new"], bs, 37)
        # the pool's blocks that no request holds, in the order they are handed out, and how
        # many of them earlier steps took
        used = torch.zeros(total, dtype=torch.bool, device="cuda")
        used[table[table >= 0].long()] = True
        free = torch.nonzero(~used).flatten().to(torch.int32)
        taken = _int(g, 1, 9, (1,))
        free = torch.cat([torch.full((int(taken),), -1, dtype=torch.int32, device="cuda"), free])
        tokens = room + case["pad"]
        return dict(op=op, case=case, cached=cached, new=new, table=table, free=free.contiguous(), taken=taken,
                    tokens=tokens)
    if op == "rope":
        dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[case["dtype"]]
        T, n = case["T"], case["n"]
        x = torch.randn((T, n, case["d_in"]), generator=g, device="cuda").to(dt)
        out = torch.zeros((T, n, case["d_out"]), device="cuda", dtype=dt)
        pos = _int(g, 0, case["pos_max"] - 1, (T,))
        w = min(case["d_in"] - case["in_off"], case["d_out"] - case["out_off"])
        return dict(op=op, case=case, x=x[..., case["in_off"]:case["in_off"] + w],
                    out=out[..., case["out_off"]:case["out_off"] + w], pos=pos,
                    inv_freq=_inv_freq(case["rot"], case["scaling"]),
                    mscale=0.1 * math.log(40.0) + 1.0 if case["scaling"] == "yarn" else 1.0)
    bs, gs = case["block_size"], case["group"]
    if op == "write":
        B, new = case["B"], case["new"]
        lens = _int(g, max(new, case["min_S"]), case["S"], (B,))
        table, total = _paged(g, lens, case["S"], bs, 3)
        # the rows that the cache holds already, and the new tokens' rows behind them
        old = _latent_rows(g, total * bs).view(total * bs // gs, gs, D_QK)
        scale = _pow2_scale(old.float().abs().amax(dim=(1, 2)))
        kv8 = _quantise(old.float(), scale[:, None, None]).view(total, bs, D_QK)
        p = (lens.long() - new)[:, None] + torch.arange(new, device="cuda")[None, :]
        slot = torch.gather(table.long(), 1, p // bs) * bs + p % bs
        rows = _latent_rows(g, B * new)
        words = 8 * (total * bs // gs)                 # the scratch words a cache of this size takes
        return dict(op=op, case=case, kv8=kv8, scales=scale.view(total, bs // gs), rows=rows,
                    slots=slot.flatten().to(torch.int32),
                    workspace=torch.zeros(words, dtype=torch.int32, device="cuda"))
    B, Q, S, k = case["B"], case["Q"], case["S"], case["k"]
    if case["kind"] == "causal":
        lens = _int(g, max(Q, S // 16), S, (B,))
    else:
        lens = torch.full((B,), S, device="cuda", dtype=torch.int32)
    table, total = _paged(g, lens, S, bs, 2)
    kv8 = torch.empty((total, bs, D_QK), device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty((total, bs // gs), device="cuda")
    step = max(1, (1 << 18) // bs)
    for b0 in range(0, total, step):
        nb = min(step, total - b0)
        x = _latent_rows(g, nb * bs).float().view(nb * bs // gs, gs, D_QK)
        sc = _pow2_scale(x.abs().amax(dim=(1, 2)))
        kv8[b0:b0 + nb] = _quantise(x, sc[:, None, None]).view(nb, bs, D_QK)
        scales[b0:b0 + nb] = sc.view(nb, bs // gs)
    q = torch.randn((B * Q, case["h"], D_QK), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.full((B * Q, k), -1, dtype=torch.int32, device="cuda")
    for t in range(B * Q):
        if case["kind"] == "dense":
            idx[t] = torch.arange(k, device="cuda", dtype=torch.int32)
            continue
        L = int(lens[t // Q]) - (Q - 1 - t % Q) if t % Q == 0 or case["kind"] == "uniform" else L + 1
        n = min(k, max(L, 0))
        idx[t, :n] = torch.randperm(max(L, 1), generator=g, device="cuda")[:n].to(torch.int32)
    return dict(op=op, case=case, q=q, kv8=kv8, scales=scales, table=table, lens=lens, idx=idx,
                scale=1.0 / math.sqrt(192.0))


# ------------------------------------------------------------------------------- runs
def run(s):
    return {"plan": _plan, "rope": _rope, "write": _write, "decode": _decode}[s["op"]](s)


def _plan(s):
    """(block_table, seq_lens, token_start, positions, slot_mapping, taken)."""
    bs, N = s["case"]["block_size"], s["tokens"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        return sfa.step_plan(s["cached"], s["new"], s["table"], s["free"], s["taken"], bs, N)
    cached, new = s["cached"].long(), s["new"].long()
    held, need = _cdiv(cached, bs), _cdiv(cached + new, bs)
    fresh = need - held
    first = s["taken"].long() + torch.cumsum(fresh, 0) - fresh
    col = torch.arange(s["table"].shape[1], device="cuda")[None, :]
    at = first[:, None] + col - held[:, None]
    take = (col >= held[:, None]) & (col < need[:, None])
    table = torch.where(take, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"])
    end = torch.cumsum(new, 0)
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), end])
    i = torch.arange(N, device="cuda")
    b = torch.searchsorted(end, i, right=True)
    real = b < cached.numel()
    b = b.clamp(max=cached.numel() - 1)
    p = cached[b] + i - start[b]
    slot = table[b, torch.div(p, bs, rounding_mode="floor").clamp(max=table.shape[1] - 1)].long() * bs + p % bs
    minus = torch.full_like(p, -1)
    return (table, (cached + new).int(), start.int(), torch.where(real, p, minus).int(),
            torch.where(real, slot, minus).int(), (s["taken"].long() + fresh.sum()).int())


def _rope(s):
    c = s["case"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        return sfa.rope(s["x"], s["pos"], s["inv_freq"], interleaved=c["interleaved"], mscale=s["mscale"],
                        inverse=c["inverse"], out=s["out"])
    rot = c["rot"]
    ang = s["pos"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    if c["inverse"]:
        sin = -sin
    x = s["x"].float()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    u, v = (a * cos - b * sin) * s["mscale"], (a * sin + b * cos) * s["mscale"]
    y = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    s["out"].copy_(torch.cat([y, x[..., rot:]], -1))
    return s["out"]


def _write(s):
    """(kv8, scales): the cache with the new rows in it."""
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        sfa.kv_write_q8(s["kv8"], s["scales"], s["slots"], s["rows"], workspace=s["workspace"])
        return s["kv8"], s["scales"]
    gs = s["case"]["group"]
    slots = s["slots"].long()
    kv = s["kv8"].view(torch.uint8).view(-1, gs, D_QK)
    scales = s["scales"].view(-1)
    x = s["rows"].float()
    need = _pow2_scale(x.abs().amax(dim=1))
    grp = slots // gs
    old = scales.index_fill(0, grp[slots % gs == 0], 0.0)
    new = old.scatter_reduce(0, grp, need, "amax")
    # rows of these groups that this call does not write go to the new scale
    held = kv[grp].view(torch.float8_e4m3fn).float() * torch.where(old > 0, old / new, torch.ones_like(old))[grp][:, None, None]
    kv[grp] = held.to(torch.float8_e4m3fn).view(torch.uint8)
    kv.view(-1, D_QK)[slots] = _quantise(x, new[grp][:, None]).view(torch.uint8)
    scales.copy_(new)
    return s["kv8"], s["scales"]


def _rows_of(s):
    """(rows [T, k] of the cache, used [T, k]) of the listed positions."""
    c = s["case"]
    bs, Q = c["block_size"], c["Q"]
    T = s["idx"].shape[0]
    b = torch.arange(T, device="cuda") // Q
    L = s["lens"].long()[b] - (Q - 1 - torch.arange(T, device="cuda") % Q)
    pos = s["idx"].long()
    used = (pos >= 0) & (pos < L[:, None])
    pos = pos.clamp(min=0)
    blk = s["table"].long()[b[:, None], (pos // bs).clamp(max=s["table"].shape[1] - 1)].clamp(min=0)
    return blk * bs + pos % bs, used


def _decode(s):
    """(out [T, h, 512] bf16, lse [T, h] fp32)."""
    c = s["case"]
    if own:
        import deepseek_sparse_mla_sfa_gb300 as sfa
        return sfa.decode_q8(s["q"], s["kv8"], s["scales"], s["table"], s["lens"], s["idx"], s["scale"],
                             n_splits=c["n_splits"], Q=c["Q"], out_dtype=torch.bfloat16)
    rows, used = _rows_of(s)
    kv = s["kv8"].view(torch.uint8).view(-1, D_QK)[rows].view(torch.float8_e4m3fn).float()
    kv *= s["scales"].view(-1)[rows // c["group"]][..., None]
    x = torch.bmm(s["q"].float(), kv.transpose(1, 2)) * s["scale"]
    x = x.masked_fill(~used[:, None, :], float("-inf"))
    top = x.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - top)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.bmm(p, kv[..., :D_V]) / total.clamp(min=1e-30)
    return out.to(torch.bfloat16), (top + torch.log(total))[..., 0]


# ------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "plan":
        B, bs = case["B"], case["block_size"]
        mean = (case["min_new"] + case["max_new"]) / 2
        if case["max_new"] > 16:
            mean = 0.34 * mean + 0.66
        tokens = B * mean + case["pad"]
        # lengths in, lengths and starts out, a position and a slot for each token, the new
        # blocks read and written, and the one table entry a running block is read from
        tokens = min(tokens, _room(case) + case["pad"])
        return dict(bytes=16 * B + 8 * tokens + 8 * B * mean / bs + 4 * B + 12, flops=4 * tokens)
    if op == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        w = min(case["d_in"] - case["in_off"], case["d_out"] - case["out_off"])
        n = case["T"] * case["n"]
        return dict(bytes=2 * n * w * size + 4 * case["T"] + 4 * case["rot"], flops=3.0 * n * case["rot"])
    if op == "write":
        n = case["B"] * case["new"]
        return dict(bytes=n * (D_QK * 3 + 4) + 8 * case["B"] * (case["new"] // case["group"] + 1), flops=3.0 * n * D_QK)
    T, h, k = case["B"] * case["Q"], case["h"], case["k"]
    n = T * min(k, case["S"])
    return dict(bytes=n * (D_QK + 4 + 4 + 4.0 / case["group"]) + T * h * (2 * D_QK + 2 * D_V + 4),
                flops=2.0 * n * h * (D_QK + D_V))


# ------------------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None                                   # whole numbers only
    if op == "rope":
        rot, x = case["rot"], s["x"].double()
        y = x.clone()
        sign = -1.0 if case["inverse"] else 1.0
        for i in range(rot // 2):
            j0, j1 = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            z = torch.polar(torch.full_like(s["pos"], 1, dtype=torch.float64) * s["mscale"],
                            sign * s["pos"].double() * s["inv_freq"][i])[:, None]
            r = torch.complex(x[..., j0], x[..., j1]) * z
            y[..., j0], y[..., j1] = r.real, r.imag
        return y
    if op == "write":
        gs = case["group"]
        vals = s["kv8"].double().view(-1, D_QK).cpu()
        scales = s["scales"].double().view(-1).cpu()
        rows, slots = s["rows"].double().cpu(), s["slots"].long().cpu()
        by = {}
        for t, slot in enumerate(slots.tolist()):
            by.setdefault(slot // gs, []).append((slot, t))
        for grp, members in by.items():
            mine = {slot for slot, _ in members}
            was = 0.0 if grp * gs in mine else float(scales[grp])
            now = was
            for _, t in members:
                a = float(rows[t].abs().max())
                e = MIN_EXP if a == 0 else min(max(math.ceil(math.log2(a / E4M3_MAX)), MIN_EXP), MAX_EXP)
                now = max(now, 2.0 ** e)
            if was and now > was:
                for slot in range(grp * gs, grp * gs + gs):
                    vals[slot] = (vals[slot] * (was / now)).float().to(torch.float8_e4m3fn).double()
            for slot, t in members:
                vals[slot] = (rows[t] / now).float().to(torch.float8_e4m3fn).double()
            scales[grp] = now
        return vals.view(s["kv8"].shape), scales.view(s["scales"].shape)
    rows, used = _rows_of(s)
    T, h = s["idx"].shape[0], case["h"]
    out = torch.zeros((T, h, D_V), dtype=torch.float64, device="cuda")
    lse = torch.full((T, h), -math.inf, dtype=torch.float64, device="cuda")
    kv = s["kv8"].view(torch.uint8).view(-1, D_QK)
    scales = s["scales"].view(-1).double()
    for t in range(T):
        r = rows[t][used[t]]
        if r.numel() == 0:
            continue
        m = kv[r].view(torch.float8_e4m3fn).double() * scales[r // case["group"]][:, None]
        x = (m @ s["q"][t].double().T) * s["scale"]                 # [rows, heads]
        lse[t] = torch.logsumexp(x, dim=0)
        out[t] = torch.exp(x - lse[t]).T @ m[:, :D_V]
    return out, lse
