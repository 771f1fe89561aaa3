"""GPU parity of the blocks that requests hold against the oracle: fork, free, compact, the copies of
cache rows, and runs of them together."""
import numpy as np
import pytest
import torch

import deepseek_sparse_mla_sfa_gb300 as sfa
from oracle import tree

pytestmark = pytest.mark.gpu

NO_BLOCKS, BAD_BLOCK = -7, -6


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def pool(rng, lens, bs, spare, wide=0, lost=0):
    """(table, shares, free list, taken, number of blocks): rows over shuffled blocks, `lost` blocks
    neither held nor free."""
    n = [-(-int(x) // bs) for x in lens]
    total = sum(n) + spare + lost
    ids, at = rng.permutation(total), lost
    table = np.full((len(lens), max(n, default=0) + 1 + wide), -1)
    for r, k in enumerate(n):
        table[r, :k] = ids[at:at + k]
        at += k
    taken = int(rng.integers(0, 4))
    return table, np.zeros(total, int), np.concatenate([np.full(taken, -1), ids[at:]]).astype(int), taken, total


def equal(got, want, what):
    assert np.array_equal(got.cpu().numpy().reshape(-1), np.asarray(want).reshape(-1)), what


# -------------------------------------------------------------------------------- fork
@pytest.mark.parametrize("R,forks,bs,most", [(1, 1, 16, 5), (1, 9, 64, 1500), (40, 3, 16, 100), (300, 2, 1, 9), (3, 200, 7, 50)])
def test_fork_matches_oracle(R, forks, bs, most):
    rng = np.random.default_rng(R + forks)
    lens = rng.integers(0, most + 1, R)
    table, shares, free, taken, nb = pool(rng, lens, bs, R * forks)
    table = np.concatenate([table, np.full((R * forks, table.shape[1]), -1)])
    lens = np.concatenate([lens, np.zeros(R * forks, int)])
    src, dst = np.repeat(np.arange(R), forks), R + rng.permutation(R * forks)
    src[rng.random(R * forks) < 0.1] = -1
    shares[:] = rng.integers(0, 3, nb)
    d = [i32(x) for x in (table, lens, shares)]
    copies, out = sfa.blocks_fork(d[0], d[1], i32(src), i32(dst), d[2], i32(free), i32([taken]), bs)
    assert sfa.last_device_status() == 0
    want = tree.blocks_fork(table, lens, src, dst, shares, free, taken, bs)
    for g, w, name in zip((*d, copies, out), want, ("table", "lens", "shares", "copies", "taken")):
        equal(g, w, name)


def test_fork_reports_what_does_not_fit():
    rng = np.random.default_rng(1)
    table, shares, free, taken, nb = pool(rng, [10, 3, 0, 0, 0], 4, 1)
    args = lambda s, t: (i32(table), i32([10, 3, 0, 0, 0]), i32(s), i32(t), i32(shares), i32(free), i32([taken]), 4)  # noqa: E731
    a = args([0, 1, 0], [2, 3, 4])                                               # three blocks wanted, one free
    copies, out = sfa.blocks_fork(*a)
    assert sfa.last_device_status() == NO_BLOCKS
    want = tree.blocks_fork(table, [10, 3, 0, 0, 0], [0, 1, 0], [2, 3, 4], shares, free, taken, 4)
    for g, w in zip((a[0], a[1], a[4], copies, out), want):
        equal(g, w, "short list")
    a = args([0, 7, 2, 0], [0, 2, 9, 3])                                          # itself, no such rows
    copies, out = sfa.blocks_fork(*a)
    assert sfa.last_device_status() == BAD_BLOCK
    want = tree.blocks_fork(table, [10, 3, 0, 0, 0], [0, 7, 2, 0], [0, 2, 9, 3], shares, free, taken, 4)
    for g, w in zip((a[0], a[1], a[4], copies, out), want):
        equal(g, w, "bad rows")
    bad = table.copy()
    bad[0, 0], bad[1, 0] = nb, -5
    a = (i32(bad), *args([0, 1], [2, 3])[1:])
    copies, out = sfa.blocks_fork(*a)
    # two errors at once, the bad entries and the second item's missing block: either is kept
    assert sfa.last_device_status() in (BAD_BLOCK, NO_BLOCKS) and copies[1].tolist() == [-1] * 3
    copies, out = sfa.blocks_fork(*args([], []))
    assert copies.shape == (0, 3) and int(out) == taken and sfa.last_device_status() == 0


# -------------------------------------------------------------------------------- free
@pytest.mark.parametrize("R,bs,most", [(1, 16, 40), (64, 64, 8192), (700, 16, 3000), (8192, 64, 130), (400, 1, 5000), (3, 1, 2000),
                                       (0, 4, 1)])
@pytest.mark.parametrize("shared", [False, True])
def test_free_matches_oracle(R, bs, most, shared):
    rng = np.random.default_rng(R + bs)
    held = rng.integers(0, most + 1, R)
    table, shares, free, taken, nb = pool(rng, held, bs, 5)
    free = np.concatenate([np.full(nb, -1), free])
    taken += nb
    if shared and R > 1:
        for _ in range(3 * R):                              # rows take over each other's beginnings
            a, b = rng.integers(0, R, 2)
            k = int(rng.integers(0, min(held[a], held[b]) // bs + 1))
            table[a, :k] = table[b, :k]
        for x in np.unique(table):
            if x >= 0:
                shares[x] = max(int(sum(1 for r in range(R) if x in table[r, :-(-held[r] // bs)])) - 1, 0) if R < 100 \
                    else int(rng.integers(0, 3))
    keep = np.where(rng.random(R) < 0.4, 0, np.maximum(held - rng.integers(0, 3 * bs, R), -2))
    if R:
        keep[0] = held[0] + 9                               # keeps more than it holds: gives nothing back
    d = [i32(shares), i32(free)]
    out = sfa.blocks_free(i32(table), i32(held), i32(keep), *d, i32([taken]), bs)
    want = tree.blocks_free(table, held, keep, shares, free, taken, bs)
    status = sfa.last_device_status()
    assert status == 0 or (shared and R >= 100)             # (made-up shares: some are given back too often)
    for g, w, name in zip((*d, out), want, ("shares", "free", "taken")):
        equal(g, w, name)


def test_free_in_one_cluster_and_in_one_block_agree():
    # the same entries in a narrow and in a wide table
    rng = np.random.default_rng(5)
    held = rng.integers(0, 60, 50)
    table, shares, free, taken, nb = pool(rng, held, 4, 0)
    free, taken = np.full(nb, -1), nb
    wide = np.concatenate([table, np.full((50, 200), -1)], 1)
    got = []
    for t in (table, wide):
        s, f = i32(shares), i32(free)
        out = sfa.blocks_free(i32(t), i32(held), i32(held * 0), s, f, i32([taken]), 4)
        got.append((s.tolist(), f.tolist(), int(out)))
    assert got[0] == got[1] and got[0][2] == taken - sum(-(-int(x) // 4) for x in held)
    assert sfa.last_device_status() == 0


def test_free_reports_double_frees_bad_entries_and_a_full_list():
    table = np.array([[3, 1], [1, 2], [-1, 9]])
    for held, status in (([4, 4, 0], BAD_BLOCK), ([4, 0, 4], BAD_BLOCK), ([0, 0, 2], BAD_BLOCK)):
        s, f = i32(np.zeros(5)), i32(np.full(6, -1))
        out = sfa.blocks_free(i32(table), i32(held), i32([0] * 3), s, f, i32([6]), 2)
        assert sfa.last_device_status() == status
        want = tree.blocks_free(table, held, [0] * 3, np.zeros(5, int), np.full(6, -1), 6, 2)
        for g, w in zip((s, f, out), want):
            equal(g, w, held)
    s, f = i32(np.zeros(5)), i32([-1, 4])
    out = sfa.blocks_free(i32(table), i32([4, 0, 0]), i32([0] * 3), s, f, i32([1]), 2)
    assert sfa.last_device_status() == NO_BLOCKS and int(out) == 0 and f.tolist() == [1, 4]


# ----------------------------------------------------------------------------- compact
@pytest.mark.parametrize("R,bs,most,spare,lost,moves", [
    (1, 16, 40, 3, 0, 5), (20, 16, 300, 200, 7, 1000), (20, 16, 300, 200, 7, 30), (5, 64, 100, 31, 0, 0), (0, 4, 1, 40, 2, 9),
    (300, 16, 2000, 9000, 11, 20000), (300, 16, 2000, 9000, 11, 777), (2, 1, 70000, 90000, 0, 100000), (40, 8, 100, 0, 3, 50)])
def test_compact_matches_oracle(R, bs, most, spare, lost, moves):
    rng = np.random.default_rng(R + spare)
    lens = rng.integers(0, most + 1, R)
    table, shares, free, taken, nb = pool(rng, lens, bs, spare, lost=lost)
    for _ in range(R // 2):
        a, b = rng.integers(0, R, 2)
        k = int(rng.integers(0, min(lens[a], lens[b]) // bs + 1))
        table[a, :k] = table[b, :k]
    shares[:] = rng.integers(0, 4, nb)
    got = sfa.blocks_compact(i32(table), i32(lens), i32(shares), i32(free), i32([taken]), bs, moves)
    assert sfa.last_device_status() == 0
    want = tree.blocks_compact(table, lens, shares, free, taken, bs, moves)
    for g, w, name in zip(got, want, ("table", "shares", "free", "copies")):
        equal(g, w, name)


def test_compact_reports_what_does_not_fit():
    table = np.array([[9, 3], [4, 8]])
    for free, lens in (([0, 1, 3], [4, 4]), ([0, 0, 2], [4, 4]), ([0, -4, 77], [4, 4]), ([0, 1], [99, 4])):
        t = table if lens[0] == 4 else np.array([[9, -3], [4, 12]])
        got = sfa.blocks_compact(i32(t), i32(lens), i32(np.arange(10)), i32(free), i32([0]), 2, 4)
        assert sfa.last_device_status() == BAD_BLOCK, free
        want = tree.blocks_compact(t, lens, np.arange(10), free, 0, 2, 4)
        for g, w, name in zip(got, want, ("table", "shares", "free", "copies")):
            equal(g, w, (name, free))


# -------------------------------------------------------------------------------- copies
@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("bs,group", [(1, 1), (7, 7), (16, 4), (64, 16), (128, 1)])
def test_copies_match_oracle(layers, bs, group):
    rng = np.random.default_rng(bs)
    nb, n = 40, 15
    ids = rng.permutation(nb)
    copies = np.stack([ids[:n], ids[n:2 * n], rng.integers(0, bs + 1, n)], 1)
    copies[3, 0], copies[4, 2], copies[5, 2] = -1, 0, bs + 5
    kv = torch.randn(((layers or 1), nb, bs, 576)).to(torch.bfloat16)
    shape = kv.shape if layers else kv.shape[1:]
    d = kv.view(shape).cuda()
    assert sfa.kv_copy_blocks(d, i32(copies)) is d
    assert np.array_equal(d.float().cpu().numpy().reshape(kv.shape), tree.copy_blocks(kv.float().numpy(), copies))
    codes = torch.randint(0, 256, kv.shape, dtype=torch.uint8)
    scales = torch.rand((layers or 1, nb, bs // group))
    k8, sc = codes.view(shape).cuda().view(torch.float8_e4m3fn), scales.view(shape[:-2] + (bs // group,)).cuda()
    sfa.kv_copy_blocks_q8(k8, sc, i32(copies))
    assert np.array_equal(k8.view(torch.uint8).cpu().numpy().reshape(kv.shape), tree.copy_blocks(codes.numpy(), copies))
    g = copies.copy()
    g[:, 2] = -(-np.minimum(copies[:, 2], bs) // group)
    assert np.array_equal(sc.cpu().numpy().reshape(scales.shape), tree.copy_blocks(scales.numpy()[..., None], g)[..., 0])
    assert sfa.last_device_status() == 0


def test_copies_of_blocks_that_do_not_exist():
    kv = torch.randn((4, 16, 576)).to(torch.bfloat16).cuda()
    before = kv.clone()
    for c in ([4, 0, 16], [0, 4, 16], [1, -1, 16], [2 ** 31 - 1, 0, 3]):
        sfa.kv_copy_blocks(kv, i32([c]))
        assert sfa.last_device_status() == BAD_BLOCK and torch.equal(kv, before)
    sfa.kv_copy_blocks(kv, i32([[0, 1, -7], [-1, 9, 9]]))
    assert sfa.last_device_status() == 0 and torch.equal(kv, before)
    sfa.kv_copy_blocks(kv, i32(np.zeros((0, 3))))
    assert torch.equal(kv, before)


def test_rows_past_two_gigabytes():
    kv = torch.zeros((2, 9000, 128, 576), dtype=torch.bfloat16, device="cuda")        # 2.6 GB
    kv[:, 8990] = 3.0
    sfa.kv_copy_blocks(kv, i32([[8990, 8999, 128], [8990, 0, 1]]))
    assert bool((kv[:, 8999] == 3).all()) and bool((kv[:, 0, 0] == 3).all()) and not bool(kv[:, 0, 1:].any())
    kv[:, 8999, 100:] = 5.0
    table = np.full((1, 3), 8999)
    sfa.kv_commit(kv, i32(table), i32([90]), i32([[10, 12]]), i32([2]))
    assert bool((kv[:, 8999, 90:92] == 5).all()) and bool((kv[:, 8999, 92:100] == 3).all())
    assert sfa.last_device_status() == 0


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("captured", [False, True])
def test_fork_decode_free_compact(captured):
    """Requests fork, their copies attend as their sources do, write rows of their own, some end, and
    the pool is compacted: what each row reads stays what it was."""
    rng = np.random.default_rng(9)
    bs, R, F, h = 8, 6, 10, 4
    lens = np.concatenate([rng.integers(1, 60, R), np.zeros(F, int)])
    table, shares, free, taken, nb = pool(rng, lens, bs, 40, wide=2)
    kv = torch.randn((nb, bs, 576)).to(torch.bfloat16).cuda()
    T = R + F
    q1 = torch.randn((1, h, 576)).to(torch.bfloat16).cuda().expand(T, h, 576).contiguous()
    start, mask = i32(np.arange(T + 1)), torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    src = rng.integers(0, R, F)
    d = dict(t=i32(table), l=i32(lens), s=i32(shares), f=i32(free), k=i32([taken]), src=i32(src), dst=i32(R + np.arange(F)),
             rows=torch.randn((T, 576)).to(torch.bfloat16).cuda(), keep=i32(np.zeros(T)))
    ended = np.arange(0, T, 3)

    def step():
        copies, k1 = sfa.blocks_fork(d["t"], d["l"], d["src"], d["dst"], d["s"], d["f"], d["k"], bs)
        sfa.kv_copy_blocks(kv, copies)
        same = sfa.decode_tree(q1, kv, d["t"], d["l"], start, mask, 0.1)[0].clone()
        one = torch.ones_like(d["l"])
        table2, seq, _, _, slots, k2 = sfa.step_plan(d["l"], one, d["t"], d["f"], k1, bs, T)
        sfa.kv_write(kv, slots, d["rows"])
        own = sfa.decode_tree(q1, kv, d["t"], seq, start, mask, 0.1)[0].clone()
        k3 = sfa.blocks_free(d["t"], seq, d["keep"], d["s"], d["f"], k2, bs)
        t2, s2, f2, moves = sfa.blocks_compact(d["t"], d["keep"], d["s"], d["f"], k3, bs, 60)
        sfa.kv_copy_blocks(kv, moves)
        last = sfa.decode_tree(q1, kv, t2, d["keep"], start, mask, 0.1)[0].clone()
        return same, own, last, t2, s2, f2, k3, seq

    alive = np.setdiff1d(np.arange(T), ended)
    full = np.concatenate([lens[:R], lens[src]]) + 1
    d["keep"].copy_(i32(np.where(np.isin(np.arange(T), ended), 0, full)))
    if captured:
        saved = {k: v.clone() for k, v in d.items()}
        kv0 = kv.clone()
        step()                                             # first calls of a kernel outside the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            same, own, last, t2, s2, f2, k3, seq = step()
        for k, v in saved.items():
            d[k].copy_(v)
        kv.copy_(kv0)
        g.replay()
    else:
        same, own, last, t2, s2, f2, k3, seq = step()
    assert sfa.last_device_status() == 0
    assert torch.equal(same[R:], same[d["src"].long()])
    assert seq.tolist() == full.tolist()
    assert bool((own[R:] - same[R:]).abs().amax((1, 2)).min() > 0)
    assert torch.equal(last[alive], own[alive]) and not bool(last[ended].any())
    # the pool's books: held blocks are the lowest ones, each counted once or shared
    held = [int(x) for r in alive for x in t2[r, :-(-full[r] // bs)].tolist()]
    assert sorted(set(held)) == list(range(len(set(held))))
    assert [held.count(x) - 1 for x in range(nb) if x in held] == [int(s2[x]) for x in range(nb) if x in held]
    rest = f2[int(k3):].tolist()
    assert rest == list(range(len(set(held)), nb))


# ----------------------------------------------------------------------- two host threads
def test_calls_of_other_sizes_on_two_host_threads():
    """Two threads call at once, each on a stream of its own, with tables whose shared memory differs (above
    what a launch has unasked): neither changes what the other's launches may take.  Straight through the C
    ABI, so that the threads' calls follow one another closely."""
    import threading

    from deepseek_sparse_mla_sfa_gb300 import _lib

    lib = _lib.load()

    def free_of(rows):
        d = [i32(np.full((rows, 1), -1)), i32(np.zeros(rows)), i32([0, 0]), i32([-1, -1]), i32([2]), i32([0])]
        t, z, s, f, k, o = (x.data_ptr() for x in d)
        return d, lambda stream: lib.sfa_blocks_free(t, z, z, rows, 1, s, 2, f, 2, k, 16, o, 0, 0, stream)

    def compact_of(nb, rows):
        d = [i32(np.full((rows, 1), -1)), i32(np.zeros(rows)), i32(np.zeros(nb)), i32([-1]), i32([1])]
        d += [torch.empty_like(d[i]) for i in (0, 2, 3)] + [i32([0] * 3)]
        t, z, s, f, k, t2, s2, f2, c = (x.data_ptr() for x in d)
        return d, lambda stream: lib.sfa_blocks_compact(t, z, rows, 1, s, nb, f, 1, k, 16, 1, t2, s2, f2, c, stream)

    for calls in ((free_of(8192), free_of(5200)), (compact_of(1 << 20, 8192), compact_of(600000, 100))):
        torch.cuda.synchronize()
        codes, gate = [], threading.Barrier(2)

        def work(call):
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            gate.wait()
            for i in range(4000):
                code = call(stream.cuda_stream)
                if code:
                    codes.append(code)
                if i % 100 == 99:
                    stream.synchronize()

        threads = [threading.Thread(target=work, args=(c,)) for _, c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not codes, (len(codes), codes[0])
        assert sfa.last_device_status() == 0


# --------------------------------------------------------------------------- large tables
@pytest.mark.parametrize("shared", [False, True])
def test_free_of_more_entries_than_the_ctas_hold_at_once(shared):
    # 8192 rows of 300 blocks given back: 2.46 million entries, 16168 a CTA, four rounds of 4096
    rng = np.random.default_rng(60)
    R, cols = 8192, 301
    held = rng.integers(290, 301, R)
    table, shares, free, taken, nb = pool(rng, held, 1, 5)
    free = np.concatenate([np.full(nb, -1), free])
    taken += nb
    if shared:
        for r in range(1, R, 3):                            # every third row has the beginning of the one before
            k = int(rng.integers(1, 290))
            table[r, :k] = table[r - 1, :k]
            shares[table[r, :k]] = 1
        keep = np.where(rng.random(R) < 0.1, rng.integers(0, 290, R), 0)
    else:
        keep = np.zeros(R, int)
    assert table.shape[1] == cols
    d = [i32(shares), i32(free)]
    out = sfa.blocks_free(i32(table), i32(held), i32(keep), *d, i32([taken]), 1)
    assert sfa.last_device_status() == 0
    for g, w, name in zip((*d, out), tree.blocks_free(table, held, keep, shares, free, taken, 1), ("shares", "free", "taken")):
        equal(g, w, name)


@pytest.mark.parametrize("moves", [1 << 20, 1000])
def test_compact_of_the_largest_pool(moves):
    # 2^20 blocks: the bitmaps and ranks of a CTA take 80 KB of shared memory, the rows' sums 32 KB
    rng = np.random.default_rng(61)
    R, nb = 8192, 1 << 20
    lens = rng.integers(0, 121, R)
    table, shares, free, taken, total = pool(rng, lens, 1, nb - int(lens.sum()) - 50, lost=50)
    assert total == nb
    for _ in range(500):
        a, b = rng.integers(0, R, 2)
        k = int(rng.integers(0, min(lens[a], lens[b]) + 1))
        table[a, :k] = table[b, :k]
    shares[:] = rng.integers(0, 4, nb)
    got = sfa.blocks_compact(i32(table), i32(lens), i32(shares), i32(free), i32([taken]), 1, moves)
    assert sfa.last_device_status() == 0
    for g, w, name in zip(got, tree.blocks_compact(table, lens, shares, free, taken, 1, moves),
                          ("table", "shares", "free", "copies")):
        equal(g, w, name)


@pytest.mark.parametrize("layers,n,bs", [(61, 3, 7), (5, 300, 64), (7, 9000, 3), (61, 800, 16)])
def test_copies_of_many_layers_with_unused_entries(layers, n, bs):
    # a CTA takes one layer, some or all, by the numbers of copies and layers; most entries are unused
    rng = np.random.default_rng(layers)
    nb = max(40, n // 100)
    used = min(nb // 2, n)
    copies, at = np.full((n, 3), -1), rng.permutation(n)[:used]
    ids = rng.permutation(nb)
    copies[at] = np.stack([ids[:used], ids[used:2 * used], rng.integers(0, bs + 1, used)], 1)
    codes = torch.randint(0, 256, (layers, nb, bs, 576), dtype=torch.uint8)
    scales = torch.rand((layers, nb, bs))
    k8, sc = codes.cuda().view(torch.float8_e4m3fn), scales.cuda()
    sfa.kv_copy_blocks_q8(k8, sc, i32(copies))
    assert sfa.last_device_status() == 0
    assert np.array_equal(k8.view(torch.uint8).cpu().numpy(), tree.copy_blocks(codes.numpy(), copies))
    assert np.array_equal(sc.cpu().numpy(), tree.copy_blocks(scales.numpy()[..., None], copies)[..., 0])
    kv = torch.randn((layers, nb, bs, 576)).to(torch.bfloat16)
    d = sfa.kv_copy_blocks(kv.cuda(), i32(copies))
    assert np.array_equal(d.view(torch.int16).cpu().numpy(), tree.copy_blocks(kv.view(torch.int16).numpy(), copies))


def test_copies_of_nothing_cost_no_cta_a_layer():
    """4096 unused entries of 61 layers, as a compaction that moves nothing leaves them, against one such layer: at
    most ten times as long (one CTA a chunk, entry and layer took 60 times)."""
    kv = torch.zeros((61, 2, 64, 576), dtype=torch.bfloat16, device="cuda")
    copies = i32(np.full((4096, 3), -1))

    def us(x, n=20):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        g = torch.cuda.CUDAGraph()
        sfa.kv_copy_blocks(x, copies)
        with torch.cuda.graph(g):
            for _ in range(n):
                sfa.kv_copy_blocks(x, copies)
        g.replay()
        torch.cuda.synchronize()
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    assert us(kv) < 10 * us(kv[:1])


def test_large_frees_captured_and_on_two_streams():
    """The four launches of a large free, each of which begins while the one before it ends: in a graph that is
    replayed on other lengths, and two frees at once on two streams with workspaces of their own."""
    rng = np.random.default_rng(62)
    sets = []
    for seed in range(2):
        R = 600
        held = rng.integers(0, 1200, R)
        table, shares, free, taken, nb = pool(rng, held, 4, 5, wide=300 - int(held.max()) // 4)
        free = np.concatenate([np.full(nb, -1), free])
        for _ in range(300):
            a, b = rng.integers(0, R, 2)
            k = int(rng.integers(0, min(held[a], held[b]) // 4 + 1))
            table[a, :k] = table[b, :k]
        shares[:] = 700                                     # whatever is named stays or goes by this many names
        shares[rng.random(nb) < 0.7] = 0
        sets.append((table, held, shares, free, taken + nb, nb))
    cols = max(s[0].shape[1] for s in sets)
    ws = [torch.full((max(sfa.blocks_free_workspace_bytes(600, cols), 1),), 255, dtype=torch.uint8, device="cuda") for _ in sets]
    assert ws[0].numel() > 1                                # the large form

    def want(s, keep):
        return tree.blocks_free(s[0], s[1], keep, s[2], s[3], s[4], 4)

    keeps = [np.where(rng.random(600) < 0.4, 0, np.maximum(sets[0][1] - rng.integers(0, 500, 600), 0)) for _ in range(3)]
    s = sets[0]
    d = dict(t=i32(s[0]), h=i32(s[1]), k=i32(keeps[0]), s=i32(s[2]), f=i32(s[3]), n=i32([s[4]]))
    sfa.blocks_free(d["t"], d["h"], d["k"], d["s"], d["f"], d["n"], 4, workspace=ws[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sfa.blocks_free(d["t"], d["h"], d["k"], d["s"], d["f"], d["n"], 4, workspace=ws[0])
    for keep in keeps:
        for x, v in (("k", keep), ("s", s[2]), ("f", s[3])):
            d[x].copy_(i32(v))
        g.replay()
        for got, w, name in zip((d["s"], d["f"], out), want(s, keep), ("shares", "free", "taken")):
            equal(got, w, name)
    sfa.last_device_status()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        ds = [[i32(x) for x in (s[0], s[1], keeps[0] if i == 0 else s[1] // 2, s[2], s[3], [s[4]])] for i, s in enumerate(sets)]
        torch.cuda.synchronize()
        outs = [sfa.blocks_free(*d, 4, workspace=ws[i], stream=streams[i]) for i, d in enumerate(ds)]
        torch.cuda.synchronize()
        for i, (s, dd) in enumerate(zip(sets, ds)):
            for got, w, name in zip((dd[3], dd[4], outs[i]), want(s, keeps[0] if i == 0 else s[1] // 2), ("shares", "free", "taken")):
                equal(got, w, (i, name))
    sfa.last_device_status()
