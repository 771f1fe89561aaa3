"""GPU parity of a step that verifies drafted trees against the fp64 oracle: plan, attention,
accepted path, commit, and a run of them together over several steps."""
import numpy as np
import pytest
import torch

import deepseek_sparse_mla_sfa_gb300 as sfa
from oracle import tree

pytestmark = pytest.mark.gpu

BAD_BLOCK, TIMEOUT, BAD_TREE = -6, -5, -8


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def trees(rng, nodes, chain=0.3):
    """Parents of trees with these numbers of nodes; node 0 is the root."""
    out = []
    for n in nodes:
        for i in range(n):
            out.append(-1 if i == 0 else i - 1 if rng.random() < chain else int(rng.integers(0, i)))
    return out


# -------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("nodes,most", [
    ([1], 1), ([0, 3, 0], 4), ([64, 1, 63], 64), ([65, 0, 64], 65), ([256, 1, 200], 256), ([5] * 300, 8), ([], 3),
    ([33, 32, 31], 40)])
@pytest.mark.parametrize("before,behind", [(0, 0), (3, 1500)])
def test_plan_matches_oracle(nodes, most, before, behind):
    rng = np.random.default_rng(len(nodes) + most)
    parents = [7] * before + trees(rng, nodes) + [99] * behind
    start = before + np.concatenate([[0], np.cumsum(nodes)]).astype(int)
    cached = rng.integers(0, 1000, len(nodes))
    mask, pos = sfa.tree_plan(i32(parents), i32(start), i32(cached), most)
    assert sfa.last_device_status() == 0
    want, wpos = tree.tree_plan(parents, start, cached, most)
    assert np.array_equal(mask.cpu().numpy(), tree.mask_words(want, -(-most // 64)))
    assert pos.tolist() == wpos


def test_plan_reports_what_is_no_tree():
    for parents in ([-1, 1, 0], [-1, 0, 5], [-1, -2, 1]):
        mask, pos = sfa.tree_plan(i32(parents), i32([0, 3]), i32([4]), 8)
        assert sfa.last_device_status() == BAD_TREE
        want, wpos = tree.tree_plan(parents, [0, 3], [4], 8)
        assert mask.flatten().tolist() == want and pos.tolist() == wpos
    mask, pos = sfa.tree_plan(i32([-1, 0, 1, 2]), i32([0, 4]), i32([4]), 2)       # more nodes than max_nodes
    assert sfa.last_device_status() == BAD_TREE
    assert mask.flatten().tolist() == [1, 3, 0, 0] and pos.tolist() == [4, 5, -1, -1]
    mask, pos = sfa.tree_plan(i32([-1, 0, 1, 2]), i32([0, 9]), i32([-3]), 16)     # beyond the step's tokens
    assert sfa.last_device_status() == 0 and pos.tolist() == [0, 1, 2, 3]


# ------------------------------------------------------------------------------ accept
@pytest.mark.parametrize("nodes,most", [([1], 1), ([0, 3, 0, 9], 9), ([256, 100, 33, 2], 256), ([8] * 301, 8)])
@pytest.mark.parametrize("hit", [0.0, 0.5, 1.0])
def test_accept_matches_oracle(nodes, most, hit):
    rng = np.random.default_rng(most + int(10 * hit))
    parents = trees(rng, nodes, chain=0.7) + [0, 0]
    start = np.concatenate([[0], np.cumsum(nodes)]).astype(int)
    T = len(parents)
    tokens, targets = rng.integers(0, 5, T), rng.integers(0, 5, T)
    for b, n in enumerate(nodes):
        for i in range(1, n):
            if rng.random() < hit:
                targets[start[b] + parents[start[b] + i]] = tokens[start[b] + i]
    cached = rng.integers(0, 100, len(nodes))
    got = sfa.tree_accept(i32(tokens), i32(targets), i32(parents), i32(start), i32(cached), most)
    assert sfa.last_device_status() == 0
    for g, w in zip(got, tree.tree_accept(tokens, targets, parents, start, cached, most)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_accept_of_too_many_nodes_and_bad_parents():
    # parents that point ahead or at themselves never match, so the walk ends
    got = sfa.tree_accept(i32([1, 1, 1, 1]), i32([1] * 4), i32([0, 1, 3, 0]), i32([0, 4]), i32([5]), 4)
    assert sfa.last_device_status() == 0 and got[0].tolist() == [[0, 3, -1, -1]] and got[3].tolist() == [7]
    got = sfa.tree_accept(i32([1] * 4), i32([1] * 4), i32([-1, 0, 1, 2]), i32([0, 4]), i32([5]), 2)
    assert sfa.last_device_status() == BAD_TREE and got[0].tolist() == [[0, 1]] and got[1].tolist() == [2]


# ------------------------------------------------------------------------------ commit
def paged(rng, lens, bs, spare=3):
    n = [-(-int(x) // bs) for x in lens]
    ids, at, table = rng.permutation(sum(n) + spare), 0, np.full((len(lens), max(n, default=0) + 2), -1)
    for b, k in enumerate(n):
        table[b, :k] = ids[at:at + k]
        at += k
    return table, sum(n) + spare


@pytest.mark.parametrize("layers", [None, 1, 3])
@pytest.mark.parametrize("bs", [1, 7, 64])
@pytest.mark.parametrize("B,most", [(1, 1), (5, 8), (70, 33), (2, 256)])
def test_commit_matches_oracle(layers, bs, B, most):
    rng = np.random.default_rng(B + bs)
    cached = rng.integers(0, 90, B)
    path, acc = np.full((B, most), -1), np.zeros(B, int)
    for b in range(B):
        acc[b] = rng.integers(0, most + 1)
        path[b, :acc[b]] = np.sort(rng.permutation(most)[:acc[b]])
    table, nb = paged(rng, cached + most, bs)
    kv = torch.randn((layers or 1, nb, bs, 576)).to(torch.bfloat16)
    want = np.stack([tree.kv_commit(x.float().numpy(), table, cached, path, acc) for x in kv])
    dev = kv.cuda() if layers else kv[0].cuda()
    assert sfa.kv_commit(dev, i32(table), i32(cached), i32(path), i32(acc)) is dev
    assert sfa.last_device_status() == 0
    assert np.array_equal(dev.float().cpu().numpy().reshape(want.shape), want)


def test_commit_of_bad_paths_and_blocks():
    kv = torch.arange(6 * 4, dtype=torch.float32).reshape(6, 4, 1).expand(6, 4, 576).to(torch.bfloat16).cuda()
    rows = lambda x: x[..., 0].flatten().tolist()  # noqa: E731
    base = rows(kv)
    for path, status, moved in (([0, 2, 2], BAD_TREE, {1: 2}), ([2, 1, 3], BAD_TREE, {0: 2}), ([0, 256, 257], BAD_TREE, {}),
                                ([-1, 1, 2], BAD_TREE, {}), ([1, 3, -1], 0, {0: 1, 1: 3})):
        x = kv.clone()
        sfa.kv_commit(x, i32([[0, 1]]), i32([0]), i32([path + [-1] * 5]), i32([3 if path[-1] >= 0 else 2]))
        assert sfa.last_device_status() == status
        want = list(base)
        for a, b in moved.items():
            want[a] = base[b]
        assert rows(x) == want, path
    for table in ([[0, -1]], [[0, 6]]):
        x = kv.clone()
        sfa.kv_commit(x, i32(table), i32([2]), i32([[1, 2, 3]]), i32([3]))        # positions 4 and 5 have no block
        assert sfa.last_device_status() == BAD_BLOCK
        assert rows(x) == [0, 1, 3] + base[3:]
    x = kv.clone()
    sfa.kv_commit(x, i32([[0]]), i32([2 ** 31 - 2]), i32([[1, 2, 3]]), i32([7]))  # behind every table
    assert sfa.last_device_status() == BAD_BLOCK and rows(x) == base


# -------------------------------------------------------------------------------- decode
def problem(seed, cached, nodes, h, bs, most=None, before=0, behind=2, std=1.0):
    rng = np.random.default_rng(seed)
    cached, nodes = np.asarray(cached), np.asarray(nodes)
    most = most or max(int(nodes.max(initial=1)), 1)
    table, nb = paged(rng, cached + nodes, bs)
    g = torch.Generator().manual_seed(seed)
    T = before + int(nodes.sum()) + behind
    start = before + np.concatenate([[0], np.cumsum(nodes)]).astype(int)
    mask, _ = tree.tree_plan([-1] * before + trees(rng, nodes) + [-1] * behind, start, cached, most)
    return dict(q=(torch.randn((T, h, 576), generator=g) * std).to(torch.bfloat16),
                kv=torch.randn((nb, bs, 576), generator=g).to(torch.bfloat16), table=table, cached=cached, start=start,
                mask=mask, most=most, scale=192 ** -0.5)


def device(p):
    return dict(q=p["q"].cuda(), kv=p["kv"].cuda(), block_table=i32(p["table"]), cached_lens=i32(p["cached"]),
                token_start=i32(p["start"]), mask=torch.from_numpy(tree.mask_words(p["mask"], -(-p["most"] // 64))).cuda(),
                scale=p["scale"])


def check(p, got, what=""):
    """Element by element.  Bounds: the weights' rounding to bf16 (half a step, 2^-8 of each), the
    scores' fp32 sums of 576 products (at most 2^-18 of sum |q k|, which moves a weight by as much
    relatively; the same twice for numerator and sum), fp32 sums over the positions and exponentials
    (2^-20), and the rounding of a bf16 result (2^-8)."""
    out, lse = (x.double().cpu().numpy() for x in got)
    w_out, w_lse, wabs, smax = tree.decode_tree(p["q"].double().numpy(), p["kv"].double().numpy(), p["table"], p["cached"],
                                                p["start"], p["mask"], p["scale"], p["most"])
    real = ~np.isnan(w_lse)
    d = 2.0 ** -18 * smax + 2.0 ** -20
    empty = np.isneginf(w_lse)
    assert np.array_equal(np.isneginf(lse) & real, empty), what
    assert np.all(out[empty] == 0), what
    some = real & ~empty
    assert np.all(np.abs(lse - w_lse)[some] <= (d + 2.0 ** -22 * np.abs(w_lse))[some]), what
    tol = (2.0 ** -8 + 2 * d[..., None]) * wabs + (2.0 ** -8 if got[0].dtype == torch.bfloat16 else 2.0 ** -22) * np.abs(w_out)
    assert np.all(np.abs(out - w_out)[some] <= (tol + 1e-30)[some]), (what, np.nanmax((np.abs(out - w_out) / (tol + 1e-30))[some]))
    return real


def run(p, **kw):
    """The call with outputs of its own; what belongs to padding tokens has to stay."""
    d = device(p)
    T, h, _ = p["q"].shape
    out = torch.full((T, h, 512), 7.0, device="cuda", dtype=kw.pop("out_dtype", torch.float32))
    lse = torch.full((T, h), 7.0, device="cuda")
    got = sfa.decode_tree(**d, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    assert sfa.last_device_status() == 0
    real = check(p, got)
    none = torch.from_numpy(~real[:, 0]).cuda()
    assert bool((out[none] == 7).all()) and bool((lse[none] == 7).all())
    return got


@pytest.fixture(params=[0, 1], ids=["auto", "cuda_cores"])
def path(request):
    old = sfa.set_kernel_path(request.param)
    yield request.param
    sfa.set_kernel_path(old)


@pytest.mark.parametrize("cached,nodes,h,bs", [
    ([0], [1], 1, 16), ([1], [1], 3, 16), ([0, 5, 0], [4, 0, 1], 16, 7), ([200], [6], 4, 64),
    ([127, 128, 129], [1, 2, 3], 16, 64), ([63, 64, 65, 120], [9, 8, 1, 60], 8, 16),
    ([300, 10, 77], [16, 3, 8], 128, 64), ([256], [64], 27, 128), ([130], [65], 5, 24), ([5, 400], [130, 7], 2, 16),
    ([900], [256], 1, 64), ([33] * 40, [3] * 40, 16, 16), ([1000, 0, 513], [7, 5, 0], 64, 1), ([640], [5], 72, 4),
    ([700], [3], 100, 40), ([1500], [2], 32, 8)])
def test_decode_matches_oracle(path, cached, nodes, h, bs):
    p = problem(len(cached) + h, cached, nodes, h, bs)
    run(p)
    run(p, out_dtype=torch.bfloat16)


def test_decode_of_long_sequences(path):
    run(problem(3, [9000, 4321], [5, 12], 16, 64))
    run(problem(4, [20011], [2], 3, 16))


@pytest.mark.parametrize("cached,nodes,h", [([70000], [5], 64), ([40000, 300, 33000], [4, 9, 3], 128), ([66000], [33], 4)])
def test_decode_of_units_dealt_in_chunks(cached, nodes, h):
    # several units over more rows than stay in L2: whole units or chunks of them by turns, the rest in ranges
    run(problem(h, cached, nodes, h, 64))


def test_decode_of_many_short_requests(path):
    rng = np.random.default_rng(40)
    for B, h, most in ((300, 4, 3), (1500, 16, 2)):
        run(problem(B, rng.integers(0, 40, B), rng.integers(0, most + 1, B), h, 16))


def test_decode_with_padding_before_and_behind(path):
    run(problem(5, [40, 9], [6, 2], 16, 16, before=5, behind=9))


def test_decode_with_any_mask_and_rows_that_see_nothing(path):
    rng = np.random.default_rng(6)
    for c, n, h in ((0, 20, 16), (0, 70, 4), (130, 33, 8), (0, 130, 2), (126, 5, 128)):
        p = problem(n, [c, 3], [n, 2], h, 16)
        for t in range(n):
            p["mask"][t] = sum(1 << j for j in range(n) if rng.random() < 0.5) if t % 3 else 0
        p["mask"][n - 1] |= 1 << (n + 2)              # a bit behind the last node counts for nothing
        p["most"] = max(p["most"], n + 3)
        run(p)


def test_decode_of_large_scores_and_other_scales(path):
    for scale in (4.0, -0.5, 0.0, 1e-3):
        p = problem(7, [300, 61], [9, 4], 16, 64)
        p["scale"] = scale
        run(p)


def test_decode_rows_that_a_node_does_not_see_do_not_reach_it(path):
    for bad in (float("nan"), float("inf"), -float("inf")):
        for c, n, h in ((5, 9, 16), (120, 17, 128), (256, 70, 3)):
            p = problem(8, [c, 40], [n, 5], h, 16)
            kv = p["kv"].float()
            row = lambda pos: (int(p["table"][0, pos // 16]), pos % 16)  # noqa: E731
            victim = n // 2
            seen = [t for t in range(n) if p["mask"][t] >> victim & 1]
            kv[row(c + victim)] = bad
            for pos in range(c + n, -(-(c + n) // 16) * 16):       # behind the last node
                kv[row(pos)] = bad
            p["kv"] = kv.to(torch.bfloat16)
            d = device(p)
            out, lse = sfa.decode_tree(**d)
            assert sfa.last_device_status() == 0
            o, l = out.cpu(), lse.cpu()
            assert bool((~torch.isfinite(o[seen])).any(-1).all()), "a node that sees the row has no finite result"
            clean = dict(p, kv=torch.where(torch.isfinite(kv), kv, torch.zeros(())).to(torch.bfloat16))
            rest = [t for t in range(n + 5) if t not in seen]
            ref = sfa.decode_tree(**device(clean))
            w = tree.decode_tree(clean["q"].double().numpy(), clean["kv"].double().numpy(), p["table"], p["cached"], p["start"],
                                 p["mask"], p["scale"], p["most"])
            tol = (2.0 ** -8 + 2.0 ** -16 * (1 + w[3][..., None])) * w[2] + 1e-6
            assert np.all(np.abs(o.double().numpy() - w[0])[rest] <= tol[rest])
            assert np.all(np.abs(l.double().numpy() - w[1])[rest] <= 1e-3)
            assert bool(torch.isfinite(ref[0][:n + 5]).all())


def test_decode_of_a_query_that_is_no_number(path):
    p = problem(9, [100, 20], [5, 3], 16, 16)
    p["q"][2, 3, 100] = float("nan")
    p["q"][4, 0, 7] = float("inf")
    out, lse = sfa.decode_tree(**device(p))
    assert sfa.last_device_status() == 0
    bad = torch.zeros((10, 16), dtype=torch.bool)
    bad[2, 3] = bad[4, 0] = True
    assert bool(torch.isnan(out[:8].cpu())[bad[:8]].all()) and not bool(torch.isfinite(lse[:8].cpu()[bad[:8]]).any())
    assert bool(torch.isfinite(out[:8].cpu()[~bad[:8]]).all()) and bool(torch.isfinite(lse[:8].cpu()[~bad[:8]]).all())


@pytest.mark.parametrize("bs", [7, 16, 64])
def test_decode_skips_bad_blocks(path, bs):
    p = problem(10, [200, 30], [6, 4], 8, bs)
    p["table"][0, 1], p["table"][1, 0] = -1, p["kv"].shape[0]
    d = device(p)
    got = sfa.decode_tree(**d)
    assert sfa.last_device_status() == BAD_BLOCK
    check(p, [x.clone() for x in got])


def test_decode_gives_the_same_bits_on_every_call(path):
    p = problem(11, [5000, 700, 3], [16, 1, 30], 32, 64)
    d = device(p)
    first = [x[:47].clone() for x in sfa.decode_tree(**d)]
    for _ in range(5):
        again = sfa.decode_tree(**d)
        assert all(torch.equal(x, y[:47]) for x, y in zip(first, again))


def test_decode_captured_and_replayed_with_other_lengths(path):
    sizes = [([300, 20], [8, 3]), ([10, 2000], [1, 7]), ([0, 0], [4, 8])]
    probs = [problem(20 + i, c, n, 16, 16, most=8, behind=16 - sum(n)) for i, (c, n) in enumerate(sizes)]
    nb, mb = max(p["kv"].shape[0] for p in probs), max(p["table"].shape[1] for p in probs)
    buf = dict(q=torch.zeros((16, 16, 576), dtype=torch.bfloat16, device="cuda"),
               kv=torch.zeros((nb, 16, 576), dtype=torch.bfloat16, device="cuda"), block_table=i32(np.full((2, mb), -1)),
               cached_lens=i32([0, 0]), token_start=i32([0, 0, 0]), mask=torch.zeros((16, 1), dtype=torch.int64, device="cuda"))
    ws = torch.full((max(sfa.decode_tree_workspace_bytes(2, 16, 16), 1),), 255, dtype=torch.uint8, device="cuda")

    def fill(p):
        d = device(p)
        buf["q"].copy_(d["q"])
        buf["kv"][:d["kv"].shape[0]].copy_(d["kv"])
        buf["block_table"][:, :d["block_table"].shape[1]].copy_(d["block_table"])
        for k in ("cached_lens", "token_start", "mask"):
            buf[k].copy_(d[k])

    fill(probs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sfa.decode_tree(**buf, scale=192 ** -0.5, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sfa.decode_tree(**buf, scale=192 ** -0.5, workspace=ws)
    for p in probs + probs[:1]:
        fill(p)
        g.replay()
        torch.cuda.synchronize()
        check(p, got)
    assert sfa.last_device_status() == 0


def test_decode_on_a_stream_of_its_own(path):
    p = problem(12, [600], [9], 16, 64)
    s = torch.cuda.Stream()
    d = device(p)
    torch.cuda.synchronize()
    got = sfa.decode_tree(**d, stream=s)
    s.synchronize()
    check(p, got)


def test_decode_of_nothing(path):
    p = problem(13, [5], [2], 4, 16)
    d = device(p)
    out = torch.full((4, 4, 512), 3.0, device="cuda")
    for kw in (dict(token_start=i32([0, 0])), dict(token_start=i32([4, 4])), dict(token_start=i32([3, 1]))):
        sfa.decode_tree(**dict(d, **kw), out=out)
        assert sfa.last_device_status() == 0 and bool((out == 3).all())
    d = dict(d, block_table=i32(np.zeros((0, 3))), cached_lens=i32([]), token_start=i32([0]))
    sfa.decode_tree(**d, out=out)
    assert sfa.last_device_status() == 0 and bool((out == 3).all())


def test_decode_of_more_nodes_than_the_mask_has_bits(path):
    p = problem(14, [50], [70], 4, 16)                    # two words a node
    d = device(p)
    out = torch.full((72, 4, 512), 3.0, device="cuda")
    sfa.decode_tree(**dict(d, mask=d["mask"][:, :1].contiguous()), out=out)
    assert sfa.last_device_status() == BAD_TREE and bool((out[64:] == 3).all())
    p["most"] = 64
    w = tree.decode_tree(p["q"].double().numpy(), p["kv"].double().numpy(), p["table"], p["cached"], p["start"], p["mask"],
                         p["scale"], 64)
    assert np.nanmax(np.abs(out.double().cpu().numpy() - w[0])[:64]) < 2e-2


@pytest.mark.parametrize("cached,nodes,h,bs", [([3], [4], 16, 16), ([60, 250], [4, 9], 128, 64), ([300], [16], 5, 7)])
def test_decode_in_fp32_is_closer_than_bf16_weights(path, cached, nodes, h, bs):
    # fp32 results take the weights in two bf16 terms: what the second leaves is half a step of half a step, 2^-16 of
    # a weight.  Besides it the scores' 2^-18 sum |q k| (twice, numerator and sum), exponentials (2^-20, twice), and
    # sums of P positions in fp32, each step at most 2^-23 of sum w |v| (by rounding or by cutting off).
    p = problem(50 + h, cached, nodes, h, bs, std=0.1)
    out, lse = sfa.decode_tree(**device(p))
    assert sfa.last_device_status() == 0
    w_out, w_lse, wabs, smax = tree.decode_tree(p["q"].double().numpy(), p["kv"].double().numpy(), p["table"], p["cached"],
                                                p["start"], p["mask"], p["scale"], p["most"])
    real = ~np.isnan(w_lse)
    tol = (2.0 ** -16 + 2 * (2.0 ** -18 * smax + 2.0 ** -20) + 2.0 ** -23 * max(np.add(cached, nodes)))[..., None] * wabs
    assert np.all(np.abs(out.double().cpu().numpy() - w_out)[real] <= (tol + 2.0 ** -22 * np.abs(w_out))[real])


def test_decode_wait_that_runs_out_is_reported_and_the_next_call_is_right():
    p = problem(60, [700, 30], [9, 4], 128, 64)
    d = device(p)
    prev, stall = sfa.set_wait_limit(1000), sfa.set_stall_injection(True)
    try:
        sfa.decode_tree(**d)
        status = sfa.last_device_status()
    finally:
        sfa.set_stall_injection(stall)
        sfa.set_wait_limit(prev)
    assert status == TIMEOUT
    run(p)


def test_decode_on_two_streams_at_once(path):
    probs = [problem(70 + i, c, n, 32, 64) for i, (c, n) in enumerate((([5000, 40], [12, 3]), ([300] * 9, [5] * 9)))]
    ds = [device(p) for p in probs]
    streams = [torch.cuda.Stream() for _ in probs]
    ws = [torch.full((max(sfa.decode_tree_workspace_bytes(len(p["cached"]), p["q"].shape[0], 32), 1),), 255, dtype=torch.uint8,
                     device="cuda") for p in probs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(10):
        for i in (0, 1):
            got[i] = sfa.decode_tree(**ds[i], workspace=ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert sfa.last_device_status() == 0
    for p, x in zip(probs, got):
        check(p, x)


@pytest.mark.parametrize("bs", [64, 24, 7])
def test_decode_of_blocks_past_four_gigabytes(path, bs):
    p = problem(80, [333, 100], [5, 9], 8, bs)
    d = device(p)
    nb = (1 << 22) // bs                                   # 4.8 GB of rows; the sequences' blocks lie at the end
    small, kv = d["kv"], torch.empty((nb, bs, 576), dtype=torch.bfloat16, device="cuda")
    kv[nb - small.shape[0]:] = small
    table = np.where(p["table"] >= 0, p["table"] + nb - small.shape[0], -1)
    got = sfa.decode_tree(**dict(d, kv=kv, block_table=i32(table)))
    assert sfa.last_device_status() == 0
    check(p, got)
    path_, acc = i32([[1, 4, -1], [2, 3, 8]]), i32([2, 3])
    sfa.kv_commit(kv, i32(table), i32(p["cached"]), path_, acc)
    assert sfa.last_device_status() == 0
    want = tree.kv_commit(p["kv"].float().numpy(), p["table"], p["cached"], path_.cpu().numpy(), [2, 3])
    assert np.array_equal(kv[nb - small.shape[0]:].float().cpu().numpy(), want)


def test_decode_of_lengths_behind_the_table(path):
    # positions behind the table have no block: what is left is the attention over the table's own
    for h, n, bs, length in ((16, 5, 16, 4), (8, 3, 7, 2 ** 31 - 1), (128, 2, 64, 70)):
        p = problem(100 + n, [200, 90], [n, 4], h, bs)
        reach = p["table"].shape[1] * bs
        p["table"][0] = np.where(p["table"][0] < 0, p["table"][1, 0], p["table"][0])
        p["cached"][0] = length if length > reach else reach + length
        got = sfa.decode_tree(**device(p))
        assert sfa.last_device_status() == BAD_BLOCK
        p["cached"][0] = reach
        p["table"] = np.concatenate([p["table"], np.full((2, 2), -1)], 1)
        check(p, got, (h, length))


def test_decode_of_requests_whose_tokens_overlap(path):
    p = problem(110, [3], [256], 128, 16, behind=0)
    d = device(p)
    B = 19
    d.update(block_table=d["block_table"].expand(B, -1).contiguous(), cached_lens=d["cached_lens"].expand(B).contiguous(),
             token_start=i32([0, 256] * 10))
    out = torch.full((258, 128, 512), 3.0, device="cuda")
    lse = torch.full((258, 128), 3.0, device="cuda")
    sfa.decode_tree(**d, out=out[:256], lse=lse[:256])
    assert sfa.last_device_status() in (0, BAD_TREE)       # more units than 256 tokens have: refused, or any of them
    assert bool((out[256:] == 3).all()) and bool((lse[256:] == 3).all())
    run(p)


def test_decode_refuses_other_shapes_and_devices():
    p = problem(90, [20], [4], 4, 16)
    d = device(p)
    for kw, err in ((dict(q=d["q"].float()), TypeError), (dict(kv=d["kv"][:, :, :512].contiguous()), ValueError),
                    (dict(mask=d["mask"].int()), TypeError), (dict(mask=d["mask"][:-1]), ValueError),
                    (dict(block_table=d["block_table"].cpu()), ValueError), (dict(cached_lens=d["cached_lens"].cpu()), ValueError),
                    (dict(token_start=d["token_start"][:1]), ValueError), (dict(q=d["q"].transpose(0, 1)), ValueError),
                    (dict(out=torch.empty((6, 4, 512), device="cuda", dtype=torch.float16)), TypeError),
                    (dict(out=torch.empty((5, 4, 512), device="cuda")), ValueError),
                    (dict(lse=torch.empty((6, 4, 1), device="cuda")), ValueError),
                    (dict(workspace=torch.empty(1 << 20, dtype=torch.uint8)), ValueError),
                    (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), sfa.SfaError)):
        with pytest.raises(err):
            sfa.decode_tree(**dict(d, **kw))
    with pytest.raises(ValueError):
        sfa.decode_tree(**dict(d, q=torch.zeros((6, 129, 576), dtype=torch.bfloat16, device="cuda")), out=torch.empty((6, 4, 512), device="cuda"))
    with pytest.raises(sfa.SfaError):
        sfa.decode_tree(**dict(d, q=torch.zeros((6, 129, 576), dtype=torch.bfloat16, device="cuda")))
    assert sfa.last_device_status() == 0


# ------------------------------------------------------------------------------ together
def test_steps_of_drafted_trees():
    """Three steps over one pool: blocks from the step plan, rows by the cache write, attention, path,
    commit, the rejected nodes' blocks back; against the oracle's state throughout."""
    rng = np.random.default_rng(30)
    B, bs, most, h, T, width = 5, 4, 12, 8, 64, 24
    table, free = np.full((B, width), -1), rng.permutation(120)
    kv = torch.zeros((120, bs, 576), dtype=torch.bfloat16)
    cached, taken, shares = np.zeros(B, int), 0, np.zeros(120, int)
    d = dict(kv=kv.cuda(), table=i32(table), free=i32(free), taken=i32([0]), cached=i32(cached), shares=i32(shares))
    for step in range(4):
        nodes = rng.integers(0, most + 1, B)
        parents = trees(rng, nodes, 0.8)
        T0 = len(parents)
        parents += [-1] * (T - T0)
        tokens, targets = rng.integers(0, 3, T), rng.integers(0, 3, T)
        rows = torch.randn((T, 576)).to(torch.bfloat16)
        q = torch.randn((T, h, 576)).to(torch.bfloat16)
        # the framework
        table_d, seq, start, _, slots, taken_d = sfa.step_plan(d["cached"], i32(nodes), d["table"], d["free"], d["taken"], bs, T)
        mask, pos = sfa.tree_plan(i32(parents), start, d["cached"], most)
        sfa.kv_write(d["kv"], slots, rows.cuda())
        out, lse = sfa.decode_tree(q.cuda(), d["kv"], table_d, d["cached"], start, mask, 0.07)
        path, acc, nxt, lens = sfa.tree_accept(i32(tokens), i32(targets), i32(parents), start, d["cached"], most)
        before = d["kv"].clone()
        sfa.kv_commit(d["kv"], table_d, d["cached"], path, acc)
        back = sfa.blocks_free(table_d, seq, lens, d["shares"], d["free"], taken_d, bs)
        assert sfa.last_device_status() == 0
        # the oracle
        from oracle import serving
        table, seq_o, start_o, _, slots_o, taken_o = serving.step_plan(cached, nodes, table, free, taken, bs, T)
        assert np.array_equal(table_d.cpu(), table) and int(taken_d) == taken_o
        m_o, pos_o = tree.tree_plan(parents, start_o, cached, most)
        assert pos.tolist() == pos_o
        flat = kv.view(-1, 576)
        for t, s in enumerate(slots_o):
            if s >= 0:
                flat[s] = rows[t]
        assert torch.equal(before.cpu(), kv)
        p = dict(q=q, kv=kv, table=table, cached=cached, start=start_o, mask=m_o, scale=0.07, most=most)
        check(p, (out, lse))
        p_o, a_o, n_o, l_o = tree.tree_accept(tokens, targets, parents, start_o, cached, most)
        assert np.array_equal(path.cpu(), p_o) and acc.tolist() == a_o.tolist() and nxt.tolist() == n_o.tolist()
        kv = torch.from_numpy(tree.kv_commit(kv.float().numpy(), table, cached, p_o, a_o)).to(torch.bfloat16)
        assert torch.equal(d["kv"].cpu(), kv)
        shares, free, taken = tree.blocks_free(table, seq_o, l_o, shares, free, taken_o, bs)
        assert int(back) == taken and np.array_equal(d["free"].cpu(), free) and lens.tolist() == l_o.tolist()
        cached = l_o
        d["cached"], d["taken"], d["table"] = lens, back, table_d


# ------------------------------------------------------------------- rounding of the weights
@pytest.mark.parametrize("cached,h,bs", [([600], 16, 64), ([300, 1500], 128, 16), ([5000], 3, 64)])
def test_decode_rounding_of_a_heavy_weight_cancels(path, cached, h, bs):
    """out is sum w (1 + r) v / sum w (1 + r) with |r| <= 2^-8, the weights' rounding to bf16, so it is off by at
    most sum w |r| |v - out| / (1 - 2^-8): next to nothing where one position has nearly all of the weight.  The
    heavy position lies in the second tile, below the 2^8 from which the maximum is taken anew, so that its weight
    has bits to round.  Scores move the weights likewise (2^-18 of sum |q k|, exponentials 2^-20), fp32 sums are
    off by at most 2^-23 of sum w |v| a position, and the result's own rounding by 2^-8 of it."""
    p = problem(200 + h, cached, [5] * len(cached), h, bs, std=0.3)
    kv = p["kv"].float()
    kv[..., 512] = 0.0
    p["q"][..., 512] = 1.0
    for b, c in enumerate(cached):
        for pos, boost in ((3, 12.0), (270, 16.5)):
            kv[int(p["table"][b, pos // bs]), pos % bs, 512] = boost / p["scale"]
    p["kv"] = kv.to(torch.bfloat16)
    out, lse = sfa.decode_tree(**device(p), out_dtype=torch.bfloat16)
    assert sfa.last_device_status() == 0
    q, k = p["q"].double(), p["kv"].double()
    check(p, (out, lse))
    for b, (c, n) in enumerate(zip(cached, [5] * len(cached))):
        t0 = int(p["start"][b])
        rows = torch.stack([k[int(p["table"][b, x // bs]), x % bs] for x in range(c + n)])
        for i in range(n):
            seen = list(range(c)) + [c + j for j in range(n) if p["mask"][t0 + i] >> j & 1]
            kk = rows[seen]
            s = p["scale"] * q[t0 + i] @ kk.T
            w, v = torch.softmax(s, -1), kk[:, :512]
            want = w @ v
            away = torch.einsum("hp,hpc->hc", w, (v[None] - want[:, None]).abs())
            d = 2.0 ** -18 * p["scale"] * (q[t0 + i].abs() @ kk.abs().T).amax(-1, keepdim=True) + 2.0 ** -20
            tol = (2.0 ** -8 + 2 * d) * away / (1 - 2.0 ** -8) + 2.0 ** -23 * len(seen) * (w @ v.abs()) + 2.0 ** -8 * want.abs()
            off = (out[t0 + i].double().cpu() - want).abs()
            assert bool((w.amax(-1) > 0.8).all()) and bool((off <= tol + 1e-30).all()), float((off / tol).max())


# ------------------------------------------------------------------------- marked requests
def hide(p, b, value):
    """A row that no other node attends to: the last node of request b, a leaf, holds `value`."""
    n = int(p["start"][b + 1] - p["start"][b])
    bs = p["kv"].shape[1]
    pos = int(p["cached"][b]) + n - 1
    p["kv"][int(p["table"][b, pos // bs]), pos % bs] = value
    return int(p["start"][b]) + n - 1


def test_decode_of_requests_beside_marked_ones_keeps_its_bits():
    """A row of NaN in a branch changes nothing but the nodes that attend to it, and the other requests not at all:
    a request is computed the other way only where it was marked itself, not where it lies between two that were."""
    p = problem(120, [40 + b % 30 for b in range(300)], [4] * 300, 16, 16)
    clean = [x[:1200].cpu() for x in sfa.decode_tree(**device(p))]
    marked = [0, 3, 4, 40, 42, 131, 160, 299]
    own = [hide(p, b, float("nan")) for b in marked]
    got = [x[:1200].cpu() for x in sfa.decode_tree(**device(p))]
    assert sfa.last_device_status() == 0
    rest = [t for t in range(1200) if t // 4 not in marked]
    for c, g in zip(clean, got):
        assert torch.equal(c[rest], g[rest])
    beside = [t for b in marked for t in range(4 * b, 4 * b + 4) if t not in own]
    assert bool(torch.isnan(got[0][own]).all()) and bool(torch.isnan(got[1][own]).all())
    # CUDA cores in fp32 against two bf16 terms (2^-16 of sum w |v|, |v| < 6) and both sides' scores (2^-18 sum |q k|)
    assert float((got[0][beside] - clean[0][beside]).abs().max()) < 6 * (2.0 ** -16 + 4 * 2.0 ** -18 * 0.08 * 576 * 2)


def test_decode_computes_a_marked_request_once():
    """However many CTAs mark it: a marked request costs about a pass on CUDA cores, here of 16 units (up to 32
    marks).  The kernel for every shape is the measure of such a pass."""
    p = problem(121, [4000], [16], 128, 64)
    hide(p, 0, float("nan"))
    d = device(p)

    def ms(n=3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        sfa.decode_tree(**d)
        torch.cuda.synchronize()
        a.record()
        for _ in range(n):
            sfa.decode_tree(**d)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n

    marked = ms()
    old = sfa.set_kernel_path(1)
    try:
        cores = ms()
    finally:
        sfa.set_kernel_path(old)
    assert marked < 4 * cores + 2, (marked, cores)


def test_decode_of_marked_requests_in_a_graph_forgets_them():
    """Marks are of one call: a replay on clean rows gives the bits of a clean call."""
    p = problem(122, [70, 3000, 9], [5, 7, 3], 32, 16)
    d = device(p)
    first = [x[:15].clone() for x in sfa.decode_tree(**d)]
    saved = d["kv"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sfa.decode_tree(**d)
    for bad in (None, 1, None, 0, None):
        d["kv"].copy_(saved)
        if bad is not None:
            q = dict(p, kv=p["kv"].clone())
            hide(q, bad, float("inf"))
            d["kv"].copy_(q["kv"])
        g.replay()
        torch.cuda.synchronize()
        if bad is None:
            assert all(torch.equal(x, y[:15]) for x, y in zip(first, got))
    assert sfa.last_device_status() == 0


# ---------------------------------------------------------------- dealt units, at the bound of two terms
def formula(p, only=None):
    """Per token: the formula in 64 bits with elementary torch operations on the GPU.  Yields (token, out [h, 512], lse
    [h], sum w |v|, sum w |v - out|, the scores' error, positions), for every token or those of `only`."""
    q, kv = p["q"].cuda().double(), p["kv"].cuda().double()
    bs = kv.shape[1]
    for b, c in enumerate(int(x) for x in p["cached"]):
        t0, n = int(p["start"][b]), int(p["start"][b + 1] - p["start"][b])
        table = torch.as_tensor(np.asarray(p["table"][b])).cuda().long()
        pos = torch.arange(c + n, device="cuda")
        rows = kv[table[pos // bs], pos % bs]
        for i in range(n):
            if only is not None and t0 + i not in only:
                continue
            k = rows[torch.tensor([j < c or bool(p["mask"][t0 + i] >> (j - c) & 1) for j in range(c + n)], device="cuda")]
            s = p["scale"] * q[t0 + i] @ k.T
            m = s.amax(-1, keepdim=True)
            e = torch.exp(s - m)
            z = e.sum(-1, keepdim=True)
            w, v = e / z, k[:, :512]
            out = w @ v
            away = torch.stack([w[x] @ (v - out[x]).abs() for x in range(w.shape[0])])
            d = 2.0 ** -18 * abs(p["scale"]) * (q[t0 + i].abs() @ k.abs().T).amax(-1, keepdim=True) + 2.0 ** -20
            yield t0 + i, out, (m + torch.log(z))[:, 0], w @ v.abs(), away, d, k.shape[0], w


def check_two_terms(p, got, only=None):
    """fp32 results: the weights' two bf16 terms leave r, |r| <= 2^-16, of each, and sum w (1 + r) v is divided by sum w, so
    that is off by at most 2^-16 sum w |v| (it does not cancel, as it would divided by sum w (1 + r)).  The scores' error d
    moves numerator and sum alike, d sum w |v - out|, and the other's second order (2 %); sums over P positions are off by
    at most 2^-23 of sum w |v| a position, lse by d and its rounding.  Returns the largest share of the bound that weights
    of one bf16 term would have used."""
    one = 0.0
    for t, out, lse, wabs, away, d, n, w in formula(p, only):
        tol = 2.0 ** -16 * wabs + 2 * d * away + 2.0 ** -23 * n * wabs + 2.0 ** -22 * out.abs()
        assert bool(((got[0][t].double() - out).abs() <= tol).all()), (t, float(((got[0][t].double() - out).abs() / tol).max()))
        assert bool(((got[1][t].double() - lse).abs() <= d[:, 0] + 2.0 ** -22 * lse.abs() + 2.0 ** -23 * n).all()), t
        r = w.bfloat16().double()                     # (as a kernel would: to 8 bits, whatever the scale)
        r = r / w - 1
        top = w.topk(min(8, w.shape[1]), -1).indices   # what the heaviest weights' rounding alone does
        one = max(one, float(((torch.gather(r * w, 1, top).sum(-1, keepdim=True) * out).abs() / tol).max()))
    return one


def heavy(p, positions, low=14.0, high=16.5):
    """Cached positions of every request that have most of the weight, by the rope columns alone: each request's
    `positions` rows get scores of `low` to `high` more than the others'."""
    rng = np.random.default_rng(7)
    kv, bs = p["kv"].float(), p["kv"].shape[1]
    kv[..., 512] = 0.0
    p["q"][..., 512] = 1.0
    for b, c in enumerate(int(x) for x in p["cached"]):
        for pos in rng.integers(0, c, positions):
            kv[int(p["table"][b, pos // bs]), pos % bs, 512] = float(rng.uniform(low, high)) / p["scale"]
    p["kv"] = kv.to(torch.bfloat16)
    return p


DEALT = [
    # (cached, nodes, h, tokens to check): whole units, more than there are pairs; two rounds and a remainder; chunks of
    # few units; chunks of units of several requests, ragged
    ([6000 + 31 * i for i in range(12)], [8] * 12, 128, range(0, 96, 7)),
    ([3300 + 17 * i for i in range(20)], [8] * 20, 128, range(0, 160, 13)),
    ([70000], [5], 64, range(5)),
    ([30000, 41000, 500, 0, 26000], [16, 3, 30, 5, 9], 96, range(0, 63, 4))]


@pytest.mark.parametrize("cached,nodes,h,only", DEALT, ids=["whole", "rounds", "chunks", "ragged"])
def test_decode_of_dealt_units_in_fp32(cached, nodes, h, only):
    p = heavy(problem(130 + h, cached, nodes, h, 64, std=0.3), 3) if min(cached) > 0 else problem(131, cached, nodes, h, 64)
    d = device(p)
    first = [x.clone() for x in sfa.decode_tree(**d)]
    assert sfa.last_device_status() == 0
    one = check_two_terms(p, first, set(only))
    # (behind 2^15 positions the bound of their sums, 2^-23 each, is above a weight's rounding, 2^-8, and hides it)
    if 0 < min(cached) and max(cached) < 1 << 13:
        assert one > 1.5, "the case would not see a second term that is missing"
    T = sum(nodes)
    for _ in range(4):                                     # the same plan and the same bits on every call
        again = sfa.decode_tree(**d)
        assert all(torch.equal(x[:T], y[:T]) for x, y in zip(first, again))
    low = sfa.decode_tree(**d, out_dtype=torch.bfloat16)
    for t, out, _, wabs, away, e, n, _ in formula(p, set(list(only)[:3])):
        tol = (2.0 ** -8 + 2 * e) * away / (1 - 2.0 ** -8) + 2.0 ** -23 * n * wabs + 2.0 ** -8 * out.abs()
        assert bool(((low[0][t].double() - out).abs() <= tol).all())


def test_decode_of_more_requests_than_chunks_are_dealt_of():
    # 257 requests with three units each, over more rows than stay in L2: ranges
    B = 257
    p = heavy(problem(140, [300 + b for b in range(B)], [3] * B, 128, 64, std=0.3), 3)
    d = device(p)
    got = [x.clone() for x in sfa.decode_tree(**d)]
    assert sfa.last_device_status() == 0
    assert check_two_terms(p, got, set(range(0, 3 * B, 37))) > 1.5
    again = sfa.decode_tree(**d)
    assert all(torch.equal(x[:3 * B], y[:3 * B]) for x, y in zip(got, again))


def test_decode_of_overlapping_requests_stays_in_its_workspace():
    """Ten requests name the same 256 tokens: 2560 units of two tiles, where the workspace of 256 tokens holds 256 + 19
    pieces and two for each of 4 slots a pair (at most 128 pairs): always refused, with outputs and what lies
    behind the workspace as they were."""
    p = problem(110, [3], [256], 128, 16, behind=0)
    d = device(p)
    B = 19
    d.update(block_table=d["block_table"].expand(B, -1).contiguous(), cached_lens=d["cached_lens"].expand(B).contiguous(),
             token_start=i32([0, 256] * 10))
    size = sfa.decode_tree_workspace_bytes(B, 256, 128)
    buffer = torch.full((size + (1 << 20),), 90, dtype=torch.uint8, device="cuda")
    out = torch.full((258, 128, 512), 3.0, device="cuda")
    lse = torch.full((258, 128), 3.0, device="cuda")
    sfa.decode_tree(**d, out=out[:256], lse=lse[:256], workspace=buffer[:size])
    assert sfa.last_device_status() == BAD_TREE
    assert bool((out == 3).all()) and bool((lse == 3).all()) and bool((buffer[size:] == 90).all())
    # and what it does do, it does in a workspace of just that size
    B = 1
    size = sfa.decode_tree_workspace_bytes(B, 256, 128)
    buffer.fill_(90)
    d = device(p)
    got = sfa.decode_tree(**d, workspace=buffer[:size])
    assert sfa.last_device_status() == 0 and bool((buffer[size:] == 90).all())
    check(p, got)


# ------------------------------------------------------------------------------ infinities
def test_decode_of_infinities_that_a_node_attends_to(path):
    """A score of -inf has weight 0: from a rope column nothing changes, from a value column that column alone is NaN
    (0 x inf) and lse stays.  A score of +inf makes out and lse of the node and head NaN."""
    for c, n, h in ((40, 5, 16), (700, 9, 128)):
        p = problem(150 + n, [c], [n], h, 16)
        for col in (530, 100):
            kv, pos = p["kv"].clone(), c // 2
            kv[int(p["table"][0, pos // 16]), pos % 16, col] = float("inf")
            q = p["q"][:n, :, col].float()
            out, lse = (x[:n].double().cpu() for x in sfa.decode_tree(**device(dict(p, kv=kv))))
            assert sfa.last_device_status() == 0
            without = p["kv"].clone()                      # the position's weight is 0: as if its score were far below
            without[int(p["table"][0, pos // 16]), pos % 16] = 0
            pw = dict(p, kv=without)
            want = {t: (o.cpu(), l.cpu(), a.cpu(), e.cpu()) for t, o, l, a, _, e, _, _ in formula_without(pw, pos)}
            for t in range(n):
                up, down = q[t] > 0, q[t] < 0
                assert bool(torch.isnan(out[t][up]).all()) and bool(torch.isnan(lse[t][up]).all())
                o, l, a, e = want[t]
                ok = torch.ones(512, dtype=torch.bool)
                if col < 512:
                    ok[col] = False
                    assert bool(torch.isnan(out[t][down][:, col]).all())
                assert bool(((lse[t] - l).abs() <= e[:, 0] + 2.0 ** -22 * l.abs() + 2.0 ** -20)[down].all())
                tol = (2.0 ** -8 + 2 * e) * a + 1e-6
                assert bool(((out[t] - o).abs() <= tol)[down][:, ok].all())


def formula_without(p, pos):
    """`formula` of one request with the cached position `pos` left out."""
    q, kv, bs = p["q"].double(), p["kv"].double(), p["kv"].shape[1]
    c, n = int(p["cached"][0]), int(p["start"][1])
    for i in range(n):
        seen = [j for j in range(c + n) if j != pos and (j < c or p["mask"][i] >> (j - c) & 1)]
        k = torch.stack([kv[int(p["table"][0, j // bs]), j % bs] for j in seen])
        s = p["scale"] * q[i] @ k.T
        w, v = torch.softmax(s, -1), k[:, :512]
        d = 2.0 ** -18 * p["scale"] * (q[i].abs() @ k.abs().T).amax(-1, keepdim=True) + 2.0 ** -20
        yield i, w @ v, torch.logsumexp(s, -1), w @ v.abs(), None, d, len(seen), w
