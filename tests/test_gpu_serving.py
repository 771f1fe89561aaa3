"""GPU parity of the calls around decode over an 8-bit latent cache against the fp64 oracle:
the step plan, rotary positions, the quantising cache write, decode_q8, and a run of them
together as a serving step uses them."""
import math
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import deepseek_sparse_mla_sfa_gb300 as sfa
import oracle
from oracle import serving

pytestmark = pytest.mark.gpu

NO_BLOCKS, BAD_BLOCK, TIMEOUT = -7, -6, -5


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()


def codes_of(kv8):
    return kv8.detach().cpu().view(torch.uint8).numpy()


# --------------------------------------------------------------------------- step plan
def _plan_case(rng, B, bs, max_cached, max_new, room=None, spare=5, width_short=0):
    cached = rng.integers(0, max_cached + 1, B)
    new = rng.integers(0, max_new + 1, B)
    held, need = -(-cached // bs), -(-(cached + new) // bs)
    width = max(1, int(need.max(initial=1)) + 1 - width_short)
    ids = rng.permutation(int(need.sum()) + spare + 8)
    table, at = np.full((B, width), -1), 0
    for b in range(B):
        k = min(int(held[b]), width)
        table[b, :k] = ids[at:at + k]
        at += int(held[b])
    free = ids[at:]
    taken = int(rng.integers(0, 3))
    N = int(new.sum()) + 3 if room is None else room
    return cached, new, table, free, taken, N


def _check_plan(case, bs, status=0):
    cached, new, table, free, taken, N = case
    got = sfa.step_plan(i32(cached), i32(new), i32(table), i32(free), i32([taken]), bs, N)
    assert sfa.last_device_status() == status
    want = serving.step_plan(cached, new, table, free, taken, bs, N)
    for g, w, name in zip(got, want, ("table", "seq_lens", "start", "positions", "slots", "taken")):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name


@pytest.mark.parametrize("B,bs,max_cached,max_new", [
    (1, 64, 0, 1), (1, 1, 5, 3), (3, 64, 200, 1), (64, 64, 5000, 1), (37, 24, 900, 70), (513, 16, 300, 9),
    (8192, 64, 300, 2), (700, 7, 50, 0), (2, 64, 100, 5000),
])
def test_step_plan_matches_oracle(B, bs, max_cached, max_new):
    _check_plan(_plan_case(np.random.default_rng(B * 1000 + bs), B, bs, max_cached, max_new), bs)


@pytest.mark.parametrize("B", [256, 257, 1024, 1025, 4096, 4097])
def test_step_plan_block_sizes_of_the_kernel(B):
    _check_plan(_plan_case(np.random.default_rng(B), B, 16, 40, 5), 16)


def test_step_plan_empty_and_negative_lengths():
    got = sfa.step_plan(i32([]), i32([]), torch.empty((0, 4), dtype=torch.int32, device="cuda"), i32([1]), i32([1]), 16, 3)
    assert got[2].tolist() == [0] and got[3].tolist() == [-1] * 3 and got[5].tolist() == [1]
    # the last request's 10 positions are in two blocks, the second of which its table lacks
    _check_plan(([-5, 3, 10], [2, -7, 1], [[-1, -1], [4, -1], [2, -1]], [9, 8], 0, 4), 8, BAD_BLOCK)
    _check_plan(([-5, 3, 10], [2, -7, 1], [[-1, -1], [4, -1], [2, 5]], [9, 8], 0, 4), 8)


def test_step_plan_reports_what_does_not_fit():
    rng = np.random.default_rng(3)
    c = _plan_case(rng, 9, 8, 40, 30)
    short = int(sum(-(-(a + b) // 8) - -(-a // 8) for a, b in zip(c[0], c[1]))) + c[4] - 2
    _check_plan((c[0], c[1], c[2], c[3][:short], c[4], c[5]), 8, NO_BLOCKS)          # two blocks too few
    _check_plan((c[0], c[1], c[2], c[3][:0], c[4], c[5]), 8, NO_BLOCKS)              # none at all
    _check_plan((*c[:5], int(c[1].sum()) - 4), 8, NO_BLOCKS)                         # no room for four tokens
    _check_plan(_plan_case(rng, 9, 8, 40, 30, width_short=3), 8, NO_BLOCKS)          # the table too narrow
    table = np.array(c[2])
    b = int(np.argmax((c[0] % 8 > 0) & (c[1] > 0)))                                  # its new token joins a held block
    table[b, c[0][b] // 8] = -1
    _check_plan((c[0], c[1], table, c[3], c[4], c[5]), 8, BAD_BLOCK)


def test_step_plan_steps_follow_each_other_in_a_graph():
    # one captured step, replayed with refilled lengths, taken handed on: equal to the
    # oracle's steps one after the other
    rng = np.random.default_rng(8)
    B, bs, N, width = 6, 4, 24, 12
    table, free = np.full((B, width), -1), rng.permutation(80)
    cached, taken = np.zeros(B, np.int64), 0
    d = dict(c=i32(cached), n=i32(np.zeros(B)), t=i32(table), f=i32(free), k=i32([0]))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        sfa.step_plan(d["c"], d["n"], d["t"], d["f"], d["k"], bs, N, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sfa.step_plan(d["c"], d["n"], d["t"], d["f"], d["k"], bs, N)
        d["c"].copy_(out[1])
        d["k"].copy_(out[5])
    d["c"].zero_(), d["k"].zero_(), d["t"].fill_(-1)
    for step in range(4):
        new = rng.integers(0, 5, B)
        d["n"].copy_(i32(new))
        g.replay()
        table, cached, start, pos, slots, taken = serving.step_plan(cached, new, table, free, taken, bs, N)
        assert np.array_equal(out[0].cpu(), table) and np.array_equal(out[3].cpu(), pos)
        assert np.array_equal(out[4].cpu(), slots) and int(out[5]) == taken
    assert sfa.last_device_status() == 0


FIRST_PLAN = """
import sys, numpy as np, torch, deepseek_sparse_mla_sfa_gb300 as sfa
from oracle import serving
i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()
for B in map(int, sys.argv[1:]):
    rng = np.random.default_rng(B)
    cached, new = rng.integers(0, 40, B), rng.integers(0, 3, B)
    held, need = -(-cached // 16), -(-(cached + new) // 16)
    ids, at, table = rng.permutation(int(need.sum()) + 5), 0, np.full((B, 4), -1)
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    N = int(new.sum()) + 3
    got = sfa.step_plan(i32(cached), i32(new), i32(table), i32(ids[at:]), i32([0]), 16, N)
    want = serving.step_plan(cached, new, table, ids[at:], 0, 16, N)
    assert sfa.last_device_status() == 0
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), B
"""


@pytest.mark.parametrize("B", [["6111"], ["6112"], ["6143"], ["6144"], ["8192"], ["6128", "8192", "6128", "40"]])
def test_step_plan_of_thousands_of_requests_as_the_first_of_a_process(B):
    # the sums of more than 6112 requests take more shared memory than a launch has unasked: whether
    # they get it does not depend on the calls before
    r = subprocess.run([sys.executable, "-c", FIRST_PLAN, *B], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


# -------------------------------------------------------------------------------- rope
ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def _check_rope(x, pos, f, out=None, **kw):
    want = serving.rope(x.double().cpu().numpy(), pos.tolist(), f.tolist(), **kw)
    m = abs(kw.get("mscale", 1.0))
    mag = np.abs(x.double().cpu().numpy()).max(axis=-1, keepdims=True) * 2 * m + 1e-30
    got = sfa.rope(x, pos, f, out=out, **kw)
    torch.cuda.synchronize()
    # one rounding of the result, and fp32 arithmetic: the angle to 2^-22 rad, sines and
    # products to a few 2^-24 of the pair's magnitude
    bound = ULP[x.dtype] * np.abs(want) + 2.0 ** -20 * mag + (2.0 ** -24 if x.dtype == torch.float16 else 0)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= bound)
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,n,width,rot", [(1, 1, 2, 2), (5, 3, 64, 64), (70, 1, 64, 48), (3, 128, 72, 64),
                                           (4, 7, 21, 14), (2, 2, 512, 512), (300, 9, 40, 40)])
def test_rope_matches_oracle(dtype, interleaved, T, n, width, rot):
    g = torch.Generator().manual_seed(T + width)
    x = torch.randn((T, n, width), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32).cuda()
    f = sfa.rope_inv_freq(rot, scaling="yarn", factor=40.0)
    _check_rope(x, pos, f, interleaved=interleaved, mscale=1.25)
    _check_rope(x, pos, f, interleaved=interleaved, inverse=True)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_in_place_on_a_strided_part_leaves_the_rest(interleaved):
    g = torch.Generator().manual_seed(2)
    q = torch.randn((6, 5, 576), generator=g).to(torch.bfloat16).cuda()
    before = q.clone()
    pos = i32([0, 7, -1, 99999, 3, -4])
    f = sfa.rope_inv_freq(64)
    want = serving.rope(before[..., 512:].double().cpu().numpy(), pos.tolist(), f.tolist(), interleaved)
    pe = q[..., 512:]
    assert sfa.rope(pe, pos, f, interleaved=interleaved, out=pe) is pe
    assert torch.equal(q[..., :512], before[..., :512])
    assert torch.equal(q[2], before[2]) and torch.equal(q[5], before[5])        # padding rows
    assert torch.equal(q[0], before[0])                                          # position 0 turns nothing
    assert np.all(np.abs(pe.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18)


def test_rope_strides_offsets_and_padding_rows_of_out():
    g = torch.Generator().manual_seed(4)
    src = torch.randn((9, 4, 100), generator=g).cuda()
    pos = i32([5, -1, 2 ** 31 - 1, 0, 1, 2, 3, 4, 123456789])
    f = sfa.rope_inv_freq(32)
    for off in (0, 1, 3):                                  # odd element offsets: no vector access
        dst = torch.full((9, 2, 200), 7.0, device="cuda")
        x, out = src[:, ::2, off:off + 40], dst[..., off:off + 40]
        want = serving.rope(x.double().cpu().numpy(), pos.tolist(), f.tolist())
        want[1] = 7.0                                      # the padding token's rows stay
        sfa.rope(x, pos, f, out=out)
        got = out.double().cpu().numpy()
        # at position 2^31 the oracle's own double angle is off by 2^-22 rad
        assert np.all(np.abs(got - want) <= 2.0 ** -18 * 8)
        assert torch.all(dst[..., :off] == 7.0) and torch.all(dst[..., off + 40:] == 7.0)
    y2 = sfa.rope(src[:, 0, :64], pos, f)                  # [T, width]: one row a token
    assert y2.shape == (9, 64) and torch.equal(y2[1], src[1, 0, :64])


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("rot", [64, 48, 40, 24, 16])
@pytest.mark.parametrize("off", [0, 1, 4, 8, 12])
def test_rope_of_16_bit_types_at_every_alignment(interleaved, rot, off):
    # 8 pairs a thread, 4 or one, by the alignment of rows and the number of pairs
    g = torch.Generator().manual_seed(100 * rot + off)
    src = torch.randn((11, 3, 96), generator=g).to(torch.bfloat16).cuda()
    dst = torch.full((11, 3, 120), 7.0, dtype=torch.bfloat16, device="cuda")
    x, out = src[..., off:off + rot + 8], dst[..., 2 * off:2 * off + rot + 8]
    pos = torch.arange(11, dtype=torch.int32).mul_(977).cuda()
    _check_rope(x, pos, sfa.rope_inv_freq(rot), out=out, interleaved=interleaved)
    assert torch.equal(out[..., rot:], x[..., rot:])
    assert torch.all(dst[..., :2 * off] == 7.0) and torch.all(dst[..., 2 * off + rot + 8:] == 7.0)


@pytest.mark.parametrize("dtype,width,rot", [(torch.bfloat16, 64, 64), (torch.float16, 72, 64), (torch.float32, 21, 14)])
def test_rope_padding_rows_of_a_new_out_are_those_of_x(dtype, width, rot):
    g = torch.Generator().manual_seed(8)
    x = torch.randn((5, 3, width), generator=g).to(dtype).cuda()
    x[1, 0], x[3, 2] = float("nan"), float("inf")          # copied, not multiplied
    pos, f = i32([4, -1, 9, -7, 0]), sfa.rope_inv_freq(rot)
    old = torch.full_like(x, 3.0)
    given = sfa.rope(x, pos, f, out=old.clone())
    for src in (x, x.expand(5, 3, width), x.repeat_interleave(2, dim=1)[:, ::2]):
        new = sfa.rope(src, pos, f)
        bits = lambda t: t.contiguous().view(torch.uint8)
        for t in range(5):
            assert torch.equal(bits(new[t]), bits(x[t] if t in (1, 3) else given[t]))
    assert torch.equal(given[1], old[1]) and torch.equal(given[3], old[3])


def test_rope_of_a_row_shared_by_heads():
    # x expanded over the heads: every head of out gets the rotated row
    g = torch.Generator().manual_seed(5)
    k = torch.randn((7, 1, 32), generator=g).to(torch.float16).cuda()
    pos, f = i32(range(7)), sfa.rope_inv_freq(32)
    out = torch.empty((7, 5, 32), dtype=torch.float16, device="cuda")
    sfa.rope(k.expand(7, 5, 32), pos, f, out=out)
    one = sfa.rope(k, pos, f)
    assert torch.equal(out, one.expand(7, 5, 32))
    with pytest.raises(sfa.SfaError):
        sfa.rope(out, pos, f, out=torch.empty((7, 1, 32), dtype=torch.float16, device="cuda").expand(7, 5, 32))


def test_rope_inverse_is_the_gradient():
    # d/dx sum(g * rope(x)) = rope^T g, against the formula and against differences in fp32
    gen = torch.Generator().manual_seed(6)
    x, gr = (torch.randn((4, 3, 24), generator=gen).cuda() for _ in range(2))
    pos, f = i32([1, 50, 4000, 77777]), sfa.rope_inv_freq(16)
    for il in (True, False):
        grad = sfa.rope(gr, pos, f, interleaved=il, mscale=1.5, inverse=True)
        want = serving.rope(gr.double().cpu().numpy(), pos.tolist(), f.tolist(), il, 1.5, True)
        assert np.all(np.abs(grad.double().cpu().numpy() - want) <= 2.0 ** -18 * 8)
        for at in ((0, 0, 0), (1, 2, 5), (3, 1, 15), (2, 0, 20)):
            e = torch.zeros_like(x)
            e[at] = 0.5
            d = (sfa.rope(x + e, pos, f, interleaved=il, mscale=1.5) - sfa.rope(x - e, pos, f, interleaved=il, mscale=1.5))
            # 16 rounded terms of size <= 8 of a linear map: the difference is exact but for them
            assert abs(float((gr.double() * d.double()).sum()) - float(grad[at])) <= 24 * 16 * 2.0 ** -22


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_of_a_frequency_that_is_no_number(dtype, interleaved):
    # its pair has no angle, at any position that is not padding; the others are as ever
    rng = np.random.default_rng(31)
    x = torch.from_numpy(rng.standard_normal((6, 3, 40))).to(dtype).cuda()
    f = sfa.rope_inv_freq(32)
    pos = i32([0, 1, -1, 77, 2 ** 31 - 1, 5])
    good = sfa.rope(x, pos, f, interleaved=interleaved)
    f[3], f[9], f[10] = float("inf"), float("nan"), float("-inf")
    got = sfa.rope(x, pos, f, interleaved=interleaved)
    spoilt = torch.zeros(40, dtype=torch.bool, device="cuda")
    for i in (3, 9, 10):
        spoilt[[2 * i, 2 * i + 1] if interleaved else [i, i + 16]] = True
    real = pos >= 0
    assert torch.all(torch.isnan(got[real][..., spoilt]))
    assert torch.equal(got[real][..., ~spoilt], good[real][..., ~spoilt]) and torch.equal(got[~real], x[~real])


@pytest.mark.parametrize("f", [3.9, 700.0, 1023.9])
def test_rope_of_fast_frequencies_at_far_positions(f):
    # the angle is known to 2^-32 turns times 2^8 below 1024 rad a position; the oracle's, by 80 digits
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    pos = [1, 12345, 2 ** 20 + 1, 2 ** 31 - 1]
    x = torch.tensor([1.0, 0.0], device="cuda").expand(4, 2).contiguous()
    got = sfa.rope(x, i32(pos), torch.tensor([f], dtype=torch.float64, device="cuda")).double().cpu().numpy()
    turns = [(Decimal(p) * Decimal(f) / (2 * pi)) % 1 for p in pos]
    want = np.array([[math.cos(2 * math.pi * float(t)), math.sin(2 * math.pi * float(t))] for t in turns])
    # 2^-24 turns, 2^-25 turns of the 24 bits that go to the sine, and its rounding
    assert np.all(np.abs(got - want) <= 2 * math.pi * (2.0 ** -24 + 2.0 ** -25) + 2.0 ** -22)


def test_rope_refusals_on_the_gpu():
    x, pos, f = torch.zeros((3, 2, 8), device="cuda"), i32([0, 1, 2]), sfa.rope_inv_freq(8)
    for bad, err in ((lambda: sfa.rope(x.double(), pos, f), TypeError), (lambda: sfa.rope(x, pos[:2], f), ValueError),
                     (lambda: sfa.rope(x, pos.long(), f), TypeError), (lambda: sfa.rope(x, pos, f.float()), TypeError),
                     (lambda: sfa.rope(x[..., :6], pos, f), ValueError), (lambda: sfa.rope(x[..., ::2], pos, f[:1]), ValueError),
                     (lambda: sfa.rope(x, pos, f, out=x[:2]), ValueError), (lambda: sfa.rope(x, pos, f, out=x.half()), ValueError),
                     (lambda: sfa.rope(x, pos, f, mscale=float("nan")), sfa.SfaError),
                     (lambda: sfa.rope(x, pos.cpu(), f), ValueError)):
        with pytest.raises(err):
            bad()
    assert sfa.rope(x[:0], pos[:0], f).shape == (0, 2, 8) and sfa.rope(x[:, :0], pos, f).shape == (3, 0, 8)


# ------------------------------------------------------------------------- cache write
def _cache(rng, num_blocks, bs, group, filled=True):
    codes = rng.integers(0, 256, (num_blocks, bs, 576), dtype=np.uint8) if filled else np.zeros((num_blocks, bs, 576), np.uint8)
    codes[(codes & 127) == 127] = 3
    scales = 2.0 ** rng.integers(-9, 2, (num_blocks, bs // group))
    kv8 = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    ws = torch.zeros(max(16, sfa.kv_write_q8_workspace_bytes(num_blocks * bs, group)), dtype=torch.uint8, device="cuda")
    return codes, scales, kv8, torch.from_numpy(scales).float().cuda(), ws


def _check_write(codes, scales, kv8, sc, ws, slots, rows, group, status=0):
    """rows bf16 [T, 576] (CPU).  Returns the oracle's state, which the cache now equals."""
    sfa.kv_write_q8(kv8, sc, i32(slots), rows.cuda(), workspace=ws)
    assert sfa.last_device_status() == status
    c, s = serving.kv_write_q8(codes.reshape(-1, 576), scales.reshape(-1), slots, rows.double().numpy(), group)
    got = codes_of(kv8).reshape(-1, 576)
    nan = (c & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], c[~nan])
    assert np.array_equal(sc.double().cpu().numpy().reshape(-1), s)
    assert int(ws.sum()) == 0                              # the records are clear again
    return c.reshape(codes.shape), s.reshape(scales.shape)


@pytest.mark.parametrize("bs,group,T", [(64, 64, 1), (64, 64, 100), (64, 16, 333), (16, 8, 7), (24, 3, 50), (64, 1, 40),
                                        (128, 64, 500), (5, 5, 21), (64, 2, 640)])
def test_kv_write_q8_matches_oracle(bs, group, T):
    rng = np.random.default_rng(bs * 100 + T)
    codes, scales, kv8, sc, ws = _cache(rng, 10, bs, group)
    for _ in range(3):                                     # writes that follow each other
        slots = rng.permutation(10 * bs)[:min(T, 10 * bs)].astype(np.int64)
        slots[::5] = -1
        rows = torch.from_numpy(rng.standard_normal((len(slots), 576)) * np.exp(3 * rng.standard_normal((len(slots), 1))))
        codes, scales = _check_write(codes, scales, kv8, sc, ws, slots, rows.to(torch.bfloat16), group)


def test_kv_write_q8_appends_a_sequence_token_by_token():
    rng = np.random.default_rng(1)
    codes, scales, kv8, sc, ws = _cache(rng, 3, 16, 16)
    for t in range(40):
        rows = torch.from_numpy(rng.standard_normal((1, 576)) * 2.0 ** (t % 7)).to(torch.bfloat16)
        codes, scales = _check_write(codes, scales, kv8, sc, ws, np.array([t]), rows, 16)


def test_kv_write_q8_special_values_and_fresh_caches():
    rng = np.random.default_rng(2)
    codes, scales, kv8, sc, ws = _cache(rng, 2, 64, 64, filled=False)
    scales[:] = 0.0                                        # a new cache: no scale yet
    sc.zero_()
    rows = torch.from_numpy(rng.standard_normal((9, 576))).to(torch.bfloat16)
    rows[0] = 0
    rows[1, 3], rows[1, 4], rows[1, 5] = float("inf"), float("-inf"), float("nan")
    rows[2] = 3e38
    rows[3] = 1e-38
    rows[4] = 448.0
    rows[5] = 449.0 * 2                                    # 900 in bf16: needs scale 4
    rows[6] = float("nan")
    rows[7, ::2] = -0.0
    for t in range(9):                                     # one a call: each meets the scales of those before
        codes, scales = _check_write(codes, scales, kv8, sc, ws, np.array([5 * t + 3]), rows[t:t + 1], 64)
    codes, scales, kv8, sc, ws = _cache(rng, 2, 64, 64)
    scales[0, 0], scales[1, 0] = np.nan, np.inf            # scales that no write left: taken as none
    sc.copy_(torch.from_numpy(scales))
    _check_write(codes, scales, kv8, sc, ws, np.array([3, 70]), rows[4:6], 64)


def test_kv_write_q8_bad_slots_repeats_and_nothing_to_do():
    rng = np.random.default_rng(3)
    codes, scales, kv8, sc, ws = _cache(rng, 4, 16, 8)
    rows = torch.from_numpy(rng.standard_normal((4, 576))).to(torch.bfloat16)
    codes, scales = _check_write(codes, scales, kv8, sc, ws, np.array([3, 64, -7, 2 ** 31 - 1]), rows, 8, BAD_BLOCK)
    sfa.kv_write_q8(kv8, sc, i32([]), rows[:0].cuda(), workspace=ws)
    assert np.array_equal(codes_of(kv8), codes)
    # a slot named twice: one of its rows' bytes in each place, the group's other rows and the
    # records as they should be, and the next call right
    sfa.kv_write_q8(kv8, sc, i32([17, 17]), rows[:2].cuda(), workspace=ws)
    torch.cuda.synchronize()
    one = [serving.kv_write_q8(codes.reshape(-1, 576), scales.reshape(-1), [17], np.maximum(np.abs(rows[:2].double().numpy()).max(), 0)
                               * np.ones((1, 576)), 8)][0]
    assert np.array_equal(sc.cpu().double().numpy().reshape(-1), one[1]) and int(ws.sum()) == 0
    got = codes_of(kv8).reshape(-1, 576)
    s17 = one[1][17 // 8]
    a, b = (serving.to_e4m3(rows[t].double().numpy() / s17) for t in (0, 1))
    assert np.all((got[17] == a) | (got[17] == b))
    others = [s for s in range(64) if s != 17]
    assert np.array_equal(got[others], one[0][others])
    _check_write(got.reshape(codes.shape), one[1].reshape(scales.shape), kv8, sc, ws, np.array([18, 17]), rows[2:], 8)
    with pytest.raises(sfa.SfaError):
        sfa.kv_write_q8(kv8, sc, i32([1]), rows[:1].cuda())                     # groups need the workspace
    with pytest.raises(ValueError):
        sfa.kv_write_q8(kv8, sc, i32([1, 2]), rows[:1].cuda(), workspace=ws)


@pytest.mark.parametrize("T", [14, 304, 305, 700])       # one launch, and two
@pytest.mark.parametrize("bs,group", [(16, 8), (64, 64), (64, 1)])
def test_kv_write_q8_few_rows_and_many_agree(T, bs, group):
    # 14 rows among padding: infinities, NaN, zeros, the largest and smallest values, several rows
    # a group, a bad slot, groups that start anew
    rng = np.random.default_rng(T)
    codes, scales, kv8, sc, ws = _cache(rng, 6, bs, group)
    rows = torch.from_numpy(rng.standard_normal((T, 576))).to(torch.bfloat16)
    slots, at = np.full(T, -1, np.int64), np.sort(rng.permutation(T)[:14])
    slots[at] = [3, 4, 70, 5, 6 * bs, 64, 11, 9, 90, 91, 1, 2, 30, 32]
    x = rows[torch.from_numpy(at)]
    x[0, 3], x[0, 4], x[0, 5], x[1] = float("inf"), float("-inf"), float("nan"), 0
    x[2], x[3], x[6], x[7] = 3e38, 1e-38, float("nan"), x[7] * 2.0 ** 40
    rows[torch.from_numpy(at)] = x
    codes, scales = _check_write(codes, scales, kv8, sc, ws, slots, rows, group, BAD_BLOCK)
    # one slot named by three rows: the bytes of one of them in each place
    before = codes_of(kv8).reshape(-1, 576)
    slots[at] = -1
    slots[at[:3]] = 20
    rows[torch.from_numpy(at)] = torch.from_numpy(rng.standard_normal((14, 576))).to(torch.bfloat16)
    sfa.kv_write_q8(kv8, sc, i32(slots), rows.cuda(), workspace=ws)
    got, s20 = codes_of(kv8).reshape(-1, 576), float(sc.reshape(-1)[20 // group])
    # (a group of one slot has a scale for each of the rows, and keeps that of one of them)
    own = [2.0 ** serving.scale_exponent(rows[int(t)].double().numpy()) for t in at[:3]]
    assert group > 1 or s20 in own
    three = [serving.to_e4m3(rows[int(t)].double().numpy() / (s20 if group > 1 else s)) for t, s in zip(at[:3], own)]
    assert np.all((got[20] == three[0]) | (got[20] == three[1]) | (got[20] == three[2]))
    others = [s for s in range(6 * bs) if s // group != 20 // group]
    assert np.array_equal(got[others], before[others]) and int(ws.sum()) == 0
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("T", [40, 400])
def test_kv_write_q8_on_two_streams_and_in_a_graph(T):
    # two caches written at the same time, then a captured write replayed over new rows and slots
    rng = np.random.default_rng(T)
    caches = [_cache(rng, 8, 64, 32) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [[(rng.permutation(512)[:T], torch.from_numpy(rng.standard_normal((T, 576)) * 2.0 ** k).to(torch.bfloat16))
              for k in range(3)] for _ in range(2)]
    dev = [[(i32(s), r.cuda()) for s, r in c] for c in calls]
    torch.cuda.synchronize()
    for k in range(3):
        for j in range(2):
            sfa.kv_write_q8(caches[j][2], caches[j][3], *dev[j][k], workspace=caches[j][4], stream=streams[j])
    torch.cuda.synchronize()
    state = []
    for j in range(2):
        c, s = caches[j][0].reshape(-1, 576), caches[j][1].reshape(-1)
        for slots, rows in calls[j]:
            c, s = serving.kv_write_q8(c, s, slots, rows.double().numpy(), 32)
        got, nan = codes_of(caches[j][2]).reshape(-1, 576), (c & 127) == 127
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], c[~nan])
        assert np.array_equal(caches[j][3].double().cpu().numpy().reshape(-1), s)
        state.append((c, s))
    _, _, kv8, sc, ws = caches[0]
    slots_d, rows_d = dev[0][0][0].clone(), dev[0][0][1].clone()
    slots_d.fill_(-1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sfa.kv_write_q8(kv8, sc, slots_d, rows_d, workspace=ws)
    c, s = state[0]
    for k in range(3):
        slots, rows = rng.permutation(512)[:T], torch.from_numpy(rng.standard_normal((T, 576)) * 3.0 ** k).to(torch.bfloat16)
        slots_d.copy_(i32(slots)), rows_d.copy_(rows)
        g.replay()
        c, s = serving.kv_write_q8(c, s, slots, rows.double().numpy(), 32)
        got, nan = codes_of(kv8).reshape(-1, 576), (c & 127) == 127
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], c[~nan])
        assert np.array_equal(sc.double().cpu().numpy().reshape(-1), s) and int(ws.sum()) == 0
    assert sfa.last_device_status() == 0


# -------------------------------------------------------------------------- decode_q8
def _problem(seed, B, Q, h, S, k, bs=64, group=64, spread=1, pow2=True, S_min=None, max_blocks_extra=0):
    rng = np.random.default_rng(seed)
    sl = rng.integers(S_min if S_min is not None else S, S + 1, B)
    nblk = -(-sl // bs)
    nb = int(nblk.sum()) + 2
    ids, at = rng.permutation(nb), 0
    bt = np.full((B, max(1, int(nblk.max())) + max_blocks_extra), -1)
    for b in range(B):
        bt[b, :nblk[b]] = ids[at:at + nblk[b]]
        at += nblk[b]
    codes = serving.to_e4m3(np.clip(rng.standard_normal((nb, bs, 576)) * 64, -448, 448))
    scales = 2.0 ** (rng.integers(-spread, spread + 1, (nb, bs // group)) - 6.0)
    if not pow2:
        scales = scales * rng.uniform(1.0, 2.0, scales.shape)
    scales = scales.astype(np.float32)
    q = torch.from_numpy(rng.standard_normal((B * Q, h, 576))).to(torch.bfloat16)
    idx = np.full((B * Q, k), -1)
    for t in range(B * Q):
        L = int(sl[t // Q]) - (Q - 1 - t % Q)
        m = min(k, max(L, 0))
        idx[t, :m] = rng.permutation(max(L, 1))[:m]
    return dict(q=q, codes=codes, scales=scales, group=group, bt=bt, sl=sl, idx=idx, Q=Q)


def _device(pr):
    return (pr["q"].cuda(), torch.from_numpy(pr["codes"]).cuda().view(torch.float8_e4m3fn),
            torch.from_numpy(pr["scales"]).cuda(), i32(pr["bt"]), i32(pr["sl"]), i32(pr["idx"]))


SCALE = float(np.float32(192 ** -0.5))


def _oracle(pr, n=1, il=0, per_token=False, scale=SCALE):
    return serving.decode_q8(pr["q"].double().numpy(), pr["codes"], pr["scales"].astype(np.float64), pr["group"],
                             pr["bt"], pr["sl"], pr["idx"], scale, pr["Q"], n, il, per_token)


def _close(out, lse, want, what=""):
    """Elementwise.  A weight w_j c_j is kept as hi + lo in e4m3: hi to 2^-4, lo to 2^-4 of the
    at most 2^-4 that is left, so 2^-8 of the weight; a small one to 2^-10 (half the spacing
    2^-9 of e4m3's smallest values) where the largest weight is at least 8 (16 under power-of-two
    scales), so to 2^-13 of the largest.  An error of w_j c_j reaches out times |e_j|: the bound
    is 2^-8 sum w_j |v_j| + 2^-13 max(w_j c_j) sum |e_j|.  Then fp32 arithmetic (a score to
    1e-3, lse likewise) and the type's rounding."""
    ro, rl, wabs, wmax = want
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert o.shape == ro.shape and l.shape == rl.shape, what
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(l), empty), what
    assert np.all(o[empty] == 0.0) and np.all(np.isfinite(o)), what
    eps = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bound = (2.0 ** -8 + 1e-3) * wabs + 2.0 ** -13 * wmax + eps * np.abs(ro)
    err = np.abs(o - ro)
    assert np.all(err <= bound + 1e-30), f"{what}: {np.max(err / (bound + 1e-30))} of the bound"
    # 1e-3 is the tolerance of lse; it is met with much to spare
    assert np.all(np.abs(l[~empty] - rl[~empty]) <= 1e-3), what


@pytest.fixture(params=[0, 1], ids=["auto", "cuda_core"])
def path(request):
    old = sfa.set_kernel_path(request.param)
    yield request.param
    sfa.set_kernel_path(old)


def _run(pr, n=1, il=0, per_token=False, scale=SCALE, dtype=torch.float32, **kw):
    return sfa.decode_q8(*_device(pr), scale, n_splits=n, Q=pr["Q"], interleave=il, block_table_per_token=per_token,
                         out_dtype=dtype, **kw)


@pytest.mark.parametrize("h", [1, 4, 16, 17, 32, 33, 48, 64, 65, 100, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_q8_head_counts(path, h, dtype):
    pr = _problem(h, 3, 1, h, 700, 300, S_min=200)
    _close(*_run(pr, dtype=dtype), [x[0] for x in _oracle(pr)])
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("k,S", [(1, 1), (1, 900), (2, 30), (31, 400), (95, 400), (96, 400), (97, 400), (193, 1000),
                                 (1000, 999), (4609, 5000), (9000, 9000)])
def test_decode_q8_list_lengths(path, k, S):
    pr = _problem(k, 2, 1, 20, S, k)
    _close(*_run(pr), [x[0] for x in _oracle(pr)])


@pytest.mark.parametrize("h", [1, 17, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("k", [384, 385, 700, 1000, 1537, 2048])
def test_decode_q8_units_shared_by_several_ctas(h, k):
    # by 1, 2, 4 and 8 CTAs a unit (more than four tiles of 96 rows for each CTA of half as many),
    # in both output types and with an empty sequence, whose CTAs have no tile
    pr = _problem(1000 + h + k, 3, 1, h, 2100, k)
    pr["sl"][1] = 0
    want = [x[0] for x in _oracle(pr)]
    for dtype in (torch.float32, torch.bfloat16):
        _close(*_run(pr, dtype=dtype), want, f"{dtype}")
    _close(*_run(pr, 3), want, "three shards")
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("h,B", [(16, 50), (33, 60), (100, 25)])
def test_decode_q8_units_shared_by_two_ctas(h, B):
    # more units than clusters of four that run at once, fewer than of two
    pr = _problem(2000 + h, B, 1, h, 900, 500, S_min=0)
    for dtype in (torch.float32, torch.bfloat16):
        _close(*_run(pr, dtype=dtype), [x[0] for x in _oracle(pr)], f"{dtype}")
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("h,B,k", [(4, 1, 20000), (4, 80, 13000), (64, 1, 12289)])
def test_decode_q8_lists_of_several_segments(h, B, k):
    # lists of more than two of the kernel's 6144-row segments, with every entry used: positions
    # come back (each entry is a term of its own); by one CTA a token and by eight
    pr = _problem(k, B, 1, h, 700, 700)
    rng = np.random.default_rng(k)
    pr["idx"] = np.stack([rng.integers(0, int(n), k) for n in pr["sl"]])
    out, lse = _run(pr)
    for t in (0, B - 1):
        one = dict(pr, q=pr["q"][t:t + 1], bt=pr["bt"][t:t + 1], sl=pr["sl"][t:t + 1], idx=pr["idx"][t:t + 1])
        _close(out[t:t + 1], lse[t:t + 1], [x[0] for x in _oracle(one)], f"token {t}")
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("h,B,k,holes", [(16, 160, 2049, False), (64, 160, 3000, True), (8, 3, 17000, True), (4, 160, 8192, False)])
def test_decode_q8_lists_staged_where_the_gathers_land(h, B, k, holes):
    # lists of more than 2048 entries a CTA wait in the stages that the first gathers fill: by one CTA
    # a token and by several, with and without entries that leave the list; the same bits every time
    pr = _problem(3000 + k, B, 1, h, 500, 500)
    rng = np.random.default_rng(k)
    pr["idx"] = np.stack([rng.integers(0, int(n), k) for n in pr["sl"]])
    if holes:
        pr["idx"][rng.random(pr["idx"].shape) < 0.3] = -1
    d = _device(pr)
    out, lse = sfa.decode_q8(*d, SCALE)
    for t in (0, B - 1):
        one = dict(pr, q=pr["q"][t:t + 1], bt=pr["bt"][t:t + 1], sl=pr["sl"][t:t + 1], idx=pr["idx"][t:t + 1])
        _close(out[t:t + 1], lse[t:t + 1], [x[0] for x in _oracle(one)], f"token {t}")
    for _ in range(10):
        o, l = sfa.decode_q8(*d, SCALE)
        assert torch.equal(o, out) and torch.equal(l, lse)
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("bs,group", [(64, 1), (64, 16), (16, 16), (24, 8), (1, 1), (128, 128), (7, 7), (100, 50)])
def test_decode_q8_block_sizes_and_scale_groups(path, bs, group):
    pr = _problem(bs + group, 2, 2, 40, 333, 200, bs=bs, group=group, S_min=50, max_blocks_extra=3)
    _close(*_run(pr, dtype=torch.bfloat16), [x[0] for x in _oracle(pr)])


@pytest.mark.parametrize("spread,pow2", [(6, True), (20, True), (3, False), (0, True)])
def test_decode_q8_scales_that_differ_between_groups(path, spread, pow2):
    pr = _problem(spread, 2, 1, 33, 640, 300, bs=16, group=8, spread=spread, pow2=pow2)
    if spread == 20:                      # scores of rows up to 2^20 large: keep their range
        pr["q"] = (pr["q"].float() * 2.0 ** -18).to(torch.bfloat16)
    _close(*_run(pr), [x[0] for x in _oracle(pr)])


def _near(out, lse, want, what=""):
    """Elementwise, relative to the output: a softmax weight keeps 8 significant bits (2^-8) at every
    size, then fp32 arithmetic (1e-3) and the type's rounding.  That is what bf16 weights give."""
    ro, rl, wabs, _ = want
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.all(np.isfinite(o)), what
    eps = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -24
    bound = (2.0 ** -8 + 1e-3) * wabs + eps * np.abs(ro)
    err = np.abs(o - ro)
    assert np.all(err <= bound + 1e-30), f"{what}: {np.max(err / (bound + 1e-30))} of the bound"
    assert np.all(np.abs(l - rl) <= 1e-3), what


def _dominated(h, k, share, same=False, group=64, spread=0):
    """k positions of one sequence, position 0's row drawing `share` of head 0's weight (the other heads
    a little more or less) with small values; the rest share what is left nearly evenly (`same`: exactly)
    and their values have a common part, so what is dropped of them does not cancel.  Scores come
    from the 64 rope columns, where q is 1 +- 2 %.  spread: scales of groups apart by up to 2^spread."""
    rng = np.random.default_rng(h + k)
    nb = -(-k // 64)
    scales = 2.0 ** (rng.integers(-spread, spread + 1, (nb, 64 // group)) - 6.0) if spread else np.full((nb, 64 // group), 2.0 ** -6)
    rope = np.zeros((nb, 64, 64)) if same else rng.standard_normal((nb, 64, 64)) * 34.0
    # scale * c * sum(e) = ln(share (k - 1) / (1 - share)) with all 64 columns alike
    rope[0, 0] = math.log(share * (k - 1) / (1.0 - share)) / (64 * SCALE * 2.0 ** -6)
    rel = np.repeat(scales * 2.0 ** 6, group, axis=1)[..., None]
    lat = rng.standard_normal((nb, 64, 512)) * 24.0 + 32.0
    lat[0, 0] = rng.standard_normal(512) * 0.5
    codes = serving.to_e4m3(np.clip(np.concatenate([lat, rope / rel], 2), -448, 448))
    q = np.zeros((1, h, 576))
    q[0, :, 512:] = 1.0 + 0.02 * np.linspace(0.0, -1.0, h)[:, None]
    return dict(q=torch.from_numpy(q).to(torch.bfloat16), codes=codes, scales=scales.astype(np.float32), group=group,
                bt=rng.permutation(nb)[None], sl=np.array([k]), idx=None, Q=1)


def _in_table_order(pr):
    # position p of the sequence is row p of the arrays made above
    for name in ("codes", "scales"):
        a = np.empty_like(pr[name])
        a[pr["bt"][0]] = pr[name]
        pr[name] = a
    return pr


@pytest.mark.parametrize("k", [64, 300, 2048, 32768])
@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("same", [False, True])
def test_decode_q8_a_dominant_row_leaves_the_tail_its_weight(path, k, share, same):
    # the row first, in the middle and last in the list; a token alone (its list goes to several CTAs)
    # and more tokens than SMs (one CTA each)
    pr = _in_table_order(_dominated(24, k, share, same))
    want, rng = None, np.random.default_rng(k)
    orders = []
    for at in (0, k // 2, k - 1):
        rest = 1 + rng.permutation(k - 1)
        orders.append(np.concatenate([rest[:at], [0], rest[at:]]))
    pr["idx"] = orders[0][None]
    want = [x[0] for x in _oracle(pr)]                     # the order of the list does not matter
    for j, order in enumerate(orders):
        _near(*_run(dict(pr, idx=order[None])), want, f"alone, order {j}")
    if path == 1 and k > 2048:
        return                                             # (160 such tokens on CUDA cores take seconds)
    many = dict(pr, q=pr["q"].expand(160, -1, -1).contiguous(), bt=np.repeat(pr["bt"], 160, 0), sl=np.repeat(pr["sl"], 160),
                idx=np.stack([orders[t % 3] for t in range(160)]))
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = _run(many, dtype=dtype)
        for t in range(3):
            _near(out[t:t + 1], lse[t:t + 1], want, f"many, order {t}, {dtype}")
            assert torch.equal(out[t::3][:53], out[t:t + 1].expand(53, -1, -1))
    assert sfa.last_device_status() == 0


@pytest.mark.parametrize("h", [8, 33, 64, 128])
@pytest.mark.parametrize("n,il", [(2, 0), (4, 16), (8, 0)])
def test_decode_q8_a_dominant_row_in_one_of_several_shards(path, h, n, il):
    pr = _in_table_order(_dominated(h, 5000, 0.95, group=16, spread=1))
    pr["idx"] = np.random.default_rng(h).permutation(5000)[None]
    _near(*_run(pr, n, il), [x[0] for x in _oracle(pr)], f"n={n}")


@pytest.mark.parametrize("h", [3, 64, 128])
@pytest.mark.parametrize("others", [0, 5, 700])
def test_decode_q8_a_row_with_all_the_weight_comes_back(path, h, others):
    # one used row, or one 60 nats above the others: out is its values, whatever its weight's rounding.
    # 2^-11 for the half-precision step of the weight, 2^-16 for fp32 arithmetic
    pr = _problem(140 + h, 3, 1, h, 800, others + 1, group=16)
    q = pr["q"].float()
    q[..., 512:] = 1.0
    pr["q"] = q.to(torch.bfloat16)
    want = np.zeros((3, h, 512))
    for t in range(3):
        for j, p in enumerate(pr["idx"][t]):
            b, r = pr["bt"][t][p // 64], p % 64
            c = pr["scales"][b, r // 16]
            pr["codes"][b, r, 512:] = serving.to_e4m3(np.clip((5.0 if j == others // 2 else -8.0) / c, -448, 448))
            pr["codes"][b, r, :512] &= 0x7f if j == others // 2 else 0xff
            if j == others // 2:
                want[t] = serving.E4M3[pr["codes"][b, r, :512]] * float(c)
    pr["q"][..., :512] = 0
    out, lse = _run(pr, scale=0.08)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= (2.0 ** -11 + 2.0 ** -16) * np.abs(want) + 1e-20)
    assert torch.all(torch.isfinite(lse))


@pytest.mark.parametrize("h", [16, 64])
@pytest.mark.parametrize("step", [0.05, 0.7, 6.0, -0.05, -0.7, -6.0])
def test_decode_q8_scores_that_climb_and_fall_through_the_list(path, h, step):
    # a list whose weights change by a factor e^(96 step) from tile to tile, up or down: nearly all of
    # the weight in the last (first) rows, where the first (last) ones are behind 2^-100 of it
    pr = _in_table_order(_dominated(h, 1500, 0.5))
    rope = np.arange(1500) * step / (64 * SCALE * 2.0 ** -6)
    rope = np.clip(rope - rope.min() - 448.0, -448.0, 448.0)       # (e4m3's range; what is beyond is even)
    codes = pr["codes"].copy()
    pos = np.arange(1500)
    codes[pr["bt"][0][pos // 64], pos % 64, 512:] = serving.to_e4m3(np.repeat(rope[:, None], 64, 1))
    pr["codes"] = codes
    q = pr["q"].float()
    q[..., 512:] *= 4.0
    pr["q"] = q.to(torch.bfloat16)
    for order in (pos, pos[::-1], np.random.default_rng(1).permutation(1500)):
        pr["idx"] = order[None].copy()
        _near(*_run(pr), [x[0] for x in _oracle(pr)], f"{step}")


@pytest.mark.parametrize("h,n,il", [(5, 2, 0), (16, 3, 16), (64, 8, 0), (128, 4, 1), (72, 64, 0), (30, 5, 7)])
def test_decode_q8_shards_and_their_merge(path, h, n, il):
    pr = _problem(n, 3, 2, h, 500, 150, bs=16, group=16, S_min=20)
    want = _oracle(pr, n, il)
    op, lp = _run(pr, n, il, merge=False)
    _close(op, lp, want, "partials")
    whole = [x[0] for x in _oracle(pr)]
    _close(*_run(pr, n, il), whole, "merged")
    _close(*_run(pr, n, il, dtype=torch.bfloat16), whole, "merged bf16")


def test_decode_q8_masked_repeated_and_empty_lists(path):
    pr = _problem(77, 4, 2, 24, 300, 128, S_min=100)
    idx = pr["idx"]
    idx[0] = -1                                            # nothing selected
    idx[1] = 299                                           # one position, every entry
    idx[2, ::2] = -1                                       # holes
    idx[3, :] = np.where(np.arange(128) % 3 == 0, idx[3], 10 ** 9)       # behind the sequence
    idx[4, 64:] = idx[4, :64]                              # every position twice
    idx[5] = int(pr["sl"][2])                              # just behind its causal range
    pr["sl"][3] = 0                                        # a sequence of no length
    for n in (1, 3):
        _close(*_run(pr, n), [x[0] for x in _oracle(pr)], f"n={n}")
    pr["idx"] = idx[:, :0]                                 # top_k = 0
    out, lse = _run(pr)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))
    assert sfa.last_device_status() == 0


def test_decode_q8_reads_only_what_is_selected(path):
    # every row and scale that no list names is NaN
    pr = _problem(5, 2, 1, 64, 500, 200, bs=16, group=1)
    used = np.zeros(pr["codes"].shape[:2], bool)
    for t in range(2):
        for p in pr["idx"][t]:
            if p >= 0:
                used[pr["bt"][t, p // 16], p % 16] = True
    pr["codes"][~used] = 127
    pr["scales"][~used] = np.nan
    _close(*_run(pr), [x[0] for x in _oracle(pr)])


@pytest.mark.parametrize("written", ["none", "half"])
@pytest.mark.parametrize("n", [1, 2])
def test_decode_q8_groups_that_no_write_reached(path, written, n):
    # a cache still zero where it was not written (the padding of a captured batch): such rows
    # are rows of zeros, score 0 and count
    pr = _problem(17, 2, 1, 64, 300, 220, bs=16, group=8)
    blank = np.ones(pr["scales"].shape, bool) if written == "none" else np.arange(pr["scales"].size).reshape(-1, 2) % 3 == 0
    pr["scales"][blank] = 0.0
    pr["codes"].reshape(-1, 2, 8, 576)[blank] = 0
    out, lse = _run(pr, n)
    _close(out, lse, [x[0] for x in _oracle(pr)], f"n={n}")
    if written == "none":
        assert torch.all(out == 0)


def test_decode_q8_per_token_tables_and_bad_blocks(path):
    pr = _problem(6, 2, 3, 16, 200, 64, bs=16, group=4)
    rng = np.random.default_rng(1)
    pr["bt"] = np.stack([pr["bt"][t // 3][rng.permutation(pr["bt"].shape[1])] for t in range(6)])
    _close(*_run(pr, per_token=True), [x[0] for x in _oracle(pr, per_token=True)])
    assert sfa.last_device_status() == 0
    bad = dict(pr, bt=pr["bt"].copy(), idx=pr["idx"].copy())
    blk = int(bad["idx"][0, 0]) // 16
    bad["bt"][0, blk] = 10 ** 6                            # skipped and reported
    out, lse = _run(bad, per_token=True)
    assert sfa.last_device_status() == BAD_BLOCK
    bad["idx"][0, bad["idx"][0] // 16 == blk] = -1
    _close(out, lse, [x[0] for x in _oracle(bad, per_token=True)])


@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-4, 3.0])
def test_decode_q8_scales_of_the_scores(path, scale):
    pr = _problem(9, 2, 1, 10, 300, 150)
    if scale == 3.0:                                       # scores of about 70: one row takes most
        pr["q"] = (pr["q"].float() * 0.3).to(torch.bfloat16)
    _close(*_run(pr, scale=scale), [x[0] for x in _oracle(pr, scale=float(np.float32(scale)))])


def test_decode_q8_rising_maxima_and_wide_ranges_of_q(path):
    # rows in ascending order of head 0's score, so its running maximum moves on every tile;
    # heads of very different size, one zero, one with a single large column
    pr = _problem(10, 1, 1, 66, 1200, 1200)
    q = pr["q"].float()
    q[0, 1] *= 1e-20
    q[0, 2] = 0
    q[0, 3] *= 1e-3
    q[0, 3, 7] = 40.0
    q[0, 0] *= 4.0
    pr["q"] = q.to(torch.bfloat16)
    k = serving.E4M3[pr["codes"]] * np.repeat(pr["scales"], pr["group"], axis=1)[..., None]
    pos = np.arange(1200)
    rows = k[pr["bt"][0][pos // 64], pos % 64]
    order = np.argsort(rows @ pr["q"].double().numpy()[0, 0])
    pr["idx"] = order[None, :].copy()
    _close(*_run(pr), [x[0] for x in _oracle(pr)], "ascending")
    pr["idx"] = order[None, ::-1].copy()
    _close(*_run(pr), [x[0] for x in _oracle(pr)], "descending")


def test_decode_q8_infinite_and_nan_queries_spoil_only_their_head(path):
    pr = _problem(11, 2, 1, 18, 200, 100)
    want = [x[0] for x in _oracle(pr)]
    pr["q"][0, 3, 9], pr["q"][1, 17, 570] = float("nan"), float("inf")
    out, lse = _run(pr)
    for t, hh in ((0, 3), (1, 17)):
        assert torch.all(torch.isnan(out[t, hh])) and torch.isnan(lse[t, hh])
        out[t, hh], lse[t, hh] = torch.from_numpy(want[0][t, hh]).float(), float(want[1][t, hh])
    _close(out, lse, want)


@pytest.mark.parametrize("n", [1, 2, 8, 9, 33, 64])
@pytest.mark.parametrize("dv", [512, 20, 7])
def test_merge_of_partials_without_a_number_is_not_empty(n, dv):
    # an lse that is NaN comes from a shard whose result is NaN: so are out and lse, whatever the
    # other shards hold; only a row of -inf throughout is empty
    rng = np.random.default_rng(n)
    op = torch.from_numpy(rng.standard_normal((n, 5, dv))).float()
    lp = torch.from_numpy(rng.standard_normal((n, 5))).float()
    lp[:, 0] = float("nan")                                # every shard
    lp[:, 1], lp[n - 1, 1] = -math.inf, float("nan")       # one, the others empty
    lp[:, 2], lp[0, 2] = 1.0, float("nan")                 # one, beside numbers
    lp[:, 3] = -math.inf                                   # empty
    out, lse = sfa.lse_merge(op.cuda(), lp.cuda())
    assert torch.all(torch.isnan(out[:3])) and torch.all(torch.isnan(lse[:3]))
    assert torch.all(out[3] == 0) and torch.isneginf(lse[3])
    w = torch.softmax(lp[:, 4].double(), 0)
    want, lse4 = (w[:, None] * op[:, 4].double()).sum(0), torch.logsumexp(lp[:, 4].double(), 0)
    # n terms with weights to 2^-20 (expf and the sum), fp32 accumulation
    assert torch.all((out[4].cpu().double() - want).abs() <= 2.0 ** -18 * (w[:, None] * op[:, 4].double().abs()).sum(0) + 1e-30)
    assert abs(float(lse[4]) - float(lse4)) <= 1e-5


@pytest.mark.parametrize("n,il", [(2, 0), (5, 7), (33, 0), (64, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_q8_infinite_and_nan_queries_spoil_their_head_of_merged_shards(n, il, dtype):
    pr = _problem(111, 2, 1, 18, 200, 100)
    want = [x[0] for x in _oracle(pr)]
    pr["q"][0, 3, 9], pr["q"][1, 17, 570] = float("nan"), float("inf")
    out, lse = _run(pr, n, il, dtype=dtype)
    for t, hh in ((0, 3), (1, 17)):
        assert torch.all(torch.isnan(out[t, hh])) and torch.isnan(lse[t, hh])
        out[t, hh], lse[t, hh] = torch.from_numpy(want[0][t, hh]).to(dtype), float(want[1][t, hh])
    _close(out, lse, want)


@pytest.mark.parametrize("k", [1, 2, 3, 5, 97])
@pytest.mark.parametrize("n", [1, 3])
def test_decode_q8_bad_queries_and_rows_over_lists_of_few_entries(path, k, n):
    # fewer entries than warps (or shards) that share them: those without one have nothing to add
    pr = _problem(112, 2, 1, 5, 300, k)
    want = [x[0] for x in _oracle(pr)]
    pr["q"][0, 2, 9], pr["q"][1, 4, 570] = float("nan"), float("-inf")
    out, lse = _run(pr, n)
    for t, hh in ((0, 2), (1, 4)):
        assert torch.all(torch.isnan(out[t, hh])) and torch.isnan(lse[t, hh])
        out[t, hh], lse[t, hh] = torch.from_numpy(want[0][t, hh]).float(), float(want[1][t, hh])
    _close(out, lse, want)
    # a NaN in the rope columns of a selected row: a score of NaN in every head of its token
    p = int(pr["idx"][0, 0])
    pr["q"] = torch.nan_to_num(pr["q"], 0.0, 0.0, 0.0)
    pr["codes"][pr["bt"][0][p // 64], p % 64, 570] = 127
    out, lse = _run(pr, n)
    assert torch.all(torch.isnan(out[0])) and torch.all(torch.isnan(lse[0]))
    assert torch.all(torch.isfinite(out[1])) and torch.all(torch.isfinite(lse[1]))


def test_decode_q8_cache_longer_than_32_bit_offsets(path):
    # 4.6 GB of cache: rows at both ends and in the middle
    nb, bs = 125000, 64
    kv8 = torch.empty((nb, bs, 576), dtype=torch.uint8, device="cuda")
    sc = torch.empty((nb, 1), device="cuda")
    pr = _problem(12, 1, 1, 8, 192, 192)
    at = [0, nb // 2, nb - 1]
    for j, b in enumerate(at):
        kv8[b] = torch.from_numpy(pr["codes"][pr["bt"][0, j]]).cuda()
        sc[b] = float(pr["scales"][pr["bt"][0, j], 0])
    out, lse = sfa.decode_q8(pr["q"].cuda(), kv8.view(torch.float8_e4m3fn), sc, i32([at]), i32([192]), i32(pr["idx"]), SCALE)
    _close(out, lse, [x[0] for x in _oracle(pr)])


def test_decode_q8_more_units_than_sms_and_the_same_bits_again(path):
    pr = _problem(13, 100, 2, 40, 260, 120, bs=16, group=16, S_min=4)
    a = _run(pr)
    _close(*a, [x[0] for x in _oracle(pr)])
    b = _run(pr)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_q8_given_buffers_and_refusals():
    pr = _problem(14, 2, 1, 4, 100, 50)
    d = _device(pr)
    out = torch.full((2, 4, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4), device="cuda")
    o, l = sfa.decode_q8(*d, SCALE, out=out, lse=lse)
    assert o is out and l is lse
    _close(o, l, [x[0] for x in _oracle(pr)])
    for bad in (dict(out=out.half()), dict(out=out[:1]), dict(lse=lse[:1]), dict(out_dtype=torch.float16), dict(Q=3),
                dict(interleave=-1), dict(n_splits=2, out_part=torch.empty((2, 2, 4, 511), device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            sfa.decode_q8(*d, SCALE, **bad)
    with pytest.raises(sfa.SfaError):
        sfa.decode_q8(*d, SCALE, n_splits=65)
    empty = sfa.decode_q8(d[0][:0], d[1], d[2], d[3][:0], d[4][:0], d[5][:0], SCALE)
    assert empty[0].shape == (0, 4, 512)


# ---------------------------------------------------------------- the calls together
def test_a_serving_step_plan_rope_write_topk_decode_uv(path):
    """Three steps of a batch (a prompt, then two decode steps with a padded token room): the
    plan, the rotation of queries and new rows, the 8-bit write, the indexer's lists, decode and
    the W_UV projection, each against the oracle on the state the oracle keeps."""
    rng = np.random.default_rng(21)
    B, bs, group, h, width = 3, 16, 16, 24, 12
    nb = B * width
    table, free = np.full((B, width), -1), rng.permutation(nb)
    cached, taken = np.zeros(B, np.int64), 0
    codes, scales = np.zeros((nb, bs, 576), np.uint8), np.zeros((nb, 1))
    kv8 = torch.zeros((nb, bs, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.zeros((nb, 1), device="cuda")
    ws = torch.zeros(sfa.kv_write_q8_workspace_bytes(nb * bs, group), dtype=torch.uint8, device="cuda")
    f = sfa.rope_inv_freq(64, scaling="yarn", factor=40.0)
    t_d, free_d, k_d, c_d = i32(table), i32(free), i32([0]), i32(cached)
    for step, new in enumerate(([90, 17, 33], [1, 1, 1], [1, 1, 1])):
        N = sum(new) + 5
        t_d, seq_d, start_d, pos_d, slot_d, k_d = sfa.step_plan(c_d, i32(new), t_d, free_d, k_d, bs, N)
        table, cached, _, pos, slots, taken = serving.step_plan(cached, new, table, free, taken, bs, N)
        assert np.array_equal(slot_d.cpu(), slots) and np.array_equal(t_d.cpu(), table)
        c_d = seq_d
        rows = torch.from_numpy(rng.standard_normal((N, 576))).to(torch.bfloat16).cuda()
        ref = rows.double().cpu().numpy()
        want = serving.rope(ref[:, None, 512:], pos, f.tolist())[:, 0]
        sfa.rope(rows[:, 512:], pos_d, f, out=rows[:, 512:])
        assert np.all(np.abs(rows[:, 512:].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 1e-4)
        sfa.kv_write_q8(kv8, sc, slot_d, rows, workspace=ws)
        codes, scales = (x.reshape(y.shape) for x, y in zip(
            serving.kv_write_q8(codes.reshape(-1, 576), scales.reshape(-1), slots, rows.double().cpu().numpy(), group),
            (codes, scales)))
        assert np.array_equal(codes_of(kv8), codes) and np.array_equal(sc.double().cpu().numpy(), scales)
        # the last token of each request attends
        q = torch.from_numpy(rng.standard_normal((B, h, 576))).to(torch.bfloat16).cuda()
        sfa.rope(q[..., 512:], seq_d - 1, f, out=q[..., 512:])
        S = int(cached.max())
        scores = torch.from_numpy(rng.standard_normal((B, -(-S // 4) * 4)).astype(np.float32)).cuda()
        idx = sfa.topk(scores, 40, seq_lens=seq_d, S=S)
        ref_idx = oracle.topk(scores, 40, seq_lens=cached, S=S)
        assert np.array_equal(idx.cpu().numpy(), ref_idx)
        out, lse = sfa.decode_q8(q, kv8, sc, t_d, seq_d, idx, SCALE)
        pr = dict(q=q.cpu(), codes=codes, scales=scales, group=group, bt=table, sl=cached, idx=ref_idx, Q=1)
        _close(out, lse, [x[0] for x in _oracle(pr)], f"step {step}")
        w = (torch.from_numpy(rng.standard_normal((h, 512, 128))) / 512 ** 0.5).to(torch.bfloat16)
        y = sfa.uv_proj(out, w.cuda())
        ry = oracle.uv_proj(out, w)
        b = 2.0 ** -8 * np.einsum("thc,hcv->thv", np.abs(out.double().cpu().numpy()), np.abs(w.double().numpy()))
        assert np.all(np.abs(y.double().cpu().numpy() - ry) <= b + 2.0 ** -8 * np.abs(ry) + 1e-6)
    assert sfa.last_device_status() == 0


def test_two_streams_and_a_graph():
    """The calls on two streams at once over two caches, then captured and replayed with
    refilled inputs: the results are those of calls one after the other."""
    prs = [_problem(30 + j, 3, 1, 40 + 60 * j, 400, 150) for j in range(2)]
    ds = [_device(pr) for pr in prs]
    ref = [[x[0] for x in _oracle(pr)] for pr in prs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for j in range(2):
            got[j].append(sfa.decode_q8(*ds[j], SCALE, n_splits=1 + j, stream=streams[j]))
    torch.cuda.synchronize()
    for j in range(2):
        for o, l in got[j]:
            _close(o, l, ref[j], f"stream {j}")
            assert torch.equal(o, got[j][0][0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = sfa.decode_q8(*ds[0], SCALE, n_splits=2)
    for seed in (40, 41):
        pr = _problem(seed, 3, 1, 40, 400, 150)
        for dst, src in zip(ds[0], _device(pr)):
            dst.copy_(src) if dst.dtype != torch.float8_e4m3fn else dst.view(torch.uint8).copy_(src.view(torch.uint8))
        g.replay()
        _close(o, l, [x[0] for x in _oracle(pr)], f"replay {seed}")
    assert sfa.last_device_status() == 0


FIRST_CALL = """
import torch, deepseek_sparse_mla_sfa_gb300 as sfa
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kv8 = torch.zeros((8, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
sc, q = torch.zeros((8, 1), device="cuda"), torch.ones((2, 16, 576), device="cuda").to(torch.bfloat16)
ws = torch.zeros(sfa.kv_write_q8_workspace_bytes(512, 64), dtype=torch.uint8, device="cuda")
rows, f = torch.ones((8, 576), device="cuda").to(torch.bfloat16), sfa.rope_inv_freq(64)
c, n, t, free, k = i32([0, 0]), i32([3, 5]), i32([[0] * 4] * 2), i32([5, 6, 7]), i32([0])
idx = torch.arange(500, device="cuda").to(torch.int32).repeat(2, 1)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    table, sl, start, pos, slots, _ = sfa.step_plan(c, n, t, free, k, 64, 8)
    y = sfa.rope(q[..., 512:], pos[:2], f)
    sfa.kv_write_q8(kv8, sc, slots, rows, workspace=ws)
    out, lse = sfa.decode_q8(q, kv8, sc, table, sl, idx, 0.01, n_splits=2)
g.replay()
torch.cuda.synchronize()
want = 5.76 + torch.tensor([3.0, 5.0], device="cuda").log()[:, None]
assert sfa.last_device_status() == 0, sfa.last_device_status()
assert (out - 1).abs().max() <= 2.0 ** -8 + 1e-3, (out - 1).abs().max()
assert (lse - want).abs().max() <= 1e-3, (lse - want).abs().max()
"""


def test_first_calls_of_a_process_may_be_captured():
    # equal rows of ones: out is 1 (a weight to 2^-8, fp32 arithmetic to 1e-3, as in _close; a
    # quotient of sums is not exact), lse 0.01 * 576 + ln of the number of rows
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_calls_from_several_threads():
    prs = [_problem(50 + j, 2, 1, 16 + 50 * j, 600, 500) for j in range(2)]
    ref = [[x[0] for x in _oracle(pr)] for pr in prs]
    ds, errors = [_device(pr) for pr in prs], []
    torch.cuda.synchronize()

    def work(j):
        try:
            s = torch.cuda.Stream()
            got = [sfa.decode_q8(*ds[j], SCALE, stream=s) for _ in range(20)]
            s.synchronize()
            for o, l in got:
                _close(o, l, ref[j], f"thread {j}")
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors[0]
    assert sfa.last_device_status() == 0


# ------------------------------------------------------------------- bounded waits
@pytest.mark.parametrize("h,n,B,k", [(4, 1, 2, 600), (64, 1, 3, 600), (128, 2, 2, 900), (64, 1, 160, 200), (30, 1, 1, 7000)])
def test_decode_q8_reports_a_wait_that_runs_out_and_recovers(h, n, B, k):
    # the score issuer first waits on a barrier that nothing completes: the call reports the
    # timeout, every warp leaves, and the next call is right
    pr = _problem(50 + h, B, 1, h, max(k, 300), k, bs=16, group=16)
    d = _device(pr)
    limit, stall = sfa.set_wait_limit(200), sfa.set_stall_injection(True)
    try:
        sfa.decode_q8(*d, SCALE, n_splits=n)
        assert sfa.last_device_status() == TIMEOUT
    finally:
        sfa.set_wait_limit(limit)
        sfa.set_stall_injection(stall)
    _close(*sfa.decode_q8(*d, SCALE, n_splits=n), [x[0] for x in _oracle(pr)])
    assert sfa.last_device_status() == 0


def test_decode_q8_with_waits_of_a_few_polls():
    # any wait may give up: a call reports a timeout or is right
    pr = _problem(61, 4, 1, 64, 900, 700)
    d, want = _device(pr), [x[0] for x in _oracle(pr)]
    for polls in (1, 2, 5, 20, 100, 1000):
        limit = sfa.set_wait_limit(polls)
        try:
            out, lse = sfa.decode_q8(*d, SCALE)
            status = sfa.last_device_status()
        finally:
            sfa.set_wait_limit(limit)
        assert status in (0, TIMEOUT)
        if status == 0:
            _close(out, lse, want, f"{polls} polls")
    _close(*sfa.decode_q8(*d, SCALE), want)
