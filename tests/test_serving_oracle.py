"""CPU pins of the oracle of the serving-step calls, the frequencies of rotary positions, and
the refusals of the bindings and the C ABI that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import deepseek_sparse_mla_sfa_gb300 as sfa
import oracle
from deepseek_sparse_mla_sfa_gb300 import _lib, build
from oracle import serving

P0 = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)   # a non-null, 256-aligned address; never dereferenced here
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ------------------------------------------------------------------------------ oracle
def test_e4m3_codec_matches_torch_on_every_code_and_rounding():
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, serving.E4M3, equal_nan=True)
    # every bf16 value that does not overflow rounds as torch's conversion does
    bits = np.arange(0, 1 << 16, dtype=np.uint32)
    x = serving.bf16_values(bits)
    x = x[np.isfinite(x) & (np.abs(x) <= 448)]
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(serving.to_e4m3(x), want)
    assert serving.to_e4m3(np.array([1e9, -1e9, np.inf, np.nan])).tolist()[:2] == [126, 254]
    assert np.all(np.isnan(serving.E4M3[serving.to_e4m3(np.array([np.inf, -np.inf, np.nan]))]))


def test_write_oracle_closed_forms():
    codes, scales = np.zeros((8, 576), np.uint8), np.zeros(2)
    row = np.full(576, 448.0)
    c, s = serving.kv_write_q8(codes, scales, [0], row[None], 4)
    assert s.tolist() == [1.0, 0.0] and np.all(serving.E4M3[c[0]] == 448.0)
    # a row four times as large: the group goes to scale 4 and its old row keeps its value
    c2, s2 = serving.kv_write_q8(c, s, [2], 4 * row[None], 4)
    assert s2[0] == 4.0 and np.all(serving.E4M3[c2[0]] * 4 == 448.0) and np.all(serving.E4M3[c2[2]] == 448.0)
    # the first slot again: the group starts anew
    c3, s3 = serving.kv_write_q8(c2, s2, [0], row[None] / 2, 4)
    assert s3[0] == 0.5 and np.all(serving.E4M3[c3[0]] == 448.0)
    assert serving.scale_exponent(np.array([448.0])) == 0 and serving.scale_exponent(np.array([449.0])) == 1
    assert serving.scale_exponent(np.zeros(4)) == serving.MIN_EXP


def test_decode_oracle_equals_the_bf16_oracle_on_the_dequantised_cache():
    # power-of-two scales: e4m3 * scale is a bf16 value, so both describe the same problem
    rng = np.random.default_rng(5)
    nb, bs, g, B, Q, h, k = 6, 16, 8, 2, 2, 3, 20
    codes = rng.integers(0, 256, (nb, bs, 576), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    scales = 2.0 ** rng.integers(-12, -6, (nb, bs // g))
    q = torch.from_numpy(rng.standard_normal((B * Q, h, 576))).to(torch.bfloat16)
    bt = rng.permutation(nb).reshape(B, 3).astype(np.int32)
    sl = np.array([40, 33], np.int32)
    idx = rng.integers(-2, 45, (B * Q, k)).astype(np.int32)
    kv = torch.from_numpy(serving.E4M3[codes] * np.repeat(scales, g, axis=1)[..., None]).to(torch.bfloat16)
    prob = oracle.Problem(q, kv, bt, sl, idx, Q, 0.07)
    for n, il in ((1, 0), (3, 0), (3, 4)):
        ro, rl = oracle.decode_ex(prob, n, il)
        out, lse, wabs, wmax = serving.decode_q8(q.double().numpy(), codes, scales, g, bt, sl, idx, np.float32(0.07),
                                                 Q, n, il)
        assert np.allclose(out, ro, atol=1e-6) and np.array_equal(np.isneginf(lse), np.isneginf(rl))
        assert np.allclose(lse[np.isfinite(lse)], rl[np.isfinite(rl)], atol=1e-6)
        assert np.all(wabs >= np.abs(out) - 1e-12) and np.all(wmax >= wabs - 1e-12)


def test_plan_oracle_worked_example():
    # block size 4; request 0 holds 2 blocks (5 positions) and gets 4 more: one fresh block;
    # request 1 is empty and gets 1; request 2 gets nothing
    table = [[7, 3, -1, -1], [-1] * 4, [5, -1, -1, -1]]
    t, seq, start, pos, slots, taken = serving.step_plan([5, 0, 4], [4, 1, 0], table, [9, 8, 6], 1, 4, 7)
    assert t.tolist() == [[7, 3, 8, -1], [6, -1, -1, -1], [5, -1, -1, -1]]
    assert seq.tolist() == [9, 1, 4] and start.tolist() == [0, 4, 5, 5] and taken == 3
    assert pos.tolist() == [5, 6, 7, 8, 0, -1, -1] and slots.tolist() == [13, 14, 15, 32, 24, -1, -1]


def test_rope_oracle_closed_forms():
    x = np.zeros((2, 1, 6))
    x[:, 0] = [1, 0, 0, 2, 9, 9]
    y = serving.rope(x, [1, -1], [math.pi / 2, math.pi], True)
    assert np.allclose(y[0, 0], [0, 1, 0, -2, 9, 9]) and np.array_equal(y[1], x[1])
    y = serving.rope(x, [1, 1], [math.pi / 2, math.pi], False)      # pairs (0, 2) and (1, 3)
    assert np.allclose(y[0, 0], [0, 0, 1, -2, 9, 9])
    z = serving.rope(y, [1, 1], [math.pi / 2, math.pi], False, inverse=True)
    assert np.allclose(z, x)


# ------------------------------------------------------------------------- frequencies
def test_rope_inv_freq_scalings():
    f = sfa.rope_inv_freq(64, device="cpu")
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64)
    assert torch.equal(f, want)
    assert torch.allclose(sfa.rope_inv_freq(64, scaling="linear", factor=8.0, device="cpu"), want / 8, rtol=1e-15)
    ntk = sfa.rope_inv_freq(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and abs(float(ntk[-1] / want[-1]) - 1 / 8) < 1e-12     # the last is divided by the factor
    y = sfa.rope_inv_freq(64, scaling="yarn", factor=40.0, original_len=4096, device="cpu")
    turns = 4096 * want / (2 * math.pi)
    assert torch.equal(y[turns >= 32], want[turns >= 32])
    assert torch.allclose(y[turns <= 1], want[turns <= 1] / 40, rtol=1e-15)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and torch.all(y[mid] < want[mid]) and torch.all(y[mid] > want[mid] / 40)
    assert sfa.rope_mscale(1.0) == 1.0 and abs(sfa.rope_mscale(40.0) - (0.1 * math.log(40) + 1)) < 1e-15


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, scaling="cubic"),
                                dict(rot_dim=8, factor=0.0), dict(rot_dim=8, base=-1.0),
                                dict(rot_dim=2, scaling="ntk"), dict(rot_dim=8, scaling="yarn", beta_fast=1.0)])
def test_rope_inv_freq_refusals(kw):
    with pytest.raises(ValueError):
        sfa.rope_inv_freq(device="cpu", **kw)


# ------------------------------------------------------------------------- C ABI checks
def _decode_q8(lib, **kw):
    a = dict(q=FAKE, kv=FAKE, sc=FAKE, g=8, bt=FAKE, sl=FAKE, idx=FAKE, B=2, Q=1, h=4, k=8, nb=4, bs=64, mb=4,
             scale=0.07, n=1, il=0, flags=0, out=FAKE, lse=FAKE, op=P0, lp=P0)
    a.update(kw)
    return lib.sfa_decode_q8(a["q"], a["kv"], a["sc"], a["g"], a["bt"], a["sl"], a["idx"], a["B"], a["Q"], a["h"],
                             a["k"], a["nb"], a["bs"], a["mb"], a["scale"], a["n"], a["il"], a["flags"], a["out"],
                             a["lse"], a["op"], a["lp"], P0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=P0), -1), (dict(kv=P0), -1), (dict(sc=P0), -1), (dict(sc=ODD), -1), (dict(idx=P0), -1), (dict(out=P0), -1),
    (dict(lse=P0), -1), (dict(g=0), -1), (dict(g=-1), -1), (dict(g=7), -1), (dict(g=128), -1), (dict(h=0), -1),
    (dict(h=129), -2), (dict(n=65), -2), (dict(n=0), -1), (dict(B=-1), -1), (dict(bs=0), -1), (dict(flags=4), -1),
    (dict(il=-1), -1), (dict(scale=float("nan")), -1), (dict(kv=ctypes.c_void_p((1 << 20) + 8)), -1),
    (dict(out=ctypes.c_void_p((1 << 20) + 8)), -1), (dict(n=2), -1), (dict(n=2, op=FAKE, lp=FAKE, lse=P0), -1),
    (dict(nb=1 << 26), -2), (dict(B=0), 0), (dict(B=0, sc=P0, q=P0), 0),
])
def test_decode_q8_argument_checks(lib, kw, code):
    assert _decode_q8(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(), -3), (dict(ws=FAKE, wsb=16 * 32 - 1), -3), (dict(ws=ODD, wsb=1 << 20), -3), (dict(T=0), 0), (dict(T=-1), -1),
    (dict(g=0), -1), (dict(slots=1023), -1), (dict(g=128), -2), (dict(kv=P0), -1), (dict(sc=P0), -1), (dict(sm=P0), -1),
    (dict(rows=P0), -1), (dict(rows=ODD), -1), (dict(kv=ODD), -1), (dict(slots=-64), -1),
])
def test_kv_write_q8_argument_checks(lib, kw, code):
    a = dict(kv=FAKE, sc=FAKE, slots=1024, g=64, sm=FAKE, rows=FAKE, T=3, ws=P0, wsb=0)
    a.update(kw)
    assert lib.sfa_kv_write_q8(a["kv"], a["sc"], a["slots"], a["g"], a["sm"], a["rows"], a["T"], a["ws"], a["wsb"],
                               P0) == code


def test_kv_write_q8_workspace_size(lib):
    assert sfa.kv_write_q8_workspace_bytes(1024, 64) == 16 * 32
    assert sfa.kv_write_q8_workspace_bytes(1024, 1) == 0 and sfa.kv_write_q8_workspace_bytes(0, 8) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -1), (dict(B=8193), -2), (dict(bs=0), -1), (dict(mb=0), -1), (dict(nf=-1), -1), (dict(N=-1), -1),
    (dict(taken=P0), -1), (dict(out=P0), -1), (dict(out=ctypes.c_void_p(2 << 20)), -1), (dict(cached=P0), -1),
    (dict(new=P0), -1), (dict(table=P0), -1), (dict(free=P0), -1), (dict(seq=P0), -1), (dict(start=P0), -1),
    (dict(pos=P0), -1), (dict(slots=P0), -1), (dict(seq=FAKE), -1), (dict(table=ctypes.c_void_p((1 << 20) + 1)), -1),
])
def test_step_plan_argument_checks(lib, kw, code):
    a = dict(cached=FAKE, new=FAKE, B=2, bs=64, table=FAKE, mb=4, free=FAKE, nf=8, taken=ctypes.c_void_p(2 << 20), N=4,
             seq=ctypes.c_void_p(3 << 20), start=FAKE, pos=FAKE, slots=FAKE, out=FAKE)
    a.update(kw)
    assert lib.sfa_step_plan(a["cached"], a["new"], a["B"], a["bs"], a["table"], a["mb"], a["free"], a["nf"],
                             a["taken"], a["N"], a["seq"], a["start"], a["pos"], a["slots"], a["out"], P0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), 0), (dict(T=-1), -1), (dict(n=0), -1), (dict(rot=0), -1), (dict(rot=7), -1), (dict(rot=66), -1),
    (dict(width=1024, rot=514), -2), (dict(dtype=3), -1), (dict(flags=4), -1), (dict(m=float("inf")), -1),
    (dict(x=P0), -1), (dict(out=P0), -1), (dict(pos=P0), -1), (dict(f=P0), -1), (dict(f=ODD), -1),
    (dict(x=ODD, dtype=2), -1), (dict(out=FAKE, os=65), -1), (dict(os=0), -1), (dict(n=2, oh=0), -1),
])
def test_rope_argument_checks(lib, kw, code):
    a = dict(x=FAKE, xs=64, out=ctypes.c_void_p(2 << 20), os=64, dtype=0, T=3, n=1, width=64, rot=64, pos=FAKE, f=FAKE,
             m=1.0, flags=0, oh=64)
    a.update(kw)
    assert lib.sfa_rope(a["x"], a["xs"], 64, a["out"], a["os"], a["oh"], a["dtype"], a["T"], a["n"], a["width"], a["rot"],
                        a["pos"], a["f"], a["m"], a["flags"], P0) == code


# -------------------------------------------------------------------- binding refusals
def test_bindings_refuse_what_is_not_on_a_cuda_device():
    i = torch.zeros(2, dtype=torch.int32)
    kv8 = torch.zeros((2, 16, 576), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.step_plan(i, i, i.view(2, 1), i, i[:1], 16, 2)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.rope(torch.zeros((2, 1, 8)), i, torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="CUDA"):
        sfa.kv_write_q8(kv8, torch.zeros((2, 2)), i, torch.zeros((2, 576), dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="float8"):
        sfa.decode_q8(None, kv8.view(torch.uint8), torch.zeros((2, 2)), i, i, i, 0.1)
    with pytest.raises(ValueError, match="scales"):
        sfa.decode_q8(None, kv8, torch.zeros((2, 3)), i, i, i, 0.1)
    with pytest.raises(ValueError, match="576"):
        sfa.decode_q8(None, kv8[:, :, :512].contiguous(), torch.zeros((2, 2)), i, i, i, 0.1)
