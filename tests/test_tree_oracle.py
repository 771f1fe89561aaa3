"""CPU checks of the oracle of drafted trees and blocks by hand-made cases, and of the host-side
refusals of their calls (C ABI and binding)."""
import ctypes

import numpy as np
import pytest
import torch

import deepseek_sparse_mla_sfa_gb300 as sfa
from deepseek_sparse_mla_sfa_gb300 import _lib, build
from oracle import tree

P0 = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)   # a non-null, 256-aligned address; never dereferenced here
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


# ------------------------------------------------------------------------- the oracle itself
def test_plan_by_hand():
    #      0          0 (second request)
    #    1   2        1
    #   3     4
    parents = [-1, 0, 0, 1, 2, -1, 0, 7]
    mask, pos = tree.tree_plan(parents, [0, 5, 7], [10, 3], 8)
    assert mask == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b1, 0b11, 0]
    assert pos == [10, 11, 11, 12, 12, 3, 4, -1]
    assert tree.mask_words([1 << 63 | 5, 1 << 64], 2).tolist() == [[-(1 << 63) + 5, 0], [0, 1]]


def test_accept_by_hand():
    parents, tokens = [-1, 0, 0, 1, 2, 2], [9, 5, 6, 7, 8, 8]
    path, acc, nxt, lens = tree.tree_accept(tokens, [6, 0, 8, 0, 4, 3], parents, [0, 6], [20], 6)
    assert path.tolist() == [[0, 2, 4, -1, -1, -1]] and acc == [3] and nxt == [4] and lens == [23]
    kv = np.arange(12.0).reshape(3, 4, 1)                  # positions 20.. in blocks 2, 0: 4 slots each
    table = np.array([[-1] * 5 + [2, 0]])
    got = tree.kv_commit(kv, table, [20], path, acc)
    assert got[2, :, 0].tolist() == [8, 10, 0, 11] and got[0, 0, 0] == 0


def test_attention_by_hand():
    # two nodes, one cached position; the second node sees itself and the cached one only
    kv = np.zeros((1, 4, 576))
    kv[0, 0, 0], kv[0, 1, 1], kv[0, 2, 2] = 1.0, 1.0, 1.0
    q = np.zeros((2, 1, 576))
    q[:, 0, 2] = np.log(3.0)
    out, lse, _, _ = tree.decode_tree(q, kv, np.array([[0]]), [1], [0, 2], [0b1, 0b10], 1.0, 2)
    assert np.allclose(out[0, 0, :3], [0.5, 0.5, 0]) and np.isclose(lse[0, 0], np.log(2))
    assert np.allclose(out[1, 0, :3], [0.25, 0, 0.75]) and np.isclose(lse[1, 0], np.log(4))


def test_blocks_by_hand():
    table = np.array([[5, 3, 7], [9, -1, -1], [-1, -1, -1]])
    t, lens, sh, copies, taken = tree.blocks_fork(table, [10, 2, 0], [0], [2], [0] * 12, [-1, 4, 6], 1, 4)
    assert t[2].tolist() == [5, 3, 4] and lens[2] == 10 and copies.tolist() == [[7, 4, 2]] and taken == 2
    assert [x for x in range(12) if sh[x]] == [3, 5]
    sh, free, taken = tree.blocks_free(t, [10, 2, 10], [0, 2, 4], sh, [-1, -1, 6], 2, 4)
    # 5 keeps its other holder; 3, named twice with one share, is free at its first place, then 7 and
    # 4; the list has room for two, the first is lost
    assert sh.tolist() == [0] * 12 and taken == 0 and free.tolist() == [7, 4, 6]


def test_compact_by_hand():
    table = np.array([[8, 2, 5], [8, 6, -1]])
    sh = np.zeros(10, int)
    sh[8] = 1
    t, s, free, copies = tree.blocks_compact(table, [12, 5], sh, [-1, 7, 0, 3, 9, 1], 1, 4, 2)
    assert copies.tolist() == [[8, 0, 4], [6, 1, 4]] and t.tolist() == [[0, 2, 5], [0, 1, -1]]
    assert s.tolist() == [1] + [0] * 9 and free.tolist() == [-1, 3, 6, 7, 8, 9]


# --------------------------------------------------------------------------------- refusals
def _call(lib, name, defaults, **kw):
    a = dict(defaults)
    a.update(kw)
    return getattr(lib, name)(*a.values())


PLAN = dict(parents=FAKE, start=FAKE, cached=FAKE, B=2, T=4, most=8, mask=FAKE, pos=FAKE, stream=P0)
ACCEPT = dict(tokens=FAKE, targets=FAKE, parents=FAKE, start=FAKE, cached=FAKE, B=2, T=4, most=8, path=FAKE, acc=FAKE,
              nxt=FAKE, lens=FAKE, stream=P0)
COMMIT = dict(kv=FAKE, layers=1, nb=4, bs=16, table=FAKE, mb=2, cached=FAKE, path=FAKE, acc=FAKE, B=2, most=8, stream=P0)
DECODE = dict(q=FAKE, kv=FAKE, table=FAKE, cached=FAKE, start=FAKE, mask=FAKE, B=2, T=4, h=4, most=8, nb=4, bs=16, mb=2,
              scale=0.1, flags=0, out=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40, stream=P0)
FORK = dict(table=FAKE, rows=3, mb=2, lens=FAKE, src=FAKE, dst=FAKE, n=1, shares=FAKE, nb=4, free=FAKE, F=4,
            taken=FAKE, bs=16, copies=FAKE, out=ctypes.c_void_p(1 << 21), stream=P0)
FREE = dict(table=FAKE, held=FAKE, keep=FAKE, rows=3, mb=2, shares=FAKE, nb=4, free=FAKE, F=4, taken=FAKE, bs=16,
            out=ctypes.c_void_p(1 << 21), ws=FAKE, wsb=1 << 20, stream=P0)
COMPACT = dict(table=FAKE, lens=FAKE, rows=3, mb=2, shares=FAKE, nb=4, free=FAKE, F=4, taken=FAKE, bs=16, moves=2,
               t2=ctypes.c_void_p(1 << 21), s2=ctypes.c_void_p(1 << 22), f2=ctypes.c_void_p(1 << 23), copies=FAKE, stream=P0)
COPY = dict(kv=FAKE, layers=1, nb=4, bs=16, copies=FAKE, n=1, stream=P0)
COPY8 = dict(kv=FAKE, scales=FAKE, group=16, layers=1, nb=4, bs=16, copies=FAKE, n=1, stream=P0)


@pytest.mark.parametrize("name,base,kw,code", [
    ("sfa_tree_plan", PLAN, dict(B=-1), -1), ("sfa_tree_plan", PLAN, dict(T=-1), -1),
    ("sfa_tree_plan", PLAN, dict(most=0), -1), ("sfa_tree_plan", PLAN, dict(most=257), -2),
    ("sfa_tree_plan", PLAN, dict(parents=P0), -1), ("sfa_tree_plan", PLAN, dict(start=P0), -1),
    ("sfa_tree_plan", PLAN, dict(mask=ctypes.c_void_p((1 << 20) + 4)), -1), ("sfa_tree_plan", PLAN, dict(T=0), 0),
    ("sfa_tree_accept", ACCEPT, dict(most=0), -1), ("sfa_tree_accept", ACCEPT, dict(most=300), -2),
    ("sfa_tree_accept", ACCEPT, dict(path=P0), -1), ("sfa_tree_accept", ACCEPT, dict(lens=ODD), -1),
    ("sfa_tree_accept", ACCEPT, dict(B=0), 0),
    ("sfa_kv_commit", COMMIT, dict(bs=0), -1), ("sfa_kv_commit", COMMIT, dict(kv=ctypes.c_void_p((1 << 20) + 8)), -1),
    ("sfa_kv_commit", COMMIT, dict(most=257), -2), ("sfa_kv_commit", COMMIT, dict(B=0), 0),
    ("sfa_kv_commit", COMMIT, dict(layers=0), 0), ("sfa_kv_commit", COMMIT, dict(acc=P0), -1),
    ("sfa_decode_tree", DECODE, dict(h=0), -1), ("sfa_decode_tree", DECODE, dict(h=129), -2),
    ("sfa_decode_tree", DECODE, dict(most=257), -2), ("sfa_decode_tree", DECODE, dict(flags=1), -1),
    ("sfa_decode_tree", DECODE, dict(scale=float("nan")), -1), ("sfa_decode_tree", DECODE, dict(mask=P0), -1),
    ("sfa_decode_tree", DECODE, dict(q=ctypes.c_void_p((1 << 20) + 8)), -1),
    ("sfa_decode_tree", DECODE, dict(B=8193), -2), ("sfa_decode_tree", DECODE, dict(nb=1 << 20, bs=1 << 11), -2),
    ("sfa_decode_tree", DECODE, dict(B=0), 0), ("sfa_decode_tree", DECODE, dict(T=0), 0),
    ("sfa_decode_tree", DECODE, dict(lse=P0), -1),
    ("sfa_blocks_fork", FORK, dict(out=FAKE), -1), ("sfa_blocks_fork", FORK, dict(n=-1), -1),
    ("sfa_blocks_fork", FORK, dict(src=P0), -1), ("sfa_blocks_fork", FORK, dict(shares=P0), -1),
    ("sfa_blocks_fork", FORK, dict(bs=0), -1), ("sfa_blocks_fork", FORK, dict(lens=ODD), -1),
    ("sfa_blocks_free", FREE, dict(out=FAKE), -1), ("sfa_blocks_free", FREE, dict(rows=8193), -2),
    ("sfa_blocks_free", FREE, dict(rows=8192, mb=1 << 18), -2), ("sfa_blocks_free", FREE, dict(held=P0), -1),
    ("sfa_blocks_compact", COMPACT, dict(t2=FAKE), -1), ("sfa_blocks_compact", COMPACT, dict(s2=FAKE), -1),
    ("sfa_blocks_compact", COMPACT, dict(f2=FAKE), -1), ("sfa_blocks_compact", COMPACT, dict(nb=(1 << 20) + 1), -2),
    ("sfa_blocks_compact", COMPACT, dict(moves=-1), -1), ("sfa_blocks_compact", COMPACT, dict(copies=P0), -1),
    ("sfa_kv_copy_blocks", COPY, dict(n=-1), -1), ("sfa_kv_copy_blocks", COPY, dict(kv=P0), -1),
    ("sfa_kv_copy_blocks", COPY, dict(n=0), 0), ("sfa_kv_copy_blocks", COPY, dict(copies=ODD), -1),
    ("sfa_kv_copy_blocks_q8", COPY8, dict(group=5), -1), ("sfa_kv_copy_blocks_q8", COPY8, dict(scales=P0), -1),
    ("sfa_kv_copy_blocks_q8", COPY8, dict(layers=0), 0),
])
def test_host_argument_checks(lib, name, base, kw, code):
    assert _call(lib, name, base, **kw) == code


def test_decode_tree_wants_its_workspace(lib):
    need = lib.sfa_decode_tree_workspace_bytes(2, 4, 4)
    assert need % 256 == 0
    if need:
        assert _call(lib, "sfa_decode_tree", DECODE, wsb=need - 1) == -3
        assert _call(lib, "sfa_decode_tree", DECODE, ws=P0, wsb=need) == -3
        assert _call(lib, "sfa_decode_tree", DECODE, ws=ctypes.c_void_p((1 << 20) + 16), wsb=need) == -3


def test_blocks_free_wants_its_workspace(lib):
    assert lib.sfa_blocks_free_workspace_bytes(512, 64) == 0     # a cluster's registers hold the entries
    assert lib.sfa_blocks_free_workspace_bytes(513, 64) > 0
    assert lib.sfa_blocks_free_workspace_bytes(8193, 64) == 0 and lib.sfa_blocks_free_workspace_bytes(-1, 64) == 0
    need = lib.sfa_blocks_free_workspace_bytes(700, 1026)
    assert need == 152 * 4
    kw = dict(rows=700, mb=1026)
    assert _call(lib, "sfa_blocks_free", FREE, wsb=need - 1, **kw) == -3
    assert _call(lib, "sfa_blocks_free", FREE, ws=P0, wsb=need, **kw) == -3
    assert _call(lib, "sfa_blocks_free", FREE, ws=ODD, wsb=need, **kw) == -1


def test_binding_refuses_what_does_not_fit():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        sfa.tree_plan(i(4), i(3), i(2), 8)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.tree_accept(i(4), i(4), i(4), i(3), i(2), 8)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.blocks_free(i(2, 3), i(2), i(2), i(9), i(9), i(1), 16)
    kv = torch.zeros((2, 4, 576), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.kv_commit(kv, i(2, 3), i(2), i(2, 8), i(2))
    with pytest.raises(TypeError):
        sfa.kv_copy_blocks(kv.float(), i(1, 3))
    with pytest.raises(ValueError, match="CUDA"):
        sfa.decode_tree(torch.zeros((4, 2, 576), dtype=torch.bfloat16), kv, i(2, 3), i(2), i(3),
                        torch.zeros((4, 1), dtype=torch.int64), 0.1)
