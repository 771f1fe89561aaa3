"""GB300 (sm_103a) sparse MLA decode (SFA) with DCP-style split partials.

A thin Python binding over the C ABI of libsfa.so (include/sfa.h).  It only
checks and marshals arguments; every step of the computation runs in the
library's CUDA kernels.  PyTorch provides device memory and streams.

    out, lse = decode(q, kv, block_table, seq_lens, topk_idx, scale)
    out_part, lse_part = decode(..., n_splits=8, merge=False)
    out, lse = lse_merge(out_part, lse_part)

and, around it, one serving step over an 8-bit cache:

    table, seq_lens, start, positions, slots, taken = step_plan(cached, new, table, free, taken, 64, T)
    rope(q_pe, positions, inv_freq, out=q[..., 512:])
    kv_write_q8(kv8, scales, slots, rows, workspace=ws)
    out, lse = decode_q8(q, kv8, scales, table, seq_lens, topk_idx, scale)

a step that verifies a tree of drafted tokens, and the blocks that requests hold:

    table, _, start, _, slots, taken = step_plan(cached, nodes, table, free, taken, 64, T)
    mask, positions = tree_plan(parents, start, cached, max_nodes)
    kv_write(kv, slots, rows)
    out, lse = decode_tree(q, kv, table, cached, start, mask, scale)
    path, accepted, next_tokens, lens = tree_accept(tokens, targets, parents, start, cached, max_nodes)
    kv_commit(kv, table, cached, path, accepted)
    taken = blocks_free(table, cached + nodes, lens, shares, free, taken, 64)
    copies, taken = blocks_fork(table, lens, src, dst, shares, free, taken, 64)
    kv_copy_blocks(kv, copies)
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import _lib
from ._lib import SfaError

D_QK = 576
D_V = 512
MAX_HEADS = 128
MAX_SPLITS = 64
BLOCK_TABLE_PER_TOKEN = 1   # sfa_decode_ex flag: one block-table row per query token
OUT_BF16 = 2                # sfa_decode_q8 flag: out is bf16

__all__ = ["decode", "lse_merge", "decode_host", "decode_host_staging_bytes",
           "workspace_bytes", "decode_noalloc", "decode_launches", "last_device_status", "set_kernel_path",
           "set_wait_limit", "set_stall_injection", "kv_write", "uv_proj", "topk", "HostPlan",
           "decode_q8", "kv_write_q8", "kv_write_q8_workspace_bytes", "step_plan",
           "rope", "rope_inv_freq", "rope_mscale",
           "tree_plan", "decode_tree", "decode_tree_workspace_bytes", "tree_accept", "kv_commit",
           "blocks_fork", "blocks_free", "blocks_free_workspace_bytes", "blocks_compact",
           "kv_copy_blocks", "kv_copy_blocks_q8",
           "SfaError", "D_QK", "D_V", "BLOCK_TABLE_PER_TOKEN"]


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


_HERE = contextlib.nullcontext()


def _on(dev, stream):
    """Context of a call: `dev` current, and what the call allocates belongs to its stream."""
    if stream is None:
        return _HERE if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"stream must be on {dev}, got {stream.device}")
    return torch.cuda.stream(stream)


def _raw_stream(dev):
    """The stream of the call (inside `_on`)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


_BF16, _F32, _F64, _I32, _E4M3 = (torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.float8_e4m3fn)
_I64 = torch.int64


def _check(t, name, dtype, dev, ndim, isinstance=isinstance, Tensor=torch.Tensor):
    """_need on a CUDA device, quick where nothing is wrong."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.get_device() == dev.index and t.dim() == ndim
            and t.is_contiguous()):
        _need(t, name, dtype, dev, ndim)


def _need(t, name, dtype, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _check_decode_inputs(q, kv, block_table, seq_lens, topk_idx, Q, block_table_per_token=False):
    """The argument checks of every decode entry point: dtypes, ranks, the 576-column
    rows and T == B*Q for q, the index lists and the block table (shapes first, so a bad
    Q is reported even off the GPU), then one CUDA device for everything.  Returns
    (T, h, B, top_k)."""
    for t, name, dt, nd in ((q, "q", torch.bfloat16, 3), (kv, "kv", torch.bfloat16, 3),
                            (block_table, "block_table", torch.int32, 2), (seq_lens, "seq_lens", torch.int32, 1),
                            (topk_idx, "topk_idx", torch.int32, 2)):
        _need(t, name, dt, None, nd)
    T, h, d = q.shape
    if d != D_QK or kv.shape[2] != D_QK:
        raise ValueError("q and kv rows must have 576 columns")
    if int(Q) != Q or Q < 1:
        raise ValueError("Q must be an integer >= 1")
    Q = int(Q)
    B = seq_lens.shape[0]
    bt_rows = T if block_table_per_token else B
    if T != B * Q or topk_idx.shape[0] != T or block_table.shape[0] != bt_rows:
        raise ValueError("inconsistent B / Q / T")
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("decode runs on a CUDA device only")
    for t, name in ((kv, "kv"), (block_table, "block_table"), (seq_lens, "seq_lens"), (topk_idx, "topk_idx")):
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
    return T, h, B, topk_idx.shape[1]


def workspace_bytes(B: int, Q: int, h: int, top_k: int, n_splits: int) -> int:
    return int(_lib.load().sfa_decode_workspace_bytes(B, Q, h, top_k, n_splits))


def decode(q, kv, block_table, seq_lens, topk_idx, scale: float, n_splits: int = 1, Q: int = 1,
           merge: bool = True, out=None, lse=None, out_part=None, lse_part=None, workspace=None,
           stream=None, interleave: int = 0, block_table_per_token: bool = False):
    """Sparse MLA decode (C ABI ``sfa_decode_ex``; ``sfa_decode`` when both layout options
    are off).

    q [B*Q, h, 576] bf16, kv [num_blocks, block_size, 576] bf16, block_table [B, max_blocks]
    int32 ([B*Q, max_blocks] with block_table_per_token), seq_lens [B] int32, topk_idx
    [B*Q, top_k] int32 (-1 = padding), all on one CUDA device.  interleave = g > 0 deals the
    cache positions to the n_splits shards g at a time (shard r holds (p // g) % n == r);
    0 keeps contiguous shards.  Returns (out [B*Q, h, 512] fp32, lse [B*Q, h] fp32); with
    n_splits > 1 and merge=False returns the shard partials (out_part [n, B*Q, h, 512],
    lse_part [n, B*Q, h]).
    """
    T, h, B, top_k = _check_decode_inputs(q, kv, block_table, seq_lens, topk_idx, Q, block_table_per_token)
    lib = _lib.load()
    dev = q.device
    if interleave < 0:
        raise ValueError("interleave must be >= 0")
    num_blocks, block_size = kv.shape[0], kv.shape[1]
    max_blocks = block_table.shape[1]
    if n_splits == 1 or merge:
        if out is None:
            out = torch.empty((T, h, D_V), dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty((T, h), dtype=torch.float32, device=dev)
        _need(out, "out", torch.float32, dev)
        _need(lse, "lse", torch.float32, dev)
        if tuple(out.shape) != (T, h, D_V) or tuple(lse.shape) != (T, h):
            raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
    if n_splits > 1:
        if out_part is None:
            out_part = torch.empty((n_splits, T, h, D_V), dtype=torch.float32, device=dev)
        if lse_part is None:
            lse_part = torch.empty((n_splits, T, h), dtype=torch.float32, device=dev)
        _need(out_part, "out_part", torch.float32, dev)
        _need(lse_part, "lse_part", torch.float32, dev)
    ws_need = int(lib.sfa_decode_workspace_bytes(B, Q, h, top_k, n_splits))
    if ws_need and workspace is None:
        workspace = torch.empty(ws_need, dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    flags = BLOCK_TABLE_PER_TOKEN if block_table_per_token else 0
    code = lib.sfa_decode_ex(_ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens), _ptr(topk_idx),
                             B, Q, h, top_k, num_blocks, block_size, max_blocks, float(scale),
                             n_splits, int(interleave), flags,
                             _ptr(out if (n_splits == 1 or merge) else None),
                             _ptr(lse if (n_splits == 1 or merge) else None),
                             _ptr(out_part if n_splits > 1 else None),
                             _ptr(lse_part if n_splits > 1 else None), _ptr(workspace), ws_bytes,
                             _stream_ptr(stream, dev))
    _lib.check("sfa_decode_ex", code)
    if n_splits > 1 and not merge:
        return out_part, lse_part
    return out, lse


def decode_noalloc(q, kv, block_table, seq_lens, topk_idx, scale: float, n_splits: int = 1,
                   Q: int = 1, out=None, lse=None, stream=None):
    """Decode + shard merge without caller-provided scratch (C ABI ``sfa_decode_noalloc``).

    For callers that cannot allocate device memory for shard partials: they live in a
    fixed device array owned by the library (include/sfa.h, SFA_NOALLOC_SCRATCH_BYTES).
    Pass preallocated `out` [B*Q, h, 512] and `lse` [B*Q, h] fp32 to allocate nothing here.
    Calls that overlap on the GPU share that array and race.
    """
    T, h, B, _ = _check_decode_inputs(q, kv, block_table, seq_lens, topk_idx, Q)
    lib = _lib.load()
    dev = q.device
    if out is None:
        out = torch.empty((T, h, D_V), dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty((T, h), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev)
    _need(lse, "lse", torch.float32, dev)
    if tuple(out.shape) != (T, h, D_V) or tuple(lse.shape) != (T, h):
        raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
    code = lib.sfa_decode_noalloc(_ptr(q), _ptr(kv), _ptr(block_table), _ptr(seq_lens),
                                  _ptr(topk_idx), B, Q, h, topk_idx.shape[1], kv.shape[0],
                                  kv.shape[1], block_table.shape[1], float(scale), n_splits,
                                  _ptr(out), _ptr(lse), _stream_ptr(stream, dev))
    _lib.check("sfa_decode_noalloc", code)
    return out, lse


def lse_merge(out_part, lse_part, out=None, lse=None, stream=None):
    """Online-softmax merge over the leading axis (C ABI ``sfa_lse_merge``).

    out_part [n, *rows, dv] fp32, lse_part [n, *rows] fp32 -> (out [*rows, dv], lse [*rows]).
    """
    lib = _lib.load()
    dev = out_part.device
    _need(out_part, "out_part", torch.float32, dev)
    _need(lse_part, "lse_part", torch.float32, dev)
    n = out_part.shape[0]
    dv = out_part.shape[-1]
    rows = lse_part[0].numel() if n > 0 else 0
    if tuple(lse_part.shape) != tuple(out_part.shape[:-1]):
        raise ValueError("lse_part must be out_part's shape without the last axis")
    if out is None:
        out = torch.empty(out_part.shape[1:], dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty(lse_part.shape[1:], dtype=torch.float32, device=dev)
    code = lib.sfa_lse_merge(_ptr(out_part), _ptr(lse_part), n, rows, dv, _ptr(out), _ptr(lse),
                             _stream_ptr(stream, dev))
    _lib.check("sfa_lse_merge", code)
    return out, lse


def decode_host_staging_bytes(B, Q, h, top_k, max_blocks, n_splits) -> int:
    return int(_lib.load().sfa_decode_host_staging_bytes(B, Q, h, top_k, max_blocks, n_splits))


def decode_host(q_host, kv, block_table_host, seq_lens_host, topk_idx_host, scale, n_splits,
                Q, out_host, lse_host, staging, stream=None):
    """One decode step with host-resident per-step inputs/outputs (C ABI ``sfa_decode_host``).

    q/block_table/seq_lens/topk_idx and out/lse are (preferably pinned) CPU tensors, kv and
    staging are on the device.  Enqueues copies + kernels on `stream`; synchronise before
    reading out_host / lse_host.
    """
    lib = _lib.load()
    dev = kv.device
    _need(kv, "kv", torch.bfloat16, dev, 3)
    for t, name, dt in ((q_host, "q_host", torch.bfloat16), (block_table_host, "block_table_host", torch.int32),
                        (seq_lens_host, "seq_lens_host", torch.int32), (topk_idx_host, "topk_idx_host", torch.int32),
                        (out_host, "out_host", torch.float32), (lse_host, "lse_host", torch.float32)):
        _need(t, name, dt, torch.device("cpu"))
    T, h, _ = q_host.shape
    B = seq_lens_host.shape[0]
    top_k = topk_idx_host.shape[1]
    code = lib.sfa_decode_host(_ptr(q_host), _ptr(kv), _ptr(block_table_host), _ptr(seq_lens_host),
                               _ptr(topk_idx_host), B, Q, h, top_k, kv.shape[0], kv.shape[1],
                               block_table_host.shape[1], float(scale), n_splits, _ptr(out_host),
                               _ptr(lse_host), _ptr(staging),
                               staging.numel() * staging.element_size(), _stream_ptr(stream, dev))
    _lib.check("sfa_decode_host", code)
    return out_host, lse_host


class HostPlan:
    """One decode_host step captured once as a CUDA graph (C ABI ``sfa_host_plan_*``), for a
    serving loop that reuses its buffers: ``launch()`` enqueues the whole step (input copies,
    kernels, result copies) with one graph launch.

    Arguments as decode_host; the host tensors must be pinned.  Every launch reads the host
    inputs as they are at that moment and writes out_host / lse_host; refill the inputs in
    place between launches and synchronise before reading the results.  The tensors are kept
    alive by the plan.  ``close()`` (or garbage collection) releases it.
    """

    def __init__(self, q_host, kv, block_table_host, seq_lens_host, topk_idx_host, scale, n_splits, Q,
                 out_host, lse_host, staging):
        lib = _lib.load()
        dev = kv.device
        _need(kv, "kv", torch.bfloat16, dev, 3)
        for t, name, dt in ((q_host, "q_host", torch.bfloat16), (block_table_host, "block_table_host", torch.int32),
                            (seq_lens_host, "seq_lens_host", torch.int32),
                            (topk_idx_host, "topk_idx_host", torch.int32),
                            (out_host, "out_host", torch.float32), (lse_host, "lse_host", torch.float32)):
            _need(t, name, dt, torch.device("cpu"))
            if not t.is_pinned():
                raise ValueError(f"{name} must be pinned host memory")
        self._keep = (q_host, kv, block_table_host, seq_lens_host, topk_idx_host, out_host, lse_host, staging)
        self._dev = dev
        T, h, _ = q_host.shape
        B = seq_lens_host.shape[0]
        top_k = topk_idx_host.shape[1]
        plan = ctypes.c_void_p(0)
        code = lib.sfa_host_plan_create(_ptr(q_host), _ptr(kv), _ptr(block_table_host), _ptr(seq_lens_host),
                                        _ptr(topk_idx_host), B, Q, h, top_k, kv.shape[0], kv.shape[1],
                                        block_table_host.shape[1], float(scale), n_splits, _ptr(out_host),
                                        _ptr(lse_host), _ptr(staging), staging.numel() * staging.element_size(),
                                        ctypes.byref(plan))
        _lib.check("sfa_host_plan_create", code)
        self._plan = plan

    def launch(self, stream=None):
        if not self._plan:
            raise ValueError("the plan is closed")
        _lib.check("sfa_host_plan_launch", _lib.load().sfa_host_plan_launch(self._plan, _stream_ptr(stream, self._dev)))

    def close(self):
        if getattr(self, "_plan", None):
            _lib.load().sfa_host_plan_destroy(self._plan)
            self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def uv_proj(out, w_uv, y=None, stream=None):
    """W_UV up-projection (C ABI ``sfa_uv_proj``): y[t, h, v] = sum_c out[t, h, c] * w_uv[h, c, v].

    out [T, h, 512] fp32 (decode's output), w_uv [h, 512, 128] bf16, y [T, h, 128] bf16
    (allocated when None), all on one CUDA device.  Returns y.
    """
    lib = _lib.load()
    dev = out.device
    if dev.type != "cuda":
        raise ValueError("uv_proj runs on a CUDA device only")
    _need(out, "out", torch.float32, dev, 3)
    _need(w_uv, "w_uv", torch.bfloat16, dev, 3)
    T, h, c = out.shape
    if c != D_V or tuple(w_uv.shape) != (h, D_V, 128):
        raise ValueError("out must be [T, h, 512] and w_uv [h, 512, 128]")
    if y is None:
        y = torch.empty((T, h, 128), dtype=torch.bfloat16, device=dev)
    _need(y, "y", torch.bfloat16, dev, 3)
    code = lib.sfa_uv_proj(_ptr(out), _ptr(w_uv), _ptr(y), T, h, _stream_ptr(stream, dev))
    _lib.check("sfa_uv_proj", code)
    return y


def kv_write(kv, slot_mapping, rows, stream=None):
    """Latent-cache write (C ABI ``sfa_kv_write``): kv viewed as [num_blocks*block_size, 576]
    gets row slot_mapping[t] = rows[t] for every t with slot_mapping[t] >= 0, in place.

    kv [num_blocks, block_size, 576] bf16, slot_mapping [T] int32, rows [T, 576] bf16, all on
    one CUDA device.  A slot named twice ends up holding parts of both rows.  Returns kv.
    """
    lib = _lib.load()
    dev = kv.device
    if dev.type != "cuda":
        raise ValueError("kv_write runs on a CUDA device only")
    _need(kv, "kv", torch.bfloat16, dev, 3)
    _need(slot_mapping, "slot_mapping", torch.int32, dev, 1)
    _need(rows, "rows", torch.bfloat16, dev, 2)
    if kv.shape[2] != D_QK or rows.shape[1] != D_QK or rows.shape[0] != slot_mapping.shape[0]:
        raise ValueError("rows must be [T, 576] with one slot per row")
    num_slots = kv.shape[0] * kv.shape[1]
    code = lib.sfa_kv_write(_ptr(kv), num_slots, _ptr(slot_mapping), _ptr(rows), rows.shape[0],
                            _stream_ptr(stream, dev))
    _lib.check("sfa_kv_write", code)
    return kv


def topk(scores, k: int, seq_lens=None, Q: int = 1, S: Optional[int] = None, out=None, stream=None):
    """Indexer top-k selection (C ABI ``sfa_topk``): for each query token t = b*Q + i, the
    positions of the k largest scores among [0, L), L = min(S, seq_lens[b] - (Q-1-i)) (S
    without seq_lens), equal scores lower position first, in ascending position, -1 padded.

    scores [B*Q, row_stride] fp32 (row_stride >= S, a multiple of 4), seq_lens [B] int32 or
    None, out [B*Q, k] int32 (allocated when None), all on one CUDA device.  Returns out,
    the topk_idx layout decode reads.
    """
    lib = _lib.load()
    dev = scores.device
    if dev.type != "cuda":
        raise ValueError("topk runs on a CUDA device only")
    _need(scores, "scores", torch.float32, dev, 2)
    T, stride = scores.shape
    S = stride if S is None else int(S)
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, dev, 1)
        B = seq_lens.shape[0]
        if B * Q != T:
            raise ValueError("scores must have B*Q rows")
    else:
        if T % Q:
            raise ValueError("the number of score rows must be a multiple of Q")
        B = T // Q
    if out is None:
        out = torch.empty((T, int(k)), dtype=torch.int32, device=dev)
    _need(out, "out", torch.int32, dev, 2)
    if tuple(out.shape) != (T, int(k)):
        raise ValueError("out must be [B*Q, k]")
    code = lib.sfa_topk(_ptr(scores), stride, _ptr(seq_lens), B, int(Q), S, int(k), _ptr(out),
                        _stream_ptr(stream, dev))
    _lib.check("sfa_topk", code)
    return out


def _need_cache_q8(kv8, scales):
    """The checks of an 8-bit cache [num_blocks, block_size, 576] and its scales [num_blocks,
    block_size / group]; returns (num_blocks, block_size, group)."""
    if not (isinstance(kv8, torch.Tensor) and kv8.dtype is _E4M3 and kv8.dim() == 3 and kv8.is_contiguous()
            and isinstance(scales, torch.Tensor) and scales.dtype is _F32 and scales.dim() == 2
            and scales.is_contiguous()):
        _need(kv8, "kv8", _E4M3, None, 3)
        _need(scales, "scales", _F32, None, 2)
    nb, bs, d = kv8.shape
    if d != D_QK:
        raise ValueError("kv8 rows must have 576 columns")
    rows, groups = scales.shape
    if rows != nb or groups < 1 or bs % groups:
        raise ValueError("scales must be [num_blocks, block_size / group] with group dividing block_size")
    if not kv8.is_cuda:
        raise ValueError("the 8-bit cache must be on a CUDA device")
    if scales.get_device() != kv8.get_device():
        raise ValueError(f"scales must be on {kv8.device}, got {scales.device}")
    return nb, bs, bs // groups


def decode_q8(q, kv8, scales, block_table, seq_lens, topk_idx, scale: float, n_splits: int = 1, Q: int = 1,
              merge: bool = True, out=None, lse=None, out_part=None, lse_part=None, stream=None,
              interleave: int = 0, block_table_per_token: bool = False, out_dtype=torch.float32):
    """Sparse MLA decode over an 8-bit latent cache (C ABI ``sfa_decode_q8``).

    kv8 [num_blocks, block_size, 576] float8_e4m3fn and scales [num_blocks, block_size / group]
    fp32: an element's value is kv8 * the scale of its group of slots (as kv_write_q8 writes
    them).  out is [B*Q, h, 512] in `out_dtype` (torch.float32 or torch.bfloat16, or the dtype
    of the `out` given).  Everything else as in ``decode``.
    """
    num_blocks, block_size, group = _need_cache_q8(kv8, scales)
    dev = kv8.device
    _check(q, "q", _BF16, dev, 3)
    _check(block_table, "block_table", _I32, dev, 2)
    _check(seq_lens, "seq_lens", _I32, dev, 1)
    _check(topk_idx, "topk_idx", _I32, dev, 2)
    T, h, d = q.shape
    if d != D_QK:
        raise ValueError("q rows must have 576 columns")
    if int(Q) != Q or Q < 1:
        raise ValueError("Q must be an integer >= 1")
    Q, n_splits = int(Q), int(n_splits)
    B = seq_lens.shape[0]
    lists, top_k = topk_idx.shape
    tables, max_blocks = block_table.shape
    if T != B * Q or lists != T or tables != (T if block_table_per_token else B):
        raise ValueError("inconsistent B / Q / T")
    if interleave < 0:
        raise ValueError("interleave must be >= 0")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype is not _F32 and out_dtype is not _BF16:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    lib = _lib.load()
    final = n_splits == 1 or merge
    out_p = lse_p = op_p = lp_p = 0
    with _on(dev, stream):
        if final:
            if out is None:
                out = torch.empty((T, h, D_V), dtype=out_dtype, device=dev)
            elif out.shape != (T, h, D_V):
                raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
            else:
                _check(out, "out", out_dtype, dev, 3)
            if lse is None:
                lse = torch.empty((T, h), dtype=_F32, device=dev)
            elif lse.shape != (T, h):
                raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
            else:
                _check(lse, "lse", _F32, dev, 2)
            out_p, lse_p = out.data_ptr(), lse.data_ptr()
        if n_splits > 1 and final and out_part is None and lse_part is None:
            # partials that nobody sees: one buffer for both
            n = n_splits * T * h
            parts = torch.empty(n * (D_V + 1), dtype=_F32, device=dev)
            op_p = parts.data_ptr()
            lp_p = op_p + 4 * n * D_V
        elif n_splits > 1:
            if out_part is None:
                out_part = torch.empty((n_splits, T, h, D_V), dtype=_F32, device=dev)
            if lse_part is None:
                lse_part = torch.empty((n_splits, T, h), dtype=_F32, device=dev)
            if out_part.shape != (n_splits, T, h, D_V) or lse_part.shape != (n_splits, T, h):
                raise ValueError(f"out_part must be [{n_splits}, {T}, {h}, {D_V}] and lse_part [{n_splits}, {T}, {h}]")
            _check(out_part, "out_part", _F32, dev, 4)
            _check(lse_part, "lse_part", _F32, dev, 3)
            op_p, lp_p = out_part.data_ptr(), lse_part.data_ptr()
        flags = (BLOCK_TABLE_PER_TOKEN if block_table_per_token else 0) | \
                (OUT_BF16 if final and out_dtype is _BF16 else 0)
        code = lib.sfa_decode_q8(q.data_ptr(), kv8.data_ptr(), scales.data_ptr(), group, block_table.data_ptr(),
                                 seq_lens.data_ptr(), topk_idx.data_ptr(), B, Q, h, top_k, num_blocks, block_size,
                                 max_blocks, float(scale), n_splits, int(interleave), flags, out_p, lse_p, op_p, lp_p,
                                 _raw_stream(dev))
    if code:
        _lib.check("sfa_decode_q8", code)
    return (out, lse) if final else (out_part, lse_part)


def kv_write_q8_workspace_bytes(num_slots: int, group: int) -> int:
    return int(_lib.load().sfa_kv_write_q8_workspace_bytes(int(num_slots), int(group)))


def kv_write_q8(kv8, scales, slot_mapping, rows, workspace=None, stream=None):
    """Quantising write into the 8-bit latent cache (C ABI ``sfa_kv_write_q8``): row t of rows
    [T, 576] bf16 goes to slot slot_mapping[t] (< 0 = padding) of kv8 [num_blocks, block_size,
    576] float8_e4m3fn under the power-of-two scale of its group, scales [num_blocks,
    block_size / group]; a group whose scale rises has its other rows stored again under it,
    and one whose first slot is written starts anew.  In place; returns (kv8, scales).

    workspace: kv_write_q8_workspace_bytes(num_blocks * block_size, group) bytes that belong to
    this cache, zeroed once before the first write (not needed for groups of one slot).
    """
    num_blocks, block_size, group = _need_cache_q8(kv8, scales)
    dev = kv8.device
    _check(slot_mapping, "slot_mapping", _I32, dev, 1)
    _check(rows, "rows", _BF16, dev, 2)
    T, d = rows.shape
    if d != D_QK or T != slot_mapping.shape[0]:
        raise ValueError("rows must be [T, 576] with one slot per row")
    ws_p = ws_bytes = 0
    if workspace is not None:
        if workspace.get_device() != dev.index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {dev}")
        ws_p, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    with _on(dev, stream):
        code = _lib.load().sfa_kv_write_q8(kv8.data_ptr(), scales.data_ptr(), num_blocks * block_size, group,
                                           slot_mapping.data_ptr(), rows.data_ptr(), T, ws_p, ws_bytes,
                                           _raw_stream(dev))
    if code:
        _lib.check("sfa_kv_write_q8", code)
    return kv8, scales


def step_plan(cached_lens, new_lens, block_table, free_blocks, taken, block_size: int, num_tokens: int, stream=None):
    """Block tables and slot maps of one step from request lengths (C ABI ``sfa_step_plan``).

    cached_lens, new_lens [B] int32; block_table [B, max_blocks] int32 (in place: the blocks
    that the new tokens need are taken from free_blocks [F] int32, from entry taken[0] on, in
    request order); num_tokens is the step's room for new tokens.  Returns (block_table,
    seq_lens [B], token_start [B + 1], positions [num_tokens], slot_mapping [num_tokens],
    taken [1]), all int32; positions and slots behind the last token are -1, which rope and the
    cache writes skip.
    """
    dev = block_table.device
    if dev.type != "cuda":
        raise ValueError("step_plan runs on a CUDA device only")
    _check(block_table, "block_table", _I32, dev, 2)
    _check(cached_lens, "cached_lens", _I32, dev, 1)
    _check(new_lens, "new_lens", _I32, dev, 1)
    _check(free_blocks, "free_blocks", _I32, dev, 1)
    _check(taken, "taken", _I32, dev, 1)
    B, max_blocks = block_table.shape
    if cached_lens.shape[0] != B or new_lens.shape[0] != B or taken.shape[0] != 1:
        raise ValueError("cached_lens and new_lens must be [B], block_table [B, max_blocks] and taken [1]")
    N = int(num_tokens)
    if N < 0:
        raise ValueError("num_tokens must be >= 0")
    with _on(dev, stream):
        # (five allocations take less of the host's time than five views of one)
        seq_lens = torch.empty(B, dtype=_I32, device=dev)
        start = torch.empty(B + 1, dtype=_I32, device=dev)
        positions = torch.empty(N, dtype=_I32, device=dev)
        slots = torch.empty(N, dtype=_I32, device=dev)
        taken_out = torch.empty(1, dtype=_I32, device=dev)
        code = _lib.load().sfa_step_plan(cached_lens.data_ptr(), new_lens.data_ptr(), B, int(block_size),
                                         block_table.data_ptr(), max_blocks, free_blocks.data_ptr(),
                                         free_blocks.shape[0], taken.data_ptr(), N, seq_lens.data_ptr(),
                                         start.data_ptr(), positions.data_ptr(), slots.data_ptr(),
                                         taken_out.data_ptr(), _raw_stream(dev))
    if code:
        _lib.check("sfa_step_plan", code)
    return block_table, seq_lens, start, positions, slots, taken_out


def rope_inv_freq(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                  original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """The frequencies ``rope`` takes, [rot_dim / 2] float64: base ** (-2i / rot_dim), scaled
    for contexts `factor` times `original_len`:

    "linear"  all divided by factor (position interpolation);
    "ntk"     the base grows by factor ** (rot_dim / (rot_dim - 2));
    "yarn"    a frequency that turns more than beta_fast times in original_len positions stays,
              one that turns less than beta_slow times is divided by factor, and those between
              are mixed linearly in the number of turns (YaRN, arXiv:2309.00071, section 3.2;
              its attention temperature is ``rope_mscale``).  Code that mixes linearly in the
              pair's index i instead gives other frequencies between the two bounds (of 64
              columns at factor 40 up to 77 % lower ones): a checkpoint trained with it needs
              those, which ``rope`` takes like any others.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and >= 2")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs rot_dim >= 4")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = torch.tensor([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must exceed beta_slow")
        turns = original_len * f / (2.0 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    return f.to(device)


def rope_mscale(factor: float) -> float:
    """The magnitude that YaRN gives rotated columns for a context `factor` times the trained."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def rope(x, positions, inv_freq, interleaved: bool = True, mscale: float = 1.0, inverse: bool = False, out=None,
         stream=None):
    """Rotary positions of the first 2 * len(inv_freq) columns of each head (C ABI ``sfa_rope``).

    x [T, n, width] or [T, width] bf16, fp16 or fp32 with any row strides (a view of the rope
    columns of wider heads); positions [T] int32 (< 0 = padding: those rows of out are left as
    they were, and are x's in a new one); inv_freq [rot_dim / 2] float64 (``rope_inv_freq``).
    interleaved pairs columns (2i, 2i + 1), else (i, i + rot_dim / 2).  inverse turns back by the
    same angles: the transpose, so that rope(grad_out, ..., inverse=True) is the gradient of x.
    out: x itself (in place), another tensor of x's shape and dtype, or None for a new one.
    Returns out.
    """
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("rope runs on a CUDA device only")
    dtype = _ROPE_DTYPES.get(x.dtype)
    if dtype is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    shape, strides = x.shape, x.stride()
    if len(shape) == 3:
        (T, n, width), (xt, xn, xd) = shape, strides
    elif len(shape) == 2:
        (T, width), (xt, xd), n, xn = shape, strides, 1, 0
    else:
        xd = 0
    if xd != 1 or width < 1:
        raise ValueError("x must be [T, n, width] or [T, width] with contiguous columns")
    _check(positions, "positions", _I32, dev, 1)
    _check(inv_freq, "inv_freq", _F64, dev, 1)
    rot = 2 * inv_freq.shape[0]
    if positions.shape[0] != T:
        raise ValueError("positions must be [T]")
    if rot < 2 or rot > width:
        raise ValueError("inv_freq must be [rot_dim / 2] with 2 <= rot_dim <= width")
    flags = (1 if interleaved else 0) | (2 if inverse else 0)
    with _on(dev, stream):
        if out is None:
            # a padding row has no result: a new tensor holds x's there
            out = torch.empty(shape, dtype=x.dtype, device=dev)
            flags |= 8
        elif out.dtype is not x.dtype or out.get_device() != dev.index or out.shape != shape or out.stride(-1) != 1:
            raise ValueError("out must have x's shape, dtype and device, and contiguous columns")
        if n == 0:
            return out
        os = out.stride()
        code = _lib.load().sfa_rope(x.data_ptr(), xt, xn, out.data_ptr(), os[0], os[1] if len(shape) == 3 else 0,
                                    dtype, T, n, width, rot, positions.data_ptr(), inv_freq.data_ptr(), float(mscale),
                                    flags, _raw_stream(dev))
    if code:
        _lib.check("sfa_rope", code)
    return out


def _need_tree(token_start, cached_lens, max_nodes, dev):
    """The checks of what every call of a drafted tree takes; returns (B, max_nodes)."""
    if dev.type != "cuda":
        raise ValueError("the calls of drafted trees run on a CUDA device only")
    _check(token_start, "token_start", _I32, dev, 1)
    _check(cached_lens, "cached_lens", _I32, dev, 1)
    B = cached_lens.shape[0]
    if token_start.shape[0] != B + 1:
        raise ValueError("token_start must be [B + 1] and cached_lens [B]")
    max_nodes = int(max_nodes)
    if max_nodes < 1:
        raise ValueError("max_nodes must be >= 1")
    return B, max_nodes


def tree_plan(parents, token_start, cached_lens, max_nodes: int, stream=None):
    """Masks and positions of drafted trees (C ABI ``sfa_tree_plan``).

    parents [T] int32: a node's parent by its number within the request (smaller than its own), -1
    for a child of the last cached token; token_start [B + 1], cached_lens [B] int32 (request b's
    nodes are the tokens token_start[b] .. token_start[b + 1] - 1, at most max_nodes).  Returns
    (mask [T, ceil(max_nodes / 64)] int64, with the bits of each node and its ancestors; positions
    [T] int32 = cached_lens + depth, -1 for padding tokens).
    """
    dev = parents.device
    B, max_nodes = _need_tree(token_start, cached_lens, max_nodes, dev)
    _check(parents, "parents", _I32, dev, 1)
    T = parents.shape[0]
    with _on(dev, stream):
        mask = torch.empty((T, (max_nodes + 63) // 64), dtype=_I64, device=dev)
        positions = torch.empty(T, dtype=_I32, device=dev)
        code = _lib.load().sfa_tree_plan(parents.data_ptr(), token_start.data_ptr(), cached_lens.data_ptr(), B, T,
                                         max_nodes, mask.data_ptr(), positions.data_ptr(), _raw_stream(dev))
    if code:
        _lib.check("sfa_tree_plan", code)
    return mask, positions


def decode_tree_workspace_bytes(B: int, num_tokens: int, h: int) -> int:
    return int(_lib.load().sfa_decode_tree_workspace_bytes(int(B), int(num_tokens), int(h)))


def decode_tree(q, kv, block_table, cached_lens, token_start, mask, scale: float, out=None, lse=None, workspace=None,
                stream=None, out_dtype=torch.float32):
    """Attention of drafted nodes over every cached position of their sequence and the nodes that
    their mask names (C ABI ``sfa_decode_tree``).

    q [T, h, 576] bf16, kv [num_blocks, block_size, 576] bf16, block_table [B, max_blocks],
    cached_lens [B], token_start [B + 1] int32, mask [T, words] int64 (``tree_plan``); node j of
    request b is the token token_start[b] + j and its row lies at position cached_lens[b] + j.
    Returns (out [T, h, 512] in out_dtype, torch.float32 or torch.bfloat16, or the dtype of the `out`
    given; lse [T, h] fp32); the rows of padding tokens are left as they were.
    workspace: decode_tree_workspace_bytes(B, T, h) bytes, 80 MB from 128 rows (T * h) on (allocated when None).
    """
    dev = q.device
    if not isinstance(mask, torch.Tensor) or mask.dim() != 2:
        raise ValueError("mask must be a [T, words] tensor")
    B, max_nodes = _need_tree(token_start, cached_lens, 64 * mask.shape[1], dev)
    _check(q, "q", _BF16, dev, 3)
    _check(kv, "kv", _BF16, dev, 3)
    _check(block_table, "block_table", _I32, dev, 2)
    _check(mask, "mask", _I64, dev, 2)
    T, h, d = q.shape
    if d != D_QK or kv.shape[2] != D_QK:
        raise ValueError("q and kv rows must have 576 columns")
    if mask.shape[0] != T or block_table.shape[0] != B:
        raise ValueError("mask must be [T, words] and block_table [B, max_blocks]")
    if out is not None:
        out_dtype = out.dtype
    if out_dtype is not _F32 and out_dtype is not _BF16:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    lib = _lib.load()
    with _on(dev, stream):
        if out is None:
            out = torch.empty((T, h, D_V), dtype=out_dtype, device=dev)
        elif out.shape != (T, h, D_V):
            raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
        else:
            _check(out, "out", out_dtype, dev, 3)
        if lse is None:
            lse = torch.empty((T, h), dtype=_F32, device=dev)
        elif lse.shape != (T, h):
            raise ValueError(f"out must be [{T}, {h}, {D_V}] and lse [{T}, {h}]")
        else:
            _check(lse, "lse", _F32, dev, 2)
        need = lib.sfa_decode_tree_workspace_bytes(B, T, h)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif workspace is not None and (workspace.get_device() != dev.index or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous and on {dev}")
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        code = lib.sfa_decode_tree(q.data_ptr(), kv.data_ptr(), block_table.data_ptr(), cached_lens.data_ptr(),
                                   token_start.data_ptr(), mask.data_ptr(), B, T, h, max_nodes, kv.shape[0],
                                   kv.shape[1], block_table.shape[1], float(scale),
                                   OUT_BF16 if out_dtype is _BF16 else 0, out.data_ptr(), lse.data_ptr(),
                                   workspace.data_ptr() if ws_bytes else 0, ws_bytes, _raw_stream(dev))
    if code:
        _lib.check("sfa_decode_tree", code)
    return out, lse


def tree_accept(tokens, targets, parents, token_start, cached_lens, max_nodes: int, stream=None):
    """The accepted path of each drafted tree (C ABI ``sfa_tree_accept``): from node 0 on, the child
    with the lowest number whose token is its parent's target.

    tokens, targets, parents [T] int32 (targets: the model's token behind each node).  Returns (path
    [B, max_nodes]: the accepted nodes' numbers, then -1; accepted [B]; next_tokens [B]: the target
    behind the last accepted node; seq_lens [B] = cached_lens + accepted), all int32.
    """
    dev = tokens.device
    B, max_nodes = _need_tree(token_start, cached_lens, max_nodes, dev)
    _check(tokens, "tokens", _I32, dev, 1)
    _check(targets, "targets", _I32, dev, 1)
    _check(parents, "parents", _I32, dev, 1)
    T = tokens.shape[0]
    if targets.shape[0] != T or parents.shape[0] != T:
        raise ValueError("tokens, targets and parents must be [T]")
    with _on(dev, stream):
        path = torch.empty((B, max_nodes), dtype=_I32, device=dev)
        accepted = torch.empty(B, dtype=_I32, device=dev)
        next_tokens = torch.empty(B, dtype=_I32, device=dev)
        seq_lens = torch.empty(B, dtype=_I32, device=dev)
        code = _lib.load().sfa_tree_accept(tokens.data_ptr(), targets.data_ptr(), parents.data_ptr(),
                                           token_start.data_ptr(), cached_lens.data_ptr(), B, T, max_nodes,
                                           path.data_ptr(), accepted.data_ptr(), next_tokens.data_ptr(),
                                           seq_lens.data_ptr(), _raw_stream(dev))
    if code:
        _lib.check("sfa_tree_accept", code)
    return path, accepted, next_tokens, seq_lens


def _need_layers(kv, name, dtype):
    """A cache [num_blocks, block_size, 576] or the caches of layers, [layers, ...]; returns (layers,
    num_blocks, block_size)."""
    if not isinstance(kv, torch.Tensor) or kv.dim() not in (3, 4):
        raise ValueError(f"{name} must be a [num_blocks, block_size, 576] or [layers, num_blocks, block_size, 576] tensor")
    _need(kv, name, dtype)
    if not kv.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if kv.shape[-1] != D_QK:
        raise ValueError(f"{name} rows must have 576 columns")
    return (kv.shape[0] if kv.dim() == 4 else 1), kv.shape[-3], kv.shape[-2]


def kv_commit(kv, block_table, cached_lens, path, accepted, stream=None):
    """The accepted nodes' rows move to consecutive positions (C ABI ``sfa_kv_commit``): the row at
    position cached_lens[b] + path[b, k] goes to cached_lens[b] + k, for k < accepted[b].

    kv [num_blocks, block_size, 576] bf16, or the caches of several layers with one block table,
    [layers, num_blocks, block_size, 576]; path [B, max_nodes], accepted [B] as ``tree_accept`` gives
    them, cached_lens [B] the lengths before the step.  In place; returns kv.
    """
    layers, num_blocks, block_size = _need_layers(kv, "kv", _BF16)
    dev = kv.device
    _check(block_table, "block_table", _I32, dev, 2)
    _check(cached_lens, "cached_lens", _I32, dev, 1)
    _check(path, "path", _I32, dev, 2)
    _check(accepted, "accepted", _I32, dev, 1)
    B, max_nodes = path.shape
    if block_table.shape[0] != B or cached_lens.shape[0] != B or accepted.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks], cached_lens and accepted [B] and path [B, max_nodes]")
    with _on(dev, stream):
        code = _lib.load().sfa_kv_commit(kv.data_ptr(), layers, num_blocks, block_size, block_table.data_ptr(),
                                         block_table.shape[1], cached_lens.data_ptr(), path.data_ptr(),
                                         accepted.data_ptr(), B, max_nodes, _raw_stream(dev))
    if code:
        _lib.check("sfa_kv_commit", code)
    return kv


def _need_pool(block_table, shares, free_blocks, taken):
    """The checks of a block table and its pool; returns (device, rows, max_blocks)."""
    if not isinstance(block_table, torch.Tensor) or not block_table.is_cuda:
        raise ValueError("block_table must be on a CUDA device")
    dev = block_table.device
    _check(block_table, "block_table", _I32, dev, 2)
    _check(shares, "shares", _I32, dev, 1)
    _check(free_blocks, "free_blocks", _I32, dev, 1)
    _check(taken, "taken", _I32, dev, 1)
    if taken.shape[0] != 1:
        raise ValueError("taken must be [1]")
    return dev, block_table.shape[0], block_table.shape[1]


def blocks_fork(block_table, lens, src, dst, shares, free_blocks, taken, block_size: int, stream=None):
    """Rows dst become copies of rows src (C ABI ``sfa_blocks_fork``): whole blocks are shared, the
    last, partial one gets a block of its own from the free list.

    block_table [rows, max_blocks], lens [rows], shares [num_blocks] int32, in place (shares: the
    requests that hold a block beyond the first); src, dst [n] int32 rows (< 0 = padding), no row
    twice in dst and none of dst in src; free_blocks [F], taken [1] as in ``step_plan``.  Returns
    (copies [n, 3] int32 for ``kv_copy_blocks``: block, its copy, rows, or -1; taken [1]).
    """
    dev, rows, max_blocks = _need_pool(block_table, shares, free_blocks, taken)
    _check(lens, "lens", _I32, dev, 1)
    _check(src, "src", _I32, dev, 1)
    _check(dst, "dst", _I32, dev, 1)
    n = src.shape[0]
    if lens.shape[0] != rows or dst.shape[0] != n:
        raise ValueError("lens must be [rows], src and dst [n]")
    with _on(dev, stream):
        copies = torch.empty((n, 3), dtype=_I32, device=dev)
        taken_out = torch.empty(1, dtype=_I32, device=dev)
        code = _lib.load().sfa_blocks_fork(block_table.data_ptr(), rows, max_blocks, lens.data_ptr(), src.data_ptr(),
                                           dst.data_ptr(), n, shares.data_ptr(), shares.shape[0],
                                           free_blocks.data_ptr(), free_blocks.shape[0], taken.data_ptr(),
                                           int(block_size), copies.data_ptr(), taken_out.data_ptr(), _raw_stream(dev))
    if code:
        _lib.check("sfa_blocks_fork", code)
    return copies, taken_out


def blocks_free_workspace_bytes(rows: int, max_blocks: int) -> int:
    return int(_lib.load().sfa_blocks_free_workspace_bytes(int(rows), int(max_blocks)))


def blocks_free(block_table, held_lens, keep_lens, shares, free_blocks, taken, block_size: int, workspace=None,
                stream=None):
    """Rows give back the blocks between keep_lens and held_lens positions (C ABI
    ``sfa_blocks_free``): keep 0 ends a request, a little less than held drops rejected drafts.

    held_lens, keep_lens [rows] int32; shares [num_blocks] and free_blocks [F] int32 in place: a
    shared block loses a share, another goes before entry taken[0] of the free list, in the order of
    the table.  Returns taken [1].  The table is left as it is.  workspace:
    blocks_free_workspace_bytes(rows, max_blocks) bytes (allocated when None).
    """
    dev, rows, max_blocks = _need_pool(block_table, shares, free_blocks, taken)
    _check(held_lens, "held_lens", _I32, dev, 1)
    _check(keep_lens, "keep_lens", _I32, dev, 1)
    if held_lens.shape[0] != rows or keep_lens.shape[0] != rows:
        raise ValueError("held_lens and keep_lens must be [rows]")
    lib = _lib.load()
    with _on(dev, stream):
        taken_out = torch.empty(1, dtype=_I32, device=dev)
        need = lib.sfa_blocks_free_workspace_bytes(rows, max_blocks)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        elif workspace is not None and (workspace.get_device() != dev.index or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous and on {dev}")
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        code = lib.sfa_blocks_free(block_table.data_ptr(), held_lens.data_ptr(), keep_lens.data_ptr(), rows,
                                   max_blocks, shares.data_ptr(), shares.shape[0], free_blocks.data_ptr(),
                                   free_blocks.shape[0], taken.data_ptr(), int(block_size), taken_out.data_ptr(),
                                   workspace.data_ptr() if ws_bytes else 0, ws_bytes, _raw_stream(dev))
    if code:
        _lib.check("sfa_blocks_free", code)
    return taken_out


def blocks_compact(block_table, lens, shares, free_blocks, taken, block_size: int, max_moves: int, stream=None):
    """Held blocks move to the front of the pool (C ABI ``sfa_blocks_compact``): the k-th lowest free
    block takes the place of the k-th highest held one while it lies below it, at most max_moves.

    lens [rows] int32: the positions that each row holds.  Returns new (block_table, shares,
    free_blocks, copies [max_moves, 3]); ``kv_copy_blocks`` of copies moves a cache's rows, -1 behind
    the last.  taken stays.
    """
    dev, rows, max_blocks = _need_pool(block_table, shares, free_blocks, taken)
    _check(lens, "lens", _I32, dev, 1)
    if lens.shape[0] != rows:
        raise ValueError("lens must be [rows]")
    max_moves = int(max_moves)
    if max_moves < 0:
        raise ValueError("max_moves must be >= 0")
    with _on(dev, stream):
        table = torch.empty_like(block_table)
        shares_out = torch.empty_like(shares)
        free_out = torch.empty_like(free_blocks)
        copies = torch.empty((max_moves, 3), dtype=_I32, device=dev)
        code = _lib.load().sfa_blocks_compact(block_table.data_ptr(), lens.data_ptr(), rows, max_blocks,
                                              shares.data_ptr(), shares.shape[0], free_blocks.data_ptr(),
                                              free_blocks.shape[0], taken.data_ptr(), int(block_size), max_moves,
                                              table.data_ptr(), shares_out.data_ptr(), free_out.data_ptr(),
                                              copies.data_ptr(), _raw_stream(dev))
    if code:
        _lib.check("sfa_blocks_compact", code)
    return table, shares_out, free_out, copies


def _need_copies(copies, dev):
    _check(copies, "copies", _I32, dev, 2)
    if copies.shape[1] != 3:
        raise ValueError("copies must be [n, 3]")
    return copies.shape[0]


def kv_copy_blocks(kv, copies, stream=None):
    """Copies rows between blocks of a cache (C ABI ``sfa_kv_copy_blocks``): the first copies[i, 2]
    rows of block copies[i, 0] (< 0 = padding) go to block copies[i, 1].

    kv [num_blocks, block_size, 576] bf16, or the caches of several layers, [layers, num_blocks,
    block_size, 576]; copies [n, 3] int32, no block twice as a destination and none both source and
    destination.  In place; returns kv.
    """
    layers, num_blocks, block_size = _need_layers(kv, "kv", _BF16)
    dev = kv.device
    n = _need_copies(copies, dev)
    with _on(dev, stream):
        code = _lib.load().sfa_kv_copy_blocks(kv.data_ptr(), layers, num_blocks, block_size, copies.data_ptr(), n,
                                              _raw_stream(dev))
    if code:
        _lib.check("sfa_kv_copy_blocks", code)
    return kv


def kv_copy_blocks_q8(kv8, scales, copies, stream=None):
    """``kv_copy_blocks`` of an 8-bit cache (C ABI ``sfa_kv_copy_blocks_q8``): kv8 [(layers,)
    num_blocks, block_size, 576] float8_e4m3fn with scales [(layers,) num_blocks, block_size / group]
    fp32, of which the groups that the rows touch are copied too.  In place; returns (kv8, scales).
    """
    layers, num_blocks, block_size = _need_layers(kv8, "kv8", _E4M3)
    dev = kv8.device
    _need(scales, "scales", _F32, dev, kv8.dim() - 1)
    groups = scales.shape[-1]
    if scales.shape[:-1] != kv8.shape[:-2] or groups < 1 or block_size % groups:
        raise ValueError("scales must be [(layers,) num_blocks, block_size / group] with group dividing block_size")
    n = _need_copies(copies, dev)
    with _on(dev, stream):
        code = _lib.load().sfa_kv_copy_blocks_q8(kv8.data_ptr(), scales.data_ptr(), block_size // groups, layers,
                                                 num_blocks, block_size, copies.data_ptr(), n, _raw_stream(dev))
    if code:
        _lib.check("sfa_kv_copy_blocks_q8", code)
    return kv8, scales


def decode_launches(B, Q, h, top_k, block_size, n_splits, merge=True):
    """(kernels one decode call enqueues, which kernel serves it: 2 small-head tcgen05,
    3 stacked-half tcgen05, 1 CTA-pair tcgen05, 0 CUDA-core)."""
    tc = ctypes.c_int(0)
    n = int(_lib.load().sfa_decode_launches(B, Q, h, top_k, block_size, n_splits, int(bool(merge)),
                                            ctypes.byref(tc)))
    if n < 0:
        raise ValueError("invalid decode shape")
    return n, int(tc.value)


def last_device_status(stream=None) -> int:
    """Synchronise the stream, then return and clear the device status word (0 = OK)."""
    lib = _lib.load()
    dev = torch.device("cuda", torch.cuda.current_device())
    return int(lib.sfa_last_device_status(_stream_ptr(stream, dev)))


def set_kernel_path(path: int) -> int:
    """0 = automatic (small-head tcgen05 kernel for h <= 32, stacked-half tcgen05 kernel
    for h <= 64, CTA-pair tcgen05 kernel above), 1 = CUDA-core kernel only, 2 = CTA-pair
    tcgen05 kernel for every h."""
    prev = int(_lib.load().sfa_set_kernel_path(int(path)))
    if prev < 0:
        raise ValueError("path must be 0, 1 or 2")
    return prev


def set_stall_injection(on: bool) -> bool:
    """Test hook (C ABI ``sfa_set_stall_injection``): kernels with bounded waits launched
    afterwards first wait on a barrier nothing completes, so their wait limit runs out and
    they report SFA_ERR_DEVICE_TIMEOUT.  Returns the previous setting."""
    return bool(_lib.load().sfa_set_stall_injection(1 if on else 0))


def set_wait_limit(iterations: int) -> int:
    """Iteration cap of bounded device waits for later launches (0 = default)."""
    return int(_lib.load().sfa_set_wait_limit(int(iterations)))
