"""ZeRO owner-shard optimizer step on one MI355X: Python binding of libzero_shard.so.

Argument marshalling only.  Every step of the path runs in the HIP library
(``csrc/step.hip``, ``csrc/step8.hip``, ``csrc/loss.hip``, ``csrc/copy.hip``, ``csrc/launch.hip``,
``csrc/host.cpp``; C ABI in ``include/zero_shard.h``);
this module turns torch tensors into pointers, checks devices, dtypes,
contiguity and extents against what the kernels will touch, passes torch's
current stream, and raises on error codes.  There is no fallback: if the
library is missing, every call raises.

The functions carry the names of the C entry points.  ``OwnerShard`` bundles
one owner's layout, device chunk table and fp32 state for convenience; its
methods are sequences of the same calls.  ``OwnerShard8`` is the same with both
moments in 8 bits.
"""
from __future__ import annotations

import ctypes as ct
import os
from fractions import Fraction
from typing import List, Optional, Sequence, Tuple

import numpy as np

from .build import LIB_PATH, build

ZERO_OK, ZERO_EINVAL, ZERO_ERANGE, ZERO_EHIP = 0, -1, -2, -3
ZERO_NONE, ZERO_F16, ZERO_BF16, ZERO_F32 = 0, 1, 2, 3
ZERO_MAX_RANKS = 256

EXPORTED = ("zero_last_error", "zero_shard_layout", "zero_chunk_table", "zero_dense_offsets", "zero_state_bytes",
            "zero_reduce_owned", "zero_grad_check", "zero_clip_coef", "zero_step_decision", "zero_adam_step",
            "zero_owner_to_dense", "zero_dense_to_owner", "zero3_storage", "zero3_gather_spans",
            "zero3_partition_spans", "zero_copy_spans", "zero_stream_probe",
            "zero_check_workspace_bytes", "zero_chunk_groups", "zero_span_groups", "zero_reduce_owned_noalloc",
            "zero_piece_table", "zero_adam8_step", "zero_moments8_pack", "zero_moments8_unpack",
            "zero_token_logprobs", "zero_policy_loss", "zero_policy_workspace_bytes",
            "zero_preference_loss", "zero_preference_workspace_bytes")

CHUNK_DTYPE = np.dtype([("flat", "<u8"), ("len", "<u4"), ("tensor", "<u4")])
SPAN_DTYPE = np.dtype([("src", "<u8"), ("dst", "<u8"), ("len", "<u4"), ("buf", "<u4")])
PIECE_DTYPE = np.dtype([("flat", "<u8"), ("len", "<u4"), ("mask", "<u4")])
ZERO_MAX_COPY_SOURCES = 128
ZERO_MAX_PROBE_STREAMS = 64
ZERO_QBLOCK = 128
ZERO_PIECE = 2048
ZERO_PIECE_WHOLE = 0xFFFFFFFF


class ZeroShardError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class AdamArgs(ct.Structure):
    _fields_ = [
        ("chunks", ct.c_void_p), ("n_chunks", ct.c_uint64), ("groups", ct.c_void_p),
        ("n_groups", ct.c_uint64), ("begin", ct.c_uint64),
        ("end", ct.c_uint64),
        ("rank_grads", ct.c_void_p), ("R", ct.c_uint32), ("grad_dtype", ct.c_int32),
        ("grad_base", ct.c_uint64), ("divisor", ct.c_float), ("reduced_g", ct.c_void_p),
        ("master", ct.c_void_p), ("exp_avg", ct.c_void_p), ("exp_avg_sq", ct.c_void_p),
        ("local_base", ct.c_uint64),
        ("param16", ct.c_void_p), ("param_dtype", ct.c_int32), ("param_base", ct.c_uint64),
        ("lr", ct.c_double), ("beta1", ct.c_double), ("beta2", ct.c_double), ("eps", ct.c_double),
        ("weight_decay", ct.c_double), ("adamw", ct.c_int32), ("step", ct.c_uint64),
        ("clip_coef", ct.c_double), ("grid_blocks", ct.c_uint32),
    ]


class Adam8Args(ct.Structure):
    _fields_ = [
        ("pieces", ct.c_void_p), ("n_pieces", ct.c_uint64), ("masks", ct.c_void_p), ("n_masks", ct.c_uint64),
        ("begin", ct.c_uint64), ("end", ct.c_uint64),
        ("rank_grads", ct.c_void_p), ("R", ct.c_uint32), ("grad_dtype", ct.c_int32),
        ("grad_base", ct.c_uint64), ("divisor", ct.c_float), ("reduced_g", ct.c_void_p),
        ("master", ct.c_void_p), ("exp_avg8", ct.c_void_p), ("exp_rms8", ct.c_void_p),
        ("exp_avg_scale", ct.c_void_p), ("exp_rms_scale", ct.c_void_p), ("local_base", ct.c_uint64),
        ("param16", ct.c_void_p), ("param_dtype", ct.c_int32), ("param_base", ct.c_uint64),
        ("lr", ct.c_double), ("beta1", ct.c_double), ("beta2", ct.c_double), ("eps", ct.c_double),
        ("weight_decay", ct.c_double), ("adamw", ct.c_int32), ("step", ct.c_uint64),
        ("clip_coef", ct.c_double),
    ]


class PolicyArgs(ct.Structure):
    _fields_ = [
        ("logits", ct.c_void_p), ("dtype", ct.c_int32), ("n_rows", ct.c_uint64), ("vocab", ct.c_uint32),
        ("row_stride", ct.c_uint64), ("targets", ct.c_void_p), ("old_logp", ct.c_void_p), ("ref_logp", ct.c_void_p),
        ("advantage", ct.c_void_p), ("weight", ct.c_void_p), ("divisor", ct.c_double), ("clip_low", ct.c_double),
        ("clip_high", ct.c_double), ("kl_coef", ct.c_double), ("temperature", ct.c_double), ("grad_scale", ct.c_double),
        ("stats", ct.c_void_p), ("logp", ct.c_void_p), ("dlogits", ct.c_void_p), ("dlogits_stride", ct.c_uint64),
        ("workspace", ct.c_void_p), ("workspace_bytes", ct.c_size_t),
    ]


class PreferenceArgs(ct.Structure):
    _fields_ = [
        ("logits", ct.c_void_p), ("dtype", ct.c_int32), ("n_rows", ct.c_uint64), ("vocab", ct.c_uint32),
        ("row_stride", ct.c_uint64), ("targets", ct.c_void_p), ("seq_begin", ct.c_void_p), ("n_pairs", ct.c_uint32),
        ("ref_logp", ct.c_void_p), ("beta", ct.c_double), ("label_smoothing", ct.c_double), ("average", ct.c_int32),
        ("temperature", ct.c_double), ("grad_scale", ct.c_double), ("stats", ct.c_void_p), ("logp", ct.c_void_p),
        ("seq_logp", ct.c_void_p), ("reward", ct.c_void_p), ("dlogits", ct.c_void_p), ("dlogits_stride", ct.c_uint64),
        ("workspace", ct.c_void_p), ("workspace_bytes", ct.c_size_t),
    ]


class Ratio(ct.Structure):
    _fields_ = [("num", ct.c_uint64), ("den", ct.c_uint64)]


_lib = None


def load(path: str):
    """Open a build of libzero_shard and declare its signatures."""
    L = ct.CDLL(path)
    P, U32, U64, I, F, D = ct.c_void_p, ct.c_uint32, ct.c_uint64, ct.c_int, ct.c_float, ct.c_double
    L.zero_last_error.restype = ct.c_char_p
    L.zero_last_error.argtypes = []
    for name in EXPORTED[1:]:
        getattr(L, name).restype = I
    L.zero_shard_layout.argtypes = [P, U32, U32, U32, P, P, P, P]
    L.zero_chunk_table.argtypes = [P, P, U32, U64, U64, U32, P, U64, P]
    L.zero_dense_offsets.argtypes = [P, U32, P, P]
    L.zero_state_bytes.argtypes = [U64, U64, U32, U32, U32, P]
    L.zero_reduce_owned.argtypes = [P, U32, I, U64, U64, U64, F, I, P, U64, P, P, P, ct.c_size_t, P]
    L.zero_reduce_owned_noalloc.argtypes = [P, U32, I, U64, U64, U64, F, I, P, U64, P, P, P]
    L.zero_grad_check.argtypes = [P, U64, P, P, P, ct.c_size_t, P]
    L.zero_clip_coef.argtypes = [D, D, D, ct.POINTER(F)]
    L.zero_step_decision.argtypes = [P, P, U32, D, D, ct.POINTER(ct.c_int32), ct.POINTER(F)]
    L.zero_adam_step.argtypes = [ct.POINTER(AdamArgs), P]
    L.zero_owner_to_dense.argtypes = [P, U64, P, U64, U64, U64, P, P, U32, P, U64, P, U64, P]
    L.zero_dense_to_owner.argtypes = [P, U64, P, U64, U64, U64, P, P, U32, P, U64, P, U64, P]
    L.zero3_storage.argtypes = [P, U32, U32, P, U32, P, P, P]
    L.zero3_gather_spans.argtypes = [P, U32, U32, P, U32, U32, P, U64, P]
    L.zero3_partition_spans.argtypes = [P, U32, U32, U32, U32, P, U64, P]
    L.zero_copy_spans.argtypes = [P, U64, P, P, U32, P, U64, U32, P, U64, P]
    L.zero_span_groups.argtypes = [P, U64, U32, U32, P, U64, P]
    L.zero_stream_probe.argtypes = [P, P, U32, P, P, U32, U64, I, P]
    L.zero_check_workspace_bytes.argtypes = [U64, P]
    L.zero_chunk_groups.argtypes = [P, U64, U32, P, U64, P]
    L.zero_piece_table.argtypes = [P, P, U32, U64, U64, P, U64, P, U64, P, P]
    L.zero_adam8_step.argtypes = [ct.POINTER(Adam8Args), P]
    L.zero_moments8_pack.argtypes = [P, U64, P, U64, U64, U64, U64, P, P, P, P, P, P, P]
    L.zero_moments8_unpack.argtypes = [P, U64, P, U64, U64, U64, U64, P, P, P, P, P, P, P]
    L.zero_token_logprobs.argtypes = [P, I, U64, U32, U64, P, D, P, P]
    L.zero_policy_loss.argtypes = [ct.POINTER(PolicyArgs), P]
    L.zero_policy_workspace_bytes.argtypes = [U64, P]
    L.zero_preference_loss.argtypes = [ct.POINTER(PreferenceArgs), P]
    L.zero_preference_workspace_bytes.argtypes = [U64, U32, P]
    return L


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run __graft_entry__.build() "
                               "(there is no fallback path)")
        _lib = load(LIB_PATH)
    return _lib


def _check(rc: int) -> None:
    if rc != ZERO_OK:
        raise ZeroShardError(rc, lib().zero_last_error().decode())


def _u64(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.uint64))


def _sizes(numels) -> np.ndarray:
    """Tensor sizes as uint64, from any iterable of numbers (a generator over a model's parameters)."""
    if isinstance(numels, np.ndarray) and numels.dtype == np.uint64 and numels.ndim == 1:
        return np.ascontiguousarray(numels)
    return np.fromiter(map(int, numels), dtype=np.uint64)


def _p(a: np.ndarray):
    return ct.c_void_p(a.ctypes.data) if a is not None and a.size else None


# ---------------------------------------------------------------- host calls
def zero_shard_layout(numels: Sequence[int], ranks: int, align: int):
    """(tensor offsets, padded total, owner begins, owner ends) of the flat buffer."""
    n = _u64(numels)
    off = np.zeros(max(1, n.size), dtype=np.uint64)
    total = np.zeros(1, dtype=np.uint64)
    b = np.zeros(max(1, ranks), dtype=np.uint64)
    e = np.zeros(max(1, ranks), dtype=np.uint64)
    _check(lib().zero_shard_layout(_p(n), n.size, ranks, align, _p(off), _p(total), _p(b), _p(e)))
    return off[: n.size], int(total[0]), b[:ranks], e[:ranks]


def zero_chunk_table(numels: Sequence[int], offsets: Sequence[int], begin: int, end: int,
                     max_chunk: int) -> np.ndarray:
    """The owner's chunks as a structured array (flat, len, tensor)."""
    n, off = _u64(numels), _u64(offsets)
    if n.size != off.size:
        raise ValueError("numels and offsets differ in length")
    count = np.zeros(1, dtype=np.uint64)
    _check(lib().zero_chunk_table(_p(n), _p(off), n.size, begin, end, max_chunk, None, 0, _p(count)))
    out = np.zeros(int(count[0]), dtype=CHUNK_DTYPE)
    _check(lib().zero_chunk_table(_p(n), _p(off), n.size, begin, end, max_chunk,
                                  _p(out) if out.size else None, out.size, _p(count)))
    return out


def zero_dense_offsets(numels: Sequence[int]):
    """(start of each tensor in the dense unpadded layout, dense total)."""
    n = _u64(numels)
    off = np.zeros(max(1, n.size), dtype=np.uint64)
    total = np.zeros(1, dtype=np.uint64)
    _check(lib().zero_dense_offsets(_p(n), n.size, _p(off), _p(total)))
    return off[: n.size], int(total[0])


def groups_pay(n_groups: int, n_items: int) -> bool:
    """Whether a group table is worth its indirection: a group kernel block
    first reads its group bounds, then its chunks or spans, and that extra
    dependent load cost 17% on a span copy of long spans.  Packing pays when
    it at least halves the block count (512-element spans: +84%)."""
    return 2 * n_groups <= n_items


def zero_chunk_groups(chunks: np.ndarray, max_group: int) -> np.ndarray:
    """Group table (first chunk of each group, then len(chunks)) packing runs of
    short chunks for zero_adam_step; uint64, n_groups + 1 entries."""
    ch = np.ascontiguousarray(chunks, dtype=CHUNK_DTYPE)
    count = np.zeros(1, dtype=np.uint64)
    _check(lib().zero_chunk_groups(_p(ch), ch.size, max_group, None, 0, _p(count)))
    out = np.zeros(int(count[0]) + 1, dtype=np.uint64)
    _check(lib().zero_chunk_groups(_p(ch), ch.size, max_group, _p(out), out.size, _p(count)))
    return out


def zero_piece_table(numels: Sequence[int], offsets: Sequence[int], begin: int, end: int):
    """The owner's pieces as a structured array (flat, len, mask) and the mask bytes of
    those that hold padding, uint8 [n_masks, ZERO_PIECE / 8]."""
    n, off = _u64(numels), _u64(offsets)
    if n.size != off.size:
        raise ValueError("numels and offsets differ in length")
    most = max(0, end - begin) // ZERO_PIECE + 2  # windows that the range can touch
    out, masks = np.empty(most, dtype=PIECE_DTYPE), np.empty((most, ZERO_PIECE // 8), dtype=np.uint8)
    count, n_masks = np.zeros(1, dtype=np.uint64), np.zeros(1, dtype=np.uint64)
    _check(lib().zero_piece_table(_p(n), _p(off), n.size, begin, end, _p(out), most, _p(masks), most, _p(count),
                                  _p(n_masks)))
    return out[:int(count[0])].copy(), masks[:int(n_masks[0])].copy()


def zero_state_bytes(params: int, ranks: int, param: int = 2, grad: int = 2,
                     optimizer: int = 12) -> dict:
    out = (Ratio * 4)()
    _check(lib().zero_state_bytes(params, ranks, param, grad, optimizer, out))
    names = ("DP", "ZeRO-1", "ZeRO-2", "ZeRO-3")
    return {k: Fraction(out[i].num, out[i].den) for i, k in enumerate(names)}


def zero_clip_coef(sumsq: float, max_norm: float = 1.0, eps: float = 1e-6) -> float:
    c = ct.c_float()
    _check(lib().zero_clip_coef(sumsq, max_norm, eps, ct.byref(c)))
    return c.value


def zero_step_decision(overflow: Sequence[int], sumsq: Sequence[float], max_norm: float = 1.0,
                       eps: float = 1e-6):
    """(update, clip factor) from every owner's (flag, squared-norm partial), in
    owner order; the factor is None when the step is skipped."""
    fl = np.ascontiguousarray(np.asarray(overflow, dtype=np.int32))
    ss = np.ascontiguousarray(np.asarray(sumsq, dtype=np.float64))
    if fl.size != ss.size:
        raise ValueError("one flag and one partial per owner")
    up, c = ct.c_int32(), ct.c_float()
    _check(lib().zero_step_decision(_p(fl), _p(ss), fl.size, max_norm, eps, ct.byref(up), ct.byref(c)))
    return (True, c.value) if up.value else (False, None)


# ---------------------------------------------------------------- device calls
def _torch():
    import torch

    return torch


_dtype_codes = None


def _dtype_code(t) -> int:
    global _dtype_codes
    if _dtype_codes is None:
        torch = _torch()
        _dtype_codes = {torch.float16: ZERO_F16, torch.bfloat16: ZERO_BF16, torch.float32: ZERO_F32}
    return _dtype_codes[t.dtype]


def _device(device):
    """Where a call puts what it makes: the current device unless one is named (0 is one)."""
    return "cuda" if device is None else device


def _dev(t, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.device.index != _torch().cuda.current_device():
        # the kernels run on the current device's stream
        raise ValueError(f"{name} lives on {t.device}, not on the current device "
                         f"cuda:{_torch().cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _stream():
    return ct.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _device_stream():
    """(current device's index, its current stream as an address)."""
    torch = _torch()
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _addr(t, name: str, dtype, elems: int, dev: int) -> int:
    """The address of a contiguous tensor of one dtype on device `dev` with at least
    `elems` elements; a tensor that is not that gets the error of the check it fails."""
    if t.get_device() != dev or t.dtype is not dtype or not t.is_contiguous() or t.numel() < elems:
        _dev(t, name, dtype)
        _need(t, name, elems)
    return t.data_ptr()


def _need(t, name: str, elems: int) -> None:
    if t.numel() < elems:
        raise ValueError(f"{name} holds {t.numel()} elements, {elems} needed")


def _rank_ptrs(rank_grads, base: int, last: int, name="rank_grads"):
    if not rank_grads:
        raise ValueError("no rank buffers")
    dt = rank_grads[0].dtype
    dev = rank_grads[0].device
    arr = (ct.c_void_p * len(rank_grads))()
    for r, g in enumerate(rank_grads):
        _dev(g, f"{name}[{r}]", dt)
        if g.device != dev:
            raise ValueError("rank buffers on different devices")
        _need(g, f"{name}[{r}]", last - base)
        arr[r] = g.data_ptr()
    return arr, _dtype_code(rank_grads[0])


def zero_reduce_owned(rank_grads, begin: int, n: int, divisor: float, out, *, grad_base: int = 0,
                      out_base: int = 0, accumulate: int = 0, check=None) -> None:
    """Rank reduce over flat indices [begin, begin+n) into ``out[f - out_base]``.

    ``accumulate``: 0 ``out = sum/D``; 1 (or True) ``out = (out + sum)/D``;
    2 ``out = out + sum/D`` (per-backward reduce-and-accumulate).

    ``check`` = (overflow int32[1], sumsq float64[1], workspace uint8[>= check_workspace_bytes(n)])
    device tensors to also compute the overflow flag and squared norm in the same pass.
    """
    torch = _torch()
    arr, code = _rank_ptrs(rank_grads, grad_base, begin + n)
    _dev(out, "out", torch.float32)
    _need(out, "out", begin + n - out_base)
    ov = ss = ws = None
    ws_bytes = 0
    if check is not None:
        ov, ss, ws = check
        _dev(ov, "overflow", torch.int32)
        _dev(ss, "sumsq", torch.float64)
        _dev(ws, "workspace")
        ws_bytes = ws.numel() * ws.element_size()
    _check(lib().zero_reduce_owned(
        arr, len(rank_grads), code, grad_base, begin, n, divisor, int(accumulate),
        ct.c_void_p(out.data_ptr()), out_base,
        ct.c_void_p(ov.data_ptr()) if ov is not None else None,
        ct.c_void_p(ss.data_ptr()) if ss is not None else None,
        ct.c_void_p(ws.data_ptr()) if ws is not None else None, ws_bytes, _stream()))


def zero_reduce_owned_noalloc(rank_grads, begin: int, n: int, divisor: float, out, *, grad_base: int = 0,
                              out_base: int = 0, accumulate: int = 0, check=None) -> None:
    """``zero_reduce_owned`` whose check needs no workspace: ``check`` = (overflow
    int32[1], sumsq float64[1]); the partials go to the library's own device
    array (calls on one GPU must not overlap)."""
    torch = _torch()
    arr, code = _rank_ptrs(rank_grads, grad_base, begin + n)
    _dev(out, "out", torch.float32)
    _need(out, "out", begin + n - out_base)
    ov = ss = None
    if check is not None:
        ov, ss = check
        _dev(ov, "overflow", torch.int32)
        _dev(ss, "sumsq", torch.float64)
    _check(lib().zero_reduce_owned_noalloc(
        arr, len(rank_grads), code, grad_base, begin, n, divisor, int(accumulate),
        ct.c_void_p(out.data_ptr()), out_base,
        ct.c_void_p(ov.data_ptr()) if ov is not None else None,
        ct.c_void_p(ss.data_ptr()) if ss is not None else None, _stream()))


def zero_grad_check(g, overflow, sumsq, workspace) -> None:
    torch = _torch()
    _dev(g, "g", torch.float32)
    _dev(overflow, "overflow", torch.int32)
    _dev(sumsq, "sumsq", torch.float64)
    _dev(workspace, "workspace")
    _check(lib().zero_grad_check(
        ct.c_void_p(g.data_ptr()), g.numel(), ct.c_void_p(overflow.data_ptr()),
        ct.c_void_p(sumsq.data_ptr()), ct.c_void_p(workspace.data_ptr()),
        workspace.numel() * workspace.element_size(), _stream()))


def check_workspace_bytes(n: int) -> int:
    """Bytes of device workspace a check over n elements needs."""
    out = np.zeros(1, dtype=np.uint64)
    _check(lib().zero_check_workspace_bytes(n, _p(out)))
    return int(out[0])


def check_workspace(n: int, device=None):
    """A device buffer for the overflow / norm reduction over n elements."""
    torch = _torch()
    return torch.empty(check_workspace_bytes(n), dtype=torch.uint8, device=_device(device))


def chunks_to_device(chunks: np.ndarray, device=None):
    torch = _torch()
    flat = np.ascontiguousarray(chunks).view(np.uint8)
    t = torch.from_numpy(flat.copy()).to(_device(device))
    return t


def zero_adam_step(*, chunks_dev, n_chunks: int, begin: int, end: int, master, exp_avg, exp_avg_sq,
                   local_base: int, step: int, lr: float, beta1: float, beta2: float, eps: float,
                   weight_decay: float = 0.0, adamw: bool = True, rank_grads=None, grad_base: int = 0,
                   divisor: float = 1.0, reduced_g=None, param16=None, param_base: int = 0,
                   clip_coef: float = 1.0, grid_blocks: int = 0, groups_dev=None, n_groups: int = 0) -> None:
    """Fused reduce + Adam/AdamW + 16-bit write-back over a device chunk table
    (optionally packed by a device group table from ``zero_chunk_groups``).

    The kernel touches only flat indices in [begin, end) (chunk pieces outside are
    ignored), so every buffer is checked to hold those.
    """
    torch = _torch()
    last = end
    if chunks_dev is not None:
        _dev(chunks_dev, "chunks")
        if chunks_dev.numel() * chunks_dev.element_size() < n_chunks * CHUNK_DTYPE.itemsize:
            raise ValueError("chunk table smaller than n_chunks")
    for name, t in (("master", master), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)):
        _dev(t, name, torch.float32)
        _need(t, name, last - local_base)
    a = AdamArgs()
    a.chunks = chunks_dev.data_ptr() if chunks_dev is not None else None
    a.n_chunks, a.begin, a.end = n_chunks, begin, end
    if groups_dev is not None:
        _dev(groups_dev, "groups", torch.int64)
        if groups_dev.numel() < n_groups + 1:
            raise ValueError("group table smaller than n_groups + 1")
        a.groups, a.n_groups = groups_dev.data_ptr(), n_groups
    elif n_groups:
        raise ValueError("n_groups given without a group table")
    keep = None
    if reduced_g is not None:
        _dev(reduced_g, "reduced_g", torch.float32)
        _need(reduced_g, "reduced_g", last - local_base)
        a.reduced_g = reduced_g.data_ptr()
    else:
        keep, code = _rank_ptrs(rank_grads, grad_base, last)
        a.rank_grads = ct.cast(keep, ct.c_void_p)
        a.R, a.grad_dtype, a.grad_base = len(rank_grads), code, grad_base
    a.divisor = divisor
    a.master, a.exp_avg, a.exp_avg_sq = master.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr()
    a.local_base = local_base
    if param16 is not None:
        _dev(param16, "param16")
        if param16.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("param16 must be float16 or bfloat16")
        _need(param16, "param16", last - param_base)
        a.param16, a.param_dtype, a.param_base = param16.data_ptr(), _dtype_code(param16), param_base
    a.lr, a.beta1, a.beta2, a.eps, a.weight_decay = lr, beta1, beta2, eps, weight_decay
    a.adamw, a.step, a.clip_coef, a.grid_blocks = int(adamw), step, clip_coef, grid_blocks
    _check(lib().zero_adam_step(ct.byref(a), _stream()))
    del keep


def _group_ptr(groups_dev, n_groups):
    if groups_dev is None:
        if n_groups:
            raise ValueError("n_groups given without a group table")
        return None, 0
    _dev(groups_dev, "groups", _torch().int64)
    if groups_dev.numel() < n_groups + 1:
        raise ValueError("group table smaller than n_groups + 1")
    return ct.c_void_p(groups_dev.data_ptr()), n_groups


def _dense_call(name, chunks_dev, n_chunks, begin, end, tensor_offset_dev, dense_offset_dev, owner,
                owner_base, dense, groups_dev=None, n_groups=0):
    torch = _torch()
    _dev(owner, "owner", torch.float32)
    _dev(dense, "dense", torch.float32)
    _dev(tensor_offset_dev, "tensor_offset", torch.int64)
    _dev(dense_offset_dev, "dense_offset", torch.int64)
    if tensor_offset_dev.numel() != dense_offset_dev.numel():
        raise ValueError("tensor and dense offset tables differ in length")
    _need(owner, "owner", end - owner_base)
    if chunks_dev is not None and chunks_dev.numel() * chunks_dev.element_size() < n_chunks * CHUNK_DTYPE.itemsize:
        raise ValueError("chunk table smaller than n_chunks")
    L = lib()
    gptr, ng = _group_ptr(groups_dev, n_groups)
    common = (ct.c_void_p(chunks_dev.data_ptr()) if chunks_dev is not None else None, n_chunks, gptr, ng,
              begin, end, ct.c_void_p(tensor_offset_dev.data_ptr()), ct.c_void_p(dense_offset_dev.data_ptr()),
              tensor_offset_dev.numel())
    if name == "zero_owner_to_dense":
        _check(L.zero_owner_to_dense(*common, ct.c_void_p(owner.data_ptr()), owner_base,
                                     ct.c_void_p(dense.data_ptr()), dense.numel(), _stream()))
    else:
        _check(L.zero_dense_to_owner(*common, ct.c_void_p(dense.data_ptr()), dense.numel(),
                                     ct.c_void_p(owner.data_ptr()), owner_base, _stream()))


def zero_owner_to_dense(chunks_dev, n_chunks, begin, end, tensor_offset_dev, dense_offset_dev, owner,
                        owner_base, dense, groups_dev=None, n_groups: int = 0) -> None:
    """dense[dense_offset[k] + f - tensor_offset[k]] = owner[f - owner_base] for the owner's real f."""
    _dense_call("zero_owner_to_dense", chunks_dev, n_chunks, begin, end, tensor_offset_dev,
                dense_offset_dev, owner, owner_base, dense, groups_dev, n_groups)


def zero_dense_to_owner(chunks_dev, n_chunks, begin, end, tensor_offset_dev, dense_offset_dev, dense,
                        owner, owner_base, groups_dev=None, n_groups: int = 0) -> None:
    """owner[f - owner_base] = dense[dense_offset[k] + f - tensor_offset[k]] for the owner's real f."""
    _dense_call("zero_dense_to_owner", chunks_dev, n_chunks, begin, end, tensor_offset_dev,
                dense_offset_dev, owner, owner_base, dense, groups_dev, n_groups)


# ---------------------------------------------------------------- ZeRO-3 partition / gather
def _live(live):
    return np.ascontiguousarray(np.asarray(list(live), dtype=np.uint32))


def zero3_storage(numels: Sequence[int], ranks: int, live: Sequence[int] = ()):
    """(shard sizes, resident, gathered) element counts of per-tensor ZeRO-3 partitioning."""
    n, lv = _u64(numels), _live(live)
    shard = np.zeros(max(1, n.size), dtype=np.uint64)
    res, gat = np.zeros(1, dtype=np.uint64), np.zeros(1, dtype=np.uint64)
    _check(lib().zero3_storage(_p(n), n.size, ranks, _p(lv), lv.size, _p(shard), _p(res), _p(gat)))
    return shard[: n.size], int(res[0]), int(gat[0])


# Span length of the copy tables: one block copies one span, and 4096 elements
# (8 KiB of bf16 each way) measured fastest for the stage-3 gather (2048: -8%,
# 8192: -5%).
DEFAULT_SPAN = 4096


def _spans(fn, *args, max_span):
    count = np.zeros(1, dtype=np.uint64)
    _check(fn(*args, max_span, None, 0, _p(count)))
    out = np.zeros(int(count[0]), dtype=SPAN_DTYPE)
    _check(fn(*args, max_span, _p(out) if out.size else None, out.size, _p(count)))
    return out


def zero3_gather_spans(numels, ranks: int, live, max_span: int = DEFAULT_SPAN) -> np.ndarray:
    n, lv = _u64(numels), _live(live)
    return _spans(lib().zero3_gather_spans, _p(n), n.size, ranks, _p(lv), lv.size, max_span=max_span)


def zero3_partition_spans(numels, ranks: int, rank: int, max_span: int = DEFAULT_SPAN) -> np.ndarray:
    n = _u64(numels)
    return _spans(lib().zero3_partition_spans, _p(n), n.size, ranks, rank, max_span=max_span)


def spans_to_device(spans: np.ndarray, device=None):
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(spans).view(np.uint8).copy()).to(_device(device))


def zero_span_groups(spans: np.ndarray, elem_bytes: int, max_group: int = DEFAULT_SPAN) -> np.ndarray:
    """Group table (first span of each group, then len(spans)) packing runs of
    short spans for zero_copy_spans; uint64, n_groups + 1 entries."""
    sp = np.ascontiguousarray(spans, dtype=SPAN_DTYPE)
    count = np.zeros(1, dtype=np.uint64)
    _check(lib().zero_span_groups(_p(sp), sp.size, elem_bytes, max_group, None, 0, _p(count)))
    out = np.zeros(int(count[0]) + 1, dtype=np.uint64)
    _check(lib().zero_span_groups(_p(sp), sp.size, elem_bytes, max_group, _p(out), out.size, _p(count)))
    return out


def zero_copy_spans(spans_dev, n_spans: int, srcs, dst, groups_dev=None, n_groups: int = 0) -> None:
    """dst[span.dst + i] = srcs[span.buf][span.src + i] over a device span table
    (optionally packed by a device group table from ``zero_span_groups``)."""
    torch = _torch()
    if not srcs or len(srcs) > ZERO_MAX_COPY_SOURCES:
        raise ValueError(f"between 1 and {ZERO_MAX_COPY_SOURCES} source buffers")
    _dev(dst, "dst")
    if dst.element_size() not in (2, 4):
        raise TypeError("elements must be 2 or 4 bytes")
    arr = (ct.c_void_p * len(srcs))()
    sizes = np.zeros(len(srcs), dtype=np.uint64)
    for i, t in enumerate(srcs):
        _dev(t, f"srcs[{i}]", dst.dtype)
        arr[i] = t.data_ptr()
        sizes[i] = t.numel()
    if spans_dev is not None:
        _dev(spans_dev, "spans")
        if spans_dev.numel() * spans_dev.element_size() < n_spans * SPAN_DTYPE.itemsize:
            raise ValueError("span table smaller than n_spans")
    gptr, ng = _group_ptr(groups_dev, n_groups)
    _check(lib().zero_copy_spans(ct.c_void_p(spans_dev.data_ptr()) if spans_dev is not None else None,
                                 n_spans, arr, _p(sizes), len(srcs), ct.c_void_p(dst.data_ptr()),
                                 dst.numel(), dst.element_size(), gptr, ng, _stream()))


def zero_stream_probe(srcs, dsts, order: int = 0, src_widths=None, dst_widths=None) -> None:
    """Bandwidth probe: every destination gets the bytewise XOR of all sources.

    A stream of width w (1 or 2; default 1) is touched w 16-byte vectors per
    thread, as the kernels stream 16-bit (w = 1) and fp32 (w = 2) data; every
    stream's byte size is its width times one common unit (a multiple of 16).
    No destinations: reads only; no sources: writes zeros.  ``order`` 0 deals
    the pieces to the XCDs in turn, 1 gives each XCD one contiguous run.
    """
    if len(srcs) > ZERO_MAX_PROBE_STREAMS or len(dsts) > ZERO_MAX_PROBE_STREAMS or not (srcs or dsts):
        raise ValueError(f"at most {ZERO_MAX_PROBE_STREAMS} sources and destinations, not none of both")
    sw = np.ascontiguousarray(np.asarray(src_widths if src_widths is not None else [1] * len(srcs), dtype=np.uint8))
    dw = np.ascontiguousarray(np.asarray(dst_widths if dst_widths is not None else [1] * len(dsts), dtype=np.uint8))
    if sw.size != len(srcs) or dw.size != len(dsts) or not np.all((sw == 1) | (sw == 2)) or \
            not np.all((dw == 1) | (dw == 2)):
        raise ValueError("one width of 1 or 2 per stream")
    streams = list(zip(srcs, sw.tolist())) + list(zip(dsts, dw.tolist()))
    first, w0 = streams[0]
    unit = first.numel() * first.element_size() // w0
    sa, da = (ct.c_void_p * max(1, len(srcs)))(), (ct.c_void_p * max(1, len(dsts)))()
    for arr, ts, ws, name in ((sa, srcs, sw, "srcs"), (da, dsts, dw, "dsts")):
        for i, t in enumerate(ts):
            _dev(t, f"{name}[{i}]")
            if t.numel() * t.element_size() != unit * int(ws[i]):
                raise ValueError("every probe stream must hold its width times one common unit of bytes")
            arr[i] = t.data_ptr()
    _check(lib().zero_stream_probe(sa, _p(sw), len(srcs), da, _p(dw), len(dsts), unit, int(order), _stream()))


# ---------------------------------------------------------------- the step with 8-bit moments
def _pieces8(dev, pieces_dev, n_pieces, masks_dev, begin, end):
    """Checks a piece table; (pieces, n_pieces, masks, n_masks, begin, end) as the calls take them."""
    torch = _torch()
    if n_pieces < 0 or begin < 0 or end < 0:  # as unsigned they would pass the checks of sizes
        raise ValueError(f"negative n_pieces, begin or end: {n_pieces}, {begin}, {end}")
    pieces = masks = None
    n_masks = 0
    if pieces_dev is not None:
        pieces = _addr(pieces_dev, "pieces", torch.uint8, n_pieces * PIECE_DTYPE.itemsize, dev)
    if masks_dev is not None and masks_dev.numel():
        masks = _addr(masks_dev, "masks", torch.uint8, 0, dev)
        n_masks = masks_dev.numel() // (ZERO_PIECE // 8)
    return pieces, n_pieces, masks, n_masks, begin, end


def _state8(dev, end, local_base, exp_avg8, exp_avg_scale, exp_rms8, exp_rms_scale):
    """Checks the 8-bit state; its addresses (codes, scales of the first moment; codes, scales of the second)."""
    torch = _torch()
    blocks = -(-(end - local_base) // ZERO_QBLOCK)
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    return (_addr(exp_avg8, "exp_avg8", e4m3, blocks * ZERO_QBLOCK, dev),
            _addr(exp_avg_scale, "exp_avg_scale", f32, blocks, dev),
            _addr(exp_rms8, "exp_rms8", e4m3, blocks * ZERO_QBLOCK, dev),
            _addr(exp_rms_scale, "exp_rms_scale", f32, blocks, dev))


def _adam8(dev, stream, work, narrow, local_base, master, hyper, step, rank_grads, grad_base, divisor, reduced_g,
           param16, param_base, clip_coef):
    """The call itself, after _state8's checks: checks the other tensors and marshals."""
    torch = _torch()
    f32, end = torch.float32, work[5]
    ranks = g = p16 = None
    R = code = 0
    if reduced_g is not None:
        g = _addr(reduced_g, "reduced_g", f32, end - local_base, dev)
    else:
        if not rank_grads:
            raise ValueError("no rank buffers")
        R, dt, need = len(rank_grads), rank_grads[0].dtype, end - grad_base
        code = _dtype_code(rank_grads[0])
        ranks = (ct.c_void_p * R)(*[_addr(x, "rank_grads", dt, need, dev) for x in rank_grads])
    pdt = ZERO_NONE
    if param16 is not None:
        if param16.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("param16 must be float16 or bfloat16")
        p16, pdt = _addr(param16, "param16", param16.dtype, end - param_base, dev), _dtype_code(param16)
    m8, ms, r8, rs = narrow
    lr, beta1, beta2, eps, weight_decay, adamw = hyper
    a = Adam8Args(*work, ct.addressof(ranks) if ranks is not None else None, R, code, grad_base, divisor, g,
                  _addr(master, "master", f32, end - local_base, dev), m8, r8, ms, rs, local_base, p16, pdt,
                  param_base, lr, beta1, beta2, eps, weight_decay, int(adamw), step, clip_coef)
    _check(lib().zero_adam8_step(ct.byref(a), stream))


def _hyper(lr, beta1, beta2, eps, weight_decay=0.0, adamw=True):
    return lr, beta1, beta2, eps, weight_decay, adamw


def zero_adam8_step(*, pieces_dev, n_pieces: int, masks_dev=None, begin: int, end: int, master, exp_avg8,
                    exp_avg_scale, exp_rms8, exp_rms_scale, local_base: int, step: int, lr: float, beta1: float,
                    beta2: float, eps: float, weight_decay: float = 0.0, adamw: bool = True, rank_grads=None,
                    grad_base: int = 0, divisor: float = 1.0, reduced_g=None, param16=None, param_base: int = 0,
                    clip_coef: float = 1.0) -> None:
    """Fused reduce + Adam/AdamW + 16-bit write-back whose moments are held in 8 bits:
    ``exp_avg8``/``exp_rms8`` float8_e4m3fn codes, one fp32 scale per ZERO_QBLOCK of them,
    over a device piece table from ``zero_piece_table``."""
    dev, stream = _device_stream()
    work = _pieces8(dev, pieces_dev, n_pieces, masks_dev, begin, end)
    narrow = _state8(dev, end, local_base, exp_avg8, exp_avg_scale, exp_rms8, exp_rms_scale)
    _adam8(dev, stream, work, narrow, local_base, master, (lr, beta1, beta2, eps, weight_decay, adamw), step,
           rank_grads, grad_base, divisor, reduced_g, param16, param_base, clip_coef)


def _moments8(pack, dev, stream, work, narrow, local_base, exp_avg, exp_avg_sq):
    f32, need = _torch().float32, work[5] - local_base
    wide = _addr(exp_avg, "exp_avg", f32, need, dev), _addr(exp_avg_sq, "exp_avg_sq", f32, need, dev)
    if pack:
        _check(lib().zero_moments8_pack(*work, local_base, *wide, *narrow, stream))
    else:
        _check(lib().zero_moments8_unpack(*work, local_base, *narrow, *wide, stream))


def zero_moments8_pack(*, exp_avg, exp_avg_sq, pieces_dev, n_pieces, masks_dev=None, begin, end, local_base, exp_avg8,
                       exp_avg_scale, exp_rms8, exp_rms_scale) -> None:
    """The owner's fp32 moments into their 8-bit form."""
    dev, stream = _device_stream()
    _moments8(True, dev, stream, _pieces8(dev, pieces_dev, n_pieces, masks_dev, begin, end),
              _state8(dev, end, local_base, exp_avg8, exp_avg_scale, exp_rms8, exp_rms_scale), local_base, exp_avg,
              exp_avg_sq)


def zero_moments8_unpack(*, exp_avg, exp_avg_sq, pieces_dev, n_pieces, masks_dev=None, begin, end, local_base, exp_avg8,
                         exp_avg_scale, exp_rms8, exp_rms_scale) -> None:
    """The owner's 8-bit moments as fp32 (scale * code, and the root's square)."""
    dev, stream = _device_stream()
    _moments8(False, dev, stream, _pieces8(dev, pieces_dev, n_pieces, masks_dev, begin, end),
              _state8(dev, end, local_base, exp_avg8, exp_avg_scale, exp_rms8, exp_rms_scale), local_base, exp_avg,
              exp_avg_sq)


# ---------------------------------------------------------------- losses on token log-probabilities
def _rows(t, name: str, dev: int):
    """(rows, vocabulary, row stride) of a [rows, vocabulary] device tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, vocabulary], got {t.dim()} dimensions")
    if t.get_device() != dev:
        _dev(t, name)
    (n, v), (stride, inner) = t.shape, t.stride()
    if v > 1 and inner != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if n <= 1:
        stride = v
    elif stride < v:
        raise ValueError(f"the rows of {name} overlap")
    return n, v, stride


def _logits(logits, targets, dlogits=None):
    """The device's index, its stream, (logits, dtype, rows, vocabulary, row stride, targets) and (dlogits, row stride)."""
    torch = _torch()
    dt = logits.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16 and dt is not torch.float32:
        raise TypeError(f"logits must be float16, bfloat16 or float32, got {dt}")
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    dev, stream = _device_stream()
    n, v, stride = _rows(logits, "logits", dev)
    if targets.numel() != n:
        raise ValueError(f"{targets.numel()} targets for {n} rows")
    tptr = _addr(targets, "targets", torch.int64, n, dev)
    grad = (None, 0)
    if dlogits is not None:
        if dlogits.dtype is not dt or dlogits.shape != logits.shape:
            raise ValueError("dlogits must have the dtype and shape of logits")
        grad = (dlogits.data_ptr(), _rows(dlogits, "dlogits", dev)[2])
    return dev, stream, (logits.data_ptr(), _dtype_code(logits), n, v, stride, tptr), grad


def _space(t, dev: int):
    """(address, bytes) of a workspace."""
    return _addr(t, "workspace", t.dtype, 0, dev), t.numel() * t.element_size()


def zero_token_logprobs(logits, targets, logp, *, temperature: float = 1.0) -> None:
    """``logp[r]`` = log-probability of ``targets[r]`` under row r of ``logits`` / temperature.

    ``logits`` [rows, vocabulary] float16, bfloat16 or float32 with contiguous rows at
    any row stride; ``targets`` int64; ``logp`` float32.  A target outside the
    vocabulary (-100) gives 0.
    """
    dev, stream, rows, _ = _logits(logits, targets)
    _check(lib().zero_token_logprobs(*rows, temperature, _addr(logp, "logp", _torch().float32, rows[2], dev), stream))


def _workspace(fn, *sizes, device=None):
    out = np.zeros(1, dtype=np.uint64)
    _check(fn(*sizes, _p(out)))
    torch = _torch()
    return torch.zeros(int(out[0]), dtype=torch.uint8, device=_device(device))


def policy_workspace(n_rows: int, device=None):
    """The device workspace of ``zero_policy_loss`` over up to n_rows rows: zeros before
    its first use, then left ready for the next call (one call at a time).  Any other
    contents show as NaN in ``stats``."""
    return _workspace(lib().zero_policy_workspace_bytes, n_rows, device=device)


def preference_workspace(n_rows: int, n_pairs: int, device=None):
    """The device workspace of ``zero_preference_loss`` over up to n_rows rows and n_pairs pairs."""
    return _workspace(lib().zero_preference_workspace_bytes, n_rows, n_pairs, device=device)


def zero_policy_loss(logits, targets, *, old_logp, advantage, divisor: float, stats, logp, workspace, ref_logp=None,
                     weight=None, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                     temperature: float = 1.0, grad_scale: float = 1.0, dlogits=None) -> None:
    """Clipped policy loss with a KL term, and its gradient of the logits.

    With lp the targets' log-probabilities, rho = exp(lp - old_logp) and
    d = ref_logp - lp, row r adds weight * (-min(A rho, A clip(rho, 1 - clip_low,
    1 + clip_high)) + kl_coef (exp(d) - d - 1)) / divisor to the loss.

    Written: ``stats`` float32 [4] (loss, policy part, KL part without kl_coef, clipped
    share), ``logp`` float32 [rows], and ``dlogits`` (optional; dtype and shape of
    ``logits``, may be ``logits`` itself) = grad_scale * gradient, for
    ``hidden_logits.backward(dlogits)``.  A target outside the vocabulary marks a row
    that counts for nothing.  ``workspace`` from ``policy_workspace``.
    """
    f32 = _torch().float32
    dev, stream, rows, grad = _logits(logits, targets, dlogits)
    n = rows[2]
    a = PolicyArgs(*rows, _addr(old_logp, "old_logp", f32, n, dev),
                   None if ref_logp is None else _addr(ref_logp, "ref_logp", f32, n, dev),
                   _addr(advantage, "advantage", f32, n, dev),
                   None if weight is None else _addr(weight, "weight", f32, n, dev), divisor, clip_low, clip_high,
                   kl_coef, temperature, grad_scale, _addr(stats, "stats", f32, 4, dev),
                   _addr(logp, "logp", f32, n, dev), *grad, *_space(workspace, dev))
    _check(lib().zero_policy_loss(ct.byref(a), stream))


def zero_preference_loss(logits, targets, seq_begin, *, ref_logp, stats, logp, seq_logp, reward, workspace,
                         beta: float = 0.1, label_smoothing: float = 0.0, average: bool = False,
                         temperature: float = 1.0, grad_scale: float = 1.0, dlogits=None) -> None:
    """The paired log-ratio loss and its gradient of the logits.

    ``seq_begin`` int64 [2 pairs + 1]: sequence q is rows [seq_begin[q], seq_begin[q + 1]),
    sequences 2i and 2i + 1 the chosen and the rejected answer of pair i.  ``ref_logp``
    float32 [2 pairs]: the reference model's sums over each sequence.  With s the
    sequences' sums (means with ``average``; the reference's sums are then divided
    too) and h = beta ((s_c - ref_c) - (s_r - ref_r)), the loss is the mean over pairs
    of -(1 - label_smoothing) ln sigma(h) - label_smoothing ln sigma(-h).

    Written: ``stats`` float32 [2] (loss, share of pairs with h > 0), ``logp`` float32
    [rows], ``seq_logp`` and ``reward`` = beta (s - ref) float32 [2 pairs], and
    ``dlogits`` as for ``zero_policy_loss``.  ``workspace`` from ``preference_workspace``.
    """
    torch = _torch()
    f32 = torch.float32
    if seq_begin.numel() % 2 != 1 or seq_begin.numel() < 3:
        raise ValueError("seq_begin holds 2 * pairs + 1 boundaries of at least one pair")
    pairs = seq_begin.numel() // 2
    dev, stream, rows, grad = _logits(logits, targets, dlogits)
    a = PreferenceArgs(*rows, _addr(seq_begin, "seq_begin", torch.int64, 2 * pairs + 1, dev), pairs,
                       _addr(ref_logp, "ref_logp", f32, 2 * pairs, dev), beta, label_smoothing, int(average),
                       temperature, grad_scale, _addr(stats, "stats", f32, 2, dev),
                       _addr(logp, "logp", f32, rows[2], dev), _addr(seq_logp, "seq_logp", f32, 2 * pairs, dev),
                       _addr(reward, "reward", f32, 2 * pairs, dev), *grad, *_space(workspace, dev))
    _check(lib().zero_preference_loss(ct.byref(a), stream))


# ---------------------------------------------------------------- convenience
class OwnerShard:
    """One owner's layout, device chunk table and fp32 master/moment state.

    Owner-local arrays start at ``local_base = begin & ~7`` and hold
    ``end - local_base`` elements, so their 128-bit vectors line up with the
    flat buffer's.
    """

    def __init__(self, numels: Sequence[int], ranks: int, owner: int, align: int = 64,
                 max_chunk: int = 2048, device=None):
        torch = _torch()
        sizes = _sizes(numels)  # once: each of the tables below takes the sizes
        self.numels = sizes.tolist()
        self.offsets, self.padded_total, begins, ends = zero_shard_layout(sizes, ranks, align)
        self.ranks, self.owner = ranks, owner
        self.begin, self.end = int(begins[owner]), int(ends[owner])
        self.local_base = self.begin & ~7
        self.local_size = self.end - self.local_base
        self.device = torch.device(_device(device))
        self.align = align
        self.chunks = zero_chunk_table(sizes, self.offsets, self.begin, self.end, max_chunk)
        self.chunks_dev = chunks_to_device(self.chunks, self.device)
        # short chunks packed several to a block, when that saves enough blocks
        self.groups = zero_chunk_groups(self.chunks, max_chunk)
        self.n_groups = self.groups.size - 1
        self.groups_dev = None
        if groups_pay(self.n_groups, self.chunks.size):
            self.groups_dev = torch.from_numpy(self.groups.astype(np.int64)).to(self.device)
        self.n_real = int(self.chunks["len"].sum()) if self.chunks.size else 0
        self.dense_offsets, self.dense_total = zero_dense_offsets(sizes)
        self.tensor_offset_dev = torch.from_numpy(self.offsets.astype(np.int64)).to(self.device)
        self.dense_offset_dev = torch.from_numpy(self.dense_offsets.astype(np.int64)).to(self.device)

    def _group_args(self) -> dict:
        if self.groups_dev is None:
            return {}
        return {"groups_dev": self.groups_dev, "n_groups": self.n_groups}

    def alloc_state(self):
        torch = _torch()
        mk = lambda: torch.zeros(max(8, self.local_size), dtype=torch.float32, device=self.device)
        self.master, self.exp_avg, self.exp_avg_sq = mk(), mk(), mk()
        return self.master, self.exp_avg, self.exp_avg_sq

    def adam_step(self, *, step: int, hyper: dict, rank_grads=None, grad_base: int = 0,
                  divisor: float = 1.0, reduced_g=None, param16=None, param_base: int = 0,
                  clip_coef: float = 1.0, grid_blocks: int = 0) -> None:
        zero_adam_step(chunks_dev=self.chunks_dev, n_chunks=self.chunks.size, begin=self.begin,
                       end=self.end, master=self.master, exp_avg=self.exp_avg,
                       exp_avg_sq=self.exp_avg_sq, local_base=self.local_base, step=step,
                       rank_grads=rank_grads, grad_base=grad_base, divisor=divisor,
                       reduced_g=reduced_g, param16=param16, param_base=param_base,
                       **self._group_args(),
                       clip_coef=clip_coef, grid_blocks=grid_blocks, **hyper)

    def check_buffers(self):
        """(owner-local fp32 gradient, overflow flag int32[1], squared norm
        float64[1], check workspace) used by ``checked_step``, allocated on first
        use and kept.  The flag and the norm share one 16-byte buffer, so one
        copy brings both to the host."""
        torch = _torch()
        if getattr(self, "_check_bufs", None) is None:
            g = torch.zeros(max(8, self.local_size), dtype=torch.float32, device=self.device)
            flag_norm = torch.zeros(16, dtype=torch.uint8, device=self.device)
            ws = check_workspace(max(1, self.end - self.begin), self.device)
            self._flag_norm = flag_norm
            self._check_bufs = (g, flag_norm[0:4].view(torch.int32), flag_norm[8:16].view(torch.float64), ws)
        return self._check_bufs

    def reduce_and_check(self, *, rank_grads, grad_base: int = 0, divisor: float = 1.0, events=None):
        """First half of the checked step: the rank reduce with the fused check into
        the owner-local fp32 gradient, then one 16-byte copy of (overflow flag,
        squared-norm partial) to the host.  Returns that pair for this owner;
        an empty owner returns (0, 0.0) without a launch.  The reduce runs over
        the owner's whole flat range, so the rank buffers hold zeros in the
        padding between tensors (no parameter lives there).  ``divisor`` folds
        in a static loss scale.  ``events``: optional (start, end) CUDA events
        recorded around the reduce launch."""
        if self.end == self.begin:
            return 0, 0.0
        g, ov, ss, ws = self.check_buffers()
        if events is not None:
            events[0].record()
        zero_reduce_owned(rank_grads, self.begin, self.end - self.begin, divisor, g,
                          grad_base=grad_base, out_base=self.local_base, check=(ov, ss, ws))
        if events is not None:
            events[1].record()
        host = self._flag_norm.cpu().numpy()  # waits for the reduce
        return int(host[0:4].view(np.int32)[0]), float(host[8:16].view(np.float64)[0])

    def apply_update(self, *, step: int, hyper: dict, coef: float, param16=None, param_base: int = 0,
                     grid_blocks: int = 0) -> None:
        """Second half: AdamW from the stored reduced gradient scaled by ``coef``
        (nothing to do for an empty owner)."""
        if self.end == self.begin:
            return
        g = self.check_buffers()[0]
        self.adam_step(step=step, hyper=hyper, reduced_g=g, param16=param16, param_base=param_base,
                       clip_coef=coef, grid_blocks=grid_blocks)

    def checked_step(self, *, step: int, hyper: dict, rank_grads, grad_base: int = 0, divisor: float = 1.0,
                     max_norm: float = 1.0, param16=None, param_base: int = 0, grid_blocks: int = 0,
                     events=None, exchange=None, apply_events=None):
        """The two-pass step with an overflow skip and a global-norm clip.

        ``reduce_and_check`` gives this owner's (flag, partial).  The decision
        needs every owner's: ``exchange(flag, partial)`` returns the lists of
        all owners' flags and partials in owner order (across GPUs, an
        all-gather of 12 bytes per owner); without it this owner's pair stands
        for the whole gradient.  ``zero_step_decision`` then skips when any
        flag is set, else gives ``min(1, max_norm / (sqrt(sum of partials) +
        1e-6))``, and ``apply_update`` runs AdamW from the stored gradient.

        Returns ``(updated, clip_coef)``; every owner returns the same pair, and
        the caller advances its step count only when ``updated`` is True.
        ``events`` / ``apply_events``: optional (start, end) CUDA events
        recorded around the reduce and around the AdamW launch.
        """
        flag, sumsq = self.reduce_and_check(rank_grads=rank_grads, grad_base=grad_base, divisor=divisor,
                                            events=events)
        flags, sums = ([flag], [sumsq]) if exchange is None else exchange(flag, sumsq)
        updated, coef = zero_step_decision(flags, sums, max_norm)
        if updated:
            if apply_events is not None:
                apply_events[0].record()
            self.apply_update(step=step, hyper=hyper, coef=coef, param16=param16, param_base=param_base,
                              grid_blocks=grid_blocks)
            if apply_events is not None:
                apply_events[1].record()
        return updated, coef

    # -- export / import of fp32 shard data in the dense per-tensor layout
    def to_dense(self, owner_array, dense) -> None:
        """Write this owner's real elements of an owner-local fp32 array into dense weights."""
        zero_owner_to_dense(self.chunks_dev, self.chunks.size, self.begin, self.end, self.tensor_offset_dev,
                            self.dense_offset_dev, owner_array, self.local_base, dense, **self._group_args())

    def from_dense(self, dense, owner_array) -> None:
        """Fill this owner's real elements of an owner-local fp32 array from dense weights."""
        zero_dense_to_owner(self.chunks_dev, self.chunks.size, self.begin, self.end, self.tensor_offset_dev,
                            self.dense_offset_dev, dense, owner_array, self.local_base, **self._group_args())

    # -- checkpoint of the owner's optimizer state
    def save(self, path: str, step: int) -> None:
        """Owner checkpoint: fp32 master, both moments, the step count and the layout."""
        np.savez(path, master=self.master.cpu().numpy(), exp_avg=self.exp_avg.cpu().numpy(),
                 exp_avg_sq=self.exp_avg_sq.cpu().numpy(), step=np.int64(step),
                 numels=np.array(self.numels, dtype=np.int64), ranks=np.int64(self.ranks),
                 owner=np.int64(self.owner), align=np.int64(self.align))

    def load(self, path: str) -> int:
        """Restore a checkpoint written by save() for the same layout; returns its step."""
        torch = _torch()
        with np.load(path, allow_pickle=False) as z:
            same = ("exp_avg" in z.files and list(z["numels"]) == self.numels and int(z["ranks"]) == self.ranks
                    and int(z["owner"]) == self.owner and int(z["align"]) == self.align)
            if not same:
                raise ValueError("checkpoint was written for a different layout, owner or state width")
            self.master = torch.from_numpy(z["master"]).to(self.device)
            self.exp_avg = torch.from_numpy(z["exp_avg"]).to(self.device)
            self.exp_avg_sq = torch.from_numpy(z["exp_avg_sq"]).to(self.device)
            return int(z["step"])


class OwnerShard8(OwnerShard):
    """An owner whose two moments are held in 8 bits (2.0625 bytes per parameter, not 8).

    The same calls as ``OwnerShard``; the state is ``master`` (fp32), ``exp_avg8`` and
    ``exp_rms8`` (float8_e4m3fn codes of the first moment and of the root of the
    second) and ``exp_avg_scale`` / ``exp_rms_scale`` (fp32, one per ZERO_QBLOCK flat
    elements).  Owner-local arrays start at ``local_base = begin`` rounded down to a
    multiple of ZERO_QBLOCK.
    """

    def __init__(self, numels: Sequence[int], ranks: int, owner: int, align: int = 64,
                 max_chunk: int = 2048, device=None):
        sizes = _sizes(numels)
        super().__init__(sizes, ranks, owner, align, max_chunk, device)
        torch = _torch()
        self.local_base = self.begin // ZERO_QBLOCK * ZERO_QBLOCK
        self.local_size = self.end - self.local_base
        self.blocks = -(-self.local_size // ZERO_QBLOCK)
        self.pieces, masks = zero_piece_table(sizes, self.offsets, self.begin, self.end)
        self.pieces_dev = chunks_to_device(self.pieces, self.device)
        self.masks_dev = torch.from_numpy(masks).to(self.device) if masks.size else None

    def alloc_state(self):
        """master, then the moments: (codes, scales) of the first and of the second's root."""
        torch = _torch()
        n = max(1, self.blocks)
        mk = lambda k, dt: torch.zeros(k, dtype=dt, device=self.device)
        self.master = mk(n * ZERO_QBLOCK, torch.float32)
        self.exp_avg8, self.exp_rms8 = (mk(n * ZERO_QBLOCK, torch.float8_e4m3fn) for _ in range(2))
        self.exp_avg_scale, self.exp_rms_scale = mk(n, torch.float32), mk(n, torch.float32)
        return self.master, (self.exp_avg8, self.exp_avg_scale), (self.exp_rms8, self.exp_rms_scale)

    def _state8(self) -> dict:
        """The piece table and 8-bit state as keyword arguments of the module's calls."""
        return dict(pieces_dev=self.pieces_dev, n_pieces=self.pieces.size, masks_dev=self.masks_dev, begin=self.begin,
                    end=self.end, local_base=self.local_base, exp_avg8=self.exp_avg8,
                    exp_avg_scale=self.exp_avg_scale, exp_rms8=self.exp_rms8, exp_rms_scale=self.exp_rms_scale)

    def _checked(self):
        """(device, stream, piece table, 8-bit state) of a call."""
        dev, stream = _device_stream()
        return (dev, stream,
                _pieces8(dev, self.pieces_dev, self.pieces.size, self.masks_dev, self.begin, self.end),
                _state8(dev, self.end, self.local_base, self.exp_avg8, self.exp_avg_scale, self.exp_rms8,
                        self.exp_rms_scale))

    def adam_step(self, *, step: int, hyper: dict, rank_grads=None, grad_base: int = 0,
                  divisor: float = 1.0, reduced_g=None, param16=None, param_base: int = 0,
                  clip_coef: float = 1.0, grid_blocks: int = 0) -> None:
        """``grid_blocks`` is accepted for ``OwnerShard``'s callers; this step has one launch shape."""
        _adam8(*self._checked(), self.local_base, self.master, _hyper(**hyper), step, rank_grads, grad_base, divisor,
               reduced_g, param16, param_base, clip_coef)

    def pack_moments(self, exp_avg, exp_avg_sq) -> None:
        """Take over fp32 moments (owner-local, from ``local_base``)."""
        _moments8(True, *self._checked(), self.local_base, exp_avg, exp_avg_sq)

    def unpack_moments(self, exp_avg, exp_avg_sq) -> None:
        """Write the moments as fp32 (for ``to_dense``, or to go on in 32 bits)."""
        _moments8(False, *self._checked(), self.local_base, exp_avg, exp_avg_sq)

    _SAVED = ("master", "exp_avg8", "exp_avg_scale", "exp_rms8", "exp_rms_scale")

    def save(self, path: str, step: int) -> None:
        """Owner checkpoint: fp32 master, the codes (as bytes) and scales, the step count and the layout."""
        torch = _torch()
        host = lambda t: (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t).cpu().numpy()
        np.savez(path, **{k: host(getattr(self, k)) for k in self._SAVED}, step=np.int64(step),
                 numels=np.array(self.numels, dtype=np.int64), ranks=np.int64(self.ranks),
                 owner=np.int64(self.owner), align=np.int64(self.align))

    def load(self, path: str) -> int:
        """Restore a checkpoint written by save() for the same layout; returns its step."""
        torch = _torch()
        with np.load(path, allow_pickle=False) as z:
            same = ("exp_avg8" in z.files and list(z["numels"]) == self.numels and int(z["ranks"]) == self.ranks
                    and int(z["owner"]) == self.owner and int(z["align"]) == self.align)
            if not same:
                raise ValueError("checkpoint was written for a different layout, owner or state width")
            for k in self._SAVED:
                t = torch.from_numpy(z[k]).to(self.device)
                setattr(self, k, t.view(torch.float8_e4m3fn) if k.endswith("8") else t)
            return int(z["step"])
