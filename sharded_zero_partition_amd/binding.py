"""Python binding of libzero_partition.so: one rank's ZeRO-DP shard step on
MI355X (gfx950).

Argument marshalling only: every step of the path (layout, bucket pack,
reduce, overflow check, Adam, fp16 cast) runs in the C++/HIP library.  torch
provides device memory and the stream.  Importing this package fails loudly
when the library has not been built (`python -m sharded_zero_partition_amd.build`).

Names follow the C ABI in include/zero_partition.h:
  partition_layout(...)   -> Layout   (zero_partition_layout and accessors)
  Layout.arena_plan(...)               (zero_arena_plan_for); carve_arena(plan)
  Layout.bind_tensors(...)             (zero_layout_bind_tensors)
  Layout.pack_bucket(...)              (zero_pack_bucket)
  Layout.bind_contributions(...)       (zero_layout_bind_contributions)
  Layout.reduce_to_owner(...)          (zero_reduce_to_owner)
  shard_step(...), PreparedStep(...)   (zero_shard_step; zero_shard_step_noalloc with noalloc=True)
  Layout.owner_step(...)               (zero_owner_step)
  TensorSet(...)                       (zero_tensor_set_create, zero_tensor_set_m_rounding)
  TensorSet.bind_grads(...)            (zero_tensor_set_bind_grads)
  TensorSet.grad_sumsq(...)            (zero_grad_sumsq)
  StepControl(...), StepControl.begin(...)   (zero_step_control, zero_step_begin)
  TensorSet.adamw_step(...)            (zero_adamw_step)
  TensorSet.states_from(...)           (zero_states_convert)
  Checkpoint(...), .store, .load       (zero_checkpoint, zero_checkpoint_store, zero_checkpoint_load)
  activation(...), activation_grad(...)   (zero_activation, zero_activation_grad)
  weight_grad(...)                     (zero_weight_grad)
  embedding_lookup(...), embedding_grad(...)   (zero_embedding_lookup, zero_embedding_grad)
  set_kernel_timing, last_kernel_ms, kernel_times   (kernel timing)
"""

import ctypes
import math
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero_partition.so")

ZERO_OK = 0
STATUS_NAMES = {
    -1: "INVALID_ARG", -2: "ALIGNMENT", -3: "CAPACITY", -4: "INDEX_OVERFLOW",
    -5: "HIP", -6: "OUT_OF_MEMORY", -7: "STATE",
}


class ZeroError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


# ---------------------------------------------------------------------------
# ABI structs (mirror include/zero_partition.h)
# ---------------------------------------------------------------------------

class LayoutInfo(ctypes.Structure):
    _fields_ = [("psi", ctypes.c_int64), ("shard_elems", ctypes.c_int64),
                ("padded_elems", ctypes.c_int64), ("padding", ctypes.c_int64),
                ("n_tensors", ctypes.c_int64), ("align_elems", ctypes.c_int64),
                ("bucket_elems", ctypes.c_int64), ("n_fills", ctypes.c_int64),
                ("n_segments", ctypes.c_int64), ("n_ranks", ctypes.c_int32),
                ("stage", ctypes.c_int32), ("bytes_param16", ctypes.c_int64),
                ("bytes_grad16", ctypes.c_int64), ("bytes_master", ctypes.c_int64),
                ("bytes_momentum", ctypes.c_int64), ("bytes_variance", ctypes.c_int64),
                ("bytes_total", ctypes.c_int64)]


class Segment(ctypes.Structure):
    _fields_ = [("tensor", ctypes.c_int32), ("owner", ctypes.c_int32),
                ("tensor_off", ctypes.c_int64), ("flat_off", ctypes.c_int64),
                ("len", ctypes.c_int64), ("shard_off", ctypes.c_int64),
                ("fill", ctypes.c_int64), ("bucket_off", ctypes.c_int64)]

    def as_tuple(self):
        return (self.tensor, self.owner, self.tensor_off, self.flat_off, self.len,
                self.shard_off, self.fill, self.bucket_off)


class ShardStateC(ctypes.Structure):
    _fields_ = [("shard_elems", ctypes.c_int64), ("p", ctypes.c_void_p * 2),
                ("m", ctypes.c_void_p * 2), ("v", ctypes.c_void_p * 2),
                ("cur", ctypes.c_int32), ("reserved", ctypes.c_int32), ("t", ctypes.c_int64)]


class AdamHParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class LossScaler(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("backoff", ctypes.c_float),
                ("growth", ctypes.c_float), ("min_scale", ctypes.c_float),
                ("growth_interval", ctypes.c_int32), ("good_steps", ctypes.c_int32)]

    @classmethod
    def make(cls, scale=1024.0, backoff=0.5, growth=2.0, min_scale=1.0,
             growth_interval=1000, good_steps=0):
        return cls(scale, backoff, growth, min_scale, growth_interval, good_steps)


ARENA_KINDS = (["param16", "grad16", "master", "momentum", "variance", "master_alt",
                "momentum_alt", "variance_alt", "bucket"] + [f"contrib{r}" for r in range(16)])


class ArenaPlan(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_int64), ("align_bytes", ctypes.c_int64),
                ("offset", ctypes.c_int64 * 25), ("bytes", ctypes.c_int64 * 25)]

    def as_dict(self):
        return {k: (self.offset[i], self.bytes[i]) for i, k in enumerate(ARENA_KINDS)
                if self.offset[i] >= 0}


MAX_GROUPS = 16
STATE_BLOCK = 32
DTYPE_NONE, DTYPE_FP16, DTYPE_BF16, DTYPE_FP32, DTYPE_MXFP8 = range(5)


class TensorC(ctypes.Structure):
    _fields_ = [("numel", ctypes.c_int64), ("p", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("group", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class StepControlC(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int64), ("skipped", ctypes.c_int64), ("sumsq", ctypes.c_double),
                ("scale", ctypes.c_float), ("lr_mult", ctypes.c_float),
                ("good_steps", ctypes.c_int32), ("skip", ctypes.c_int32),
                ("norm", ctypes.c_float), ("grad_mult", ctypes.c_float),
                ("group", (ctypes.c_float * 8) * MAX_GROUPS)]


class MatrixC(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("stride", ctypes.c_int64), ("type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class CheckpointC(ctypes.Structure):
    _fields_ = [("code", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


ABI_STRUCTS = [LayoutInfo, Segment, ShardStateC, AdamHParams, LossScaler, ArenaPlan, TensorC,
               StepControlC, MatrixC, CheckpointC]

# exported symbol -> (restype, argtypes)
_P = ctypes.c_void_p
_I32, _I64 = ctypes.c_int32, ctypes.c_int64
SIGNATURES = {
    "zero_partition_layout": (ctypes.c_int, [_P, _I64, _I32, _I32, _I64, _I64, _P]),
    "zero_layout_destroy": (ctypes.c_int, [_P]),
    "zero_layout_get_info": (ctypes.c_int, [_P, _P]),
    "zero_layout_tensor_offsets": (ctypes.c_int, [_P, _P, _I64]),
    "zero_layout_rank_range": (ctypes.c_int, [_P, _I32, _P, _P, _P]),
    "zero_layout_segments": (ctypes.c_int, [_P, _P, _I64, _P]),
    "zero_layout_rank_segments": (ctypes.c_int, [_P, _I32, _P, _I64, _P]),
    "zero_layout_fill_segments": (ctypes.c_int, [_P, _I64, _P, _I64, _P]),
    "zero_arena_plan_for": (ctypes.c_int, [_P, _I32, _I32, _I32, _I64, _P]),
    "zero_layout_bind_tensors": (ctypes.c_int, [_P, _P, _P]),
    "zero_pack_bucket": (ctypes.c_int, [_P, _I64, _P, _P, _P]),
    "zero_layout_bind_contributions": (ctypes.c_int, [_P, _I32, _P, _P]),
    "zero_reduce_to_owner": (ctypes.c_int, [_P, _I64, _I32, _P, _P, _P]),
    "zero_shard_step": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P]),
    "zero_shard_step_noalloc": (ctypes.c_int, [_P, _P, _I32, _P, _P, _P, _P, _P]),
    "zero_owner_step": (ctypes.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P]),
    "zero_tensor_set_create": (ctypes.c_int, [_P, _I64, _I32, _I32, _I32, ctypes.c_uint32, _P, _P]),
    "zero_tensor_set_destroy": (ctypes.c_int, [_P]),
    "zero_tensor_set_m_rounding": (ctypes.c_int, [_P, _I32]),
    "zero_tensor_set_bind_grads": (ctypes.c_int, [_P, _P, _P]),
    "zero_grad_sumsq_work_bytes": (ctypes.c_int64, [_P]),
    "zero_grad_sumsq": (ctypes.c_int, [_P, _P, _I32, _P, _P]),
    "zero_step_begin": (ctypes.c_int, [_P, _P, _I32, ctypes.c_float, _I32, _P, _P]),
    "zero_adamw_step": (ctypes.c_int, [_P, _P, _I32, _P]),
    "zero_states_convert": (ctypes.c_int, [_P, _P, _P]),
    "zero_checkpoint_bytes": (ctypes.c_int, [_I64, _I64, _P, _P]),
    "zero_checkpoint_store": (ctypes.c_int, [_P, _P, _P]),
    "zero_checkpoint_load": (ctypes.c_int, [_P, _P, _P]),
    "zero_activation": (ctypes.c_int, [_I32, _P, _P, _P, _P, _P, _P, _P]),
    "zero_activation_grad": (ctypes.c_int, [_I32, _P, _P, _P, _P, _P, _P]),
    "zero_weight_grad_work_bytes": (ctypes.c_int64, [_I64, _I64, _I64, _I32]),
    "zero_weight_grad": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _P, _P]),
    "zero_embedding_lookup": (ctypes.c_int, [_P, _P, _I32, _I64, ctypes.c_float, _P, _P]),
    "zero_embedding_grad_work_bytes": (ctypes.c_int64, [_I64, _I64, _I64]),
    "zero_embedding_grad": (ctypes.c_int, [_P, _P, _I32, _I64, ctypes.c_float, _P, _I32, _P, _P]),
    "zero_set_kernel_timing": (ctypes.c_int, [_I32]),
    "zero_last_kernel_ms": (ctypes.c_int, [_P]),
    "zero_kernel_times": (ctypes.c_int, [_P, _I64, _P]),
    "zero_version": (ctypes.c_int, []),
    "zero_last_error": (ctypes.c_char_p, []),
    "zero_last_hip_error": (ctypes.c_int, []),
    "zero_abi_struct_size": (ctypes.c_int64, [_I32]),
    "zero_device_info": (ctypes.c_int, [_P, _P]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m sharded_zero_partition_amd.build` "
            "(hipcc, gfx950). There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    for i, s in enumerate(ABI_STRUCTS):
        got = lib.zero_abi_struct_size(i)
        if got != ctypes.sizeof(s):
            raise ImportError(f"ABI mismatch for {s.__name__}: library {got}, binding {ctypes.sizeof(s)}")
    return lib


# torch brings its own copy of the HIP runtime (same soname).  Importing torch
# first makes this library bind to that copy, so one runtime serves both;
# loaded the other way round, a process would hold two runtimes, and the
# second one initialised can find no device.
import numpy as np  # noqa: E402
import torch  # noqa: E402,F401

lib = _load()


def _check(rc: int):
    if rc != ZERO_OK:
        raise ZeroError(rc, lib.zero_last_error().decode(errors="replace"))


def _ref(x):
    return ctypes.byref(x)


def _stream_ptr(stream) -> Optional[int]:
    """hipStream_t of a torch stream (None -> torch's current stream)."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _current_device() -> int:
    import torch
    return torch.cuda.current_device()


def _dev_ptr(t, what: str, dtype_bytes: int, dev: int = None):
    """Device address of a contiguous tensor on the current device (`dev`,
    when the caller already knows it)."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")
    if dev is None:
        dev = _current_device()
    if t.device.index != dev:
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.element_size() != dtype_bytes:
        raise ValueError(f"{what}: expected {dtype_bytes}-byte elements")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# layout and pack
# ---------------------------------------------------------------------------

class Layout:
    """Owner of a zero_layout handle."""

    def __init__(self, numels: Sequence[int], n_ranks: int, stage: int = 2,
                 align: int = 1, bucket: int = 0):
        arr = (ctypes.c_int64 * len(numels))(*[int(n) for n in numels])
        h = ctypes.c_void_p()
        _check(lib.zero_partition_layout(arr, len(numels), int(n_ranks), int(stage),
                                         int(align), int(bucket), _ref(h)))
        self._h = h
        self._bound = None
        self._numels = [int(n) for n in numels]
        info = self.info            # fixed for the handle's life
        self._bucket_elems = info.bucket_elems
        self._shard_elems = info.shard_elems

    def close(self):
        if self._h:
            lib.zero_layout_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def info(self) -> LayoutInfo:
        out = LayoutInfo()
        _check(lib.zero_layout_get_info(self._h, _ref(out)))
        return out

    def tensor_offsets(self) -> List[int]:
        n = self.info.n_tensors
        arr = (ctypes.c_int64 * max(1, n))()
        _check(lib.zero_layout_tensor_offsets(self._h, arr, n))
        return list(arr[:n])

    def rank_range(self, rank: int):
        b, re, e = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(lib.zero_layout_rank_range(self._h, int(rank), _ref(b), _ref(re), _ref(e)))
        return b.value, re.value, e.value

    def _query(self, fn, *key) -> List[Segment]:
        n = ctypes.c_int64()
        rc = fn(self._h, *key, None, 0, _ref(n))
        if rc not in (ZERO_OK, -3):
            _check(rc)
        arr = (Segment * max(1, n.value))()
        _check(fn(self._h, *key, arr, n.value, _ref(n)))
        return list(arr[:n.value])

    def segments(self) -> List[Segment]:
        return self._query(lib.zero_layout_segments)

    def rank_segments(self, rank: int) -> List[Segment]:
        return self._query(lib.zero_layout_rank_segments, int(rank))

    def fill_segments(self, fill: int) -> List[Segment]:
        return self._query(lib.zero_layout_fill_segments, int(fill))

    def arena_plan(self, pingpong: bool = False, n_contrib: int = 0, with_bucket: bool = False,
                   align_bytes: int = 0) -> ArenaPlan:
        """zero_arena_plan_for: one rank's buffers in one contiguous block."""
        out = ArenaPlan()
        _check(lib.zero_arena_plan_for(self._h, int(bool(pingpong)), int(n_contrib),
                                       int(bool(with_bucket)), int(align_bytes), _ref(out)))
        return out

    def _check_list(self, tensors, what: str):
        """The library reads numel[i] elements from tensor i: the list must
        match the layout's tensor count and sizes exactly."""
        if len(tensors) != len(self._numels):
            raise ValueError(f"{what} has {len(tensors)} tensors, the layout {len(self._numels)}")
        for i, (t, n) in enumerate(zip(tensors, self._numels)):
            if t.numel() != n:
                raise ValueError(f"{what}: tensor {i} has {t.numel()} elements, the layout {n}")

    def bind_tensors(self, tensors, stream=None):
        """Bind the device fp16 tensors (any 2-byte dtype, contiguous) in
        list order; they must stay alive while packing."""
        self._check_list(tensors, "tensor list")
        ptrs = (ctypes.c_void_p * max(1, len(tensors)))()
        for i, t in enumerate(tensors):
            ptrs[i] = _dev_ptr(t, f"tensor {i}", 2) if t.numel() > 0 else None
        _check(lib.zero_layout_bind_tensors(self._h, ptrs, _stream_ptr(stream)))
        self._bound = list(tensors)

    def pack_bucket(self, fill: int, bucket, stream=None) -> int:
        """Write fill `fill` into the device bucket (B two-byte elements)."""
        if bucket.numel() != self._bucket_elems:
            raise ValueError("bucket must hold bucket_elems elements")
        n = ctypes.c_int64()
        _check(lib.zero_pack_bucket(self._h, int(fill), ctypes.c_void_p(_dev_ptr(bucket, "bucket", 2)),
                                    _stream_ptr(stream), _ref(n)))
        return n.value

    def bind_contributions(self, lists, stream=None):
        """Bind R lists of device fp16 tensors (one list per reducing rank, in
        the layout's tensor order) for reduce_to_owner."""
        R = len(lists)
        nt = len(self._numels)
        ptrs = (ctypes.c_void_p * max(1, R * nt))()
        for r, lst in enumerate(lists):
            self._check_list(lst, f"list {r}")
            for i, t in enumerate(lst):
                ptrs[r * nt + i] = _dev_ptr(t, f"tensor {r}/{i}", 2) if t.numel() > 0 else None
        _check(lib.zero_layout_bind_contributions(self._h, R, ptrs, _stream_ptr(stream)))
        self._contrib = [list(lst) for lst in lists]

    def reduce_to_owner(self, fill: int, rank: int, shard, stream=None) -> int:
        """Write rank `rank`'s share of fill `fill` of the reduce into its fp16
        gradient shard (S two-byte elements); returns the elements written."""
        if shard.numel() != self._shard_elems:
            raise ValueError("shard must hold shard_elems elements")
        n = ctypes.c_int64()
        _check(lib.zero_reduce_to_owner(self._h, int(fill), int(rank),
                                        ctypes.c_void_p(_dev_ptr(shard, "shard", 2)),
                                        _stream_ptr(stream), _ref(n)))
        return n.value


    def owner_step(self, rank: int, state: "ShardState", hparams: "AdamHParams",
                   scaler: "LossScaler", out_slot, stream=None) -> int:
        """zero_owner_step: rank `rank`'s ping-pong shard step with the sum
        taken straight from the bound contribution lists.  Returns the
        overflow flag; updates state.t, state.cur and the scaler in place."""
        S = self._shard_elems
        if not state.pingpong:
            raise ValueError("the owner step needs ping-pong state (p_alt, m_alt, v_alt)")
        if state.shard_elems != S:
            raise ValueError(f"state holds {state.shard_elems} elements, the layout's shard {S}")
        if out_slot.numel() != S:
            raise ValueError(f"out_slot has {out_slot.numel()} elements, expected {S}")
        dev = _current_device()
        c = state._to_c(dev)
        flag = ctypes.c_int32()
        slot = ctypes.c_void_p(_dev_ptr(out_slot, "out_slot", 2, dev) if S else None)
        _check(lib.zero_owner_step(self._h, int(rank), _ref(c), _ref(hparams), _ref(scaler), slot,
                                   _stream_ptr(stream), _ref(flag)))
        state.t = c.t
        state.cur = c.cur
        return flag.value


def partition_layout(numels: Sequence[int], n_ranks: int, stage: int = 2, align: int = 1,
                     bucket: int = 0) -> Layout:
    return Layout(numels, n_ranks, stage, align, bucket)


# ---------------------------------------------------------------------------
# shard step
# ---------------------------------------------------------------------------

@dataclass
class ShardState:
    """One rank's fp32 shard state on the device.  With p_alt/m_alt/v_alt the
    step runs single-pass ping-pong and `cur` names the live set."""
    p: object
    m: object
    v: object
    p_alt: object = None
    m_alt: object = None
    v_alt: object = None
    cur: int = 0
    t: int = 0

    @property
    def shard_elems(self) -> int:
        return self.p.numel()

    @property
    def pingpong(self) -> bool:
        return self.p_alt is not None

    def live(self):
        """(p, m, v) of the live set."""
        if self.cur == 0:
            return self.p, self.m, self.v
        return self.p_alt, self.m_alt, self.v_alt

    def _to_c(self, dev: int) -> ShardStateC:
        c = ShardStateC()
        c.shard_elems = self.shard_elems
        sets = [(self.p, self.m, self.v)]
        if self.pingpong:
            sets.append((self.p_alt, self.m_alt, self.v_alt))
        for k, (p, m, v) in enumerate(sets):
            for name, t in (("p", p), ("m", m), ("v", v)):
                if t.numel() != self.shard_elems:
                    raise ValueError(f"{name}[{k}] has {t.numel()} elements, expected {self.shard_elems}")
                getattr(c, name)[k] = _dev_ptr(t, f"{name}[{k}]", 4, dev) if t.numel() else None
        c.cur = self.cur
        c.t = self.t
        return c


def shard_step(state: ShardState, grads, hparams: AdamHParams, scaler: LossScaler, out_slot,
               stream=None, noalloc: bool = False) -> int:
    """zero_shard_step (zero_shard_step_noalloc with noalloc=True): returns
    the overflow flag; updates state.t, state.cur and the scaler in place."""
    R = len(grads)
    S = state.shard_elems
    dev = _current_device()
    ptrs = (ctypes.c_void_p * max(1, R))()
    for r, g in enumerate(grads):
        if g.numel() != S:
            raise ValueError(f"grads[{r}] has {g.numel()} elements, expected {S}")
        ptrs[r] = _dev_ptr(g, f"grads[{r}]", 2, dev) if S else None
    if out_slot.numel() != S:
        raise ValueError(f"out_slot has {out_slot.numel()} elements, expected {S}")
    c = state._to_c(dev)
    flag = ctypes.c_int32()
    slot = ctypes.c_void_p(_dev_ptr(out_slot, "out_slot", 2, dev) if S else None)
    fn = lib.zero_shard_step_noalloc if noalloc else lib.zero_shard_step
    _check(fn(_ref(c), ptrs, R, _ref(hparams), _ref(scaler), slot, _stream_ptr(stream), _ref(flag)))
    state.t = c.t
    state.cur = c.cur
    return flag.value


class PreparedStep:
    """zero_shard_step with its arguments checked and marshalled once, for
    loops that step the same tensors again and again.

    The object keeps references to the tensors; their storage must not be
    moved or resized while it is in use.  The stream is the one given (or
    torch's current stream) at preparation.  Every call writes state.cur and
    state.t into the C state first and reads them back after, updates the
    scaler in place and returns the overflow flag, like shard_step."""

    def __init__(self, state: ShardState, grads, hparams: AdamHParams, scaler: LossScaler,
                 out_slot, stream=None):
        R = len(grads)
        S = state.shard_elems
        self._dev = _current_device()
        self._ptrs = (ctypes.c_void_p * max(1, R))()
        for r, g in enumerate(grads):
            if g.numel() != S:
                raise ValueError(f"grads[{r}] has {g.numel()} elements, expected {S}")
            self._ptrs[r] = _dev_ptr(g, f"grads[{r}]", 2, self._dev) if S else None
        if out_slot.numel() != S:
            raise ValueError(f"out_slot has {out_slot.numel()} elements, expected {S}")
        self._c = state._to_c(self._dev)
        self._flag = ctypes.c_int32()
        slot = ctypes.c_void_p(_dev_ptr(out_slot, "out_slot", 2, self._dev) if S else None)
        self._args = (_ref(self._c), self._ptrs, R, _ref(hparams), _ref(scaler), slot,
                      _stream_ptr(stream), _ref(self._flag))
        self._state = state
        self._keep = (list(grads), hparams, scaler, out_slot)

    def __call__(self) -> int:
        if _current_device() != self._dev:
            raise ValueError(f"prepared on cuda:{self._dev}, the current device is another")
        st, c = self._state, self._c
        c.cur = st.cur
        c.t = st.t
        _check(lib.zero_shard_step(*self._args))
        st.t = c.t
        st.cur = c.cur
        return self._flag.value


# ---------------------------------------------------------------------------
# tensor sets: AdamW over many tensors at once
# ---------------------------------------------------------------------------

class StepControl:
    """An optimizer's step state on the device (a zero_step_control): step
    count, loss scale and the decision of the step at hand.  The attributes are
    0-dim tensors on its memory: reading one on the host waits for the device;
    writing (`control.lr_mult.fill_(0.5)`) is ordered like any other work.

      t, skipped      steps taken and skipped (int64)
      sumsq           sum of squares of the gradients (float64): where
                      TensorSet.grad_sumsq puts it, and what ranks all-reduce
      scale, lr_mult  loss scale of the next gradients, factor on every lr
      good_steps      taken steps since the scale last changed (int32)
      skip, norm, grad_mult   of the begun step: 1 when it is skipped, the
                      global norm, what gradients are multiplied by
    """

    def __init__(self, scale: float = 1.0, t: int = 0, lr_mult: float = 1.0, device=None):
        c = StepControlC()
        c.t, c.scale, c.lr_mult = int(t), float(scale), float(lr_mult)
        if c.t < 0:
            raise ValueError("t must not be negative")
        if not (c.scale >= 2.0 ** -24 and c.scale < float("inf")):
            raise ValueError("scale must be finite and at least 2^-24")
        dev = torch.device("cuda", _current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError("the control block lives on a device")
        self.buffer = torch.frombuffer(bytearray(c), dtype=torch.uint8).to(dev)
        self.device_index = self.buffer.device.index
        self._ptr = self.buffer.data_ptr()
        for name, dtype in (("t", torch.int64), ("skipped", torch.int64), ("sumsq", torch.float64),
                            ("scale", torch.float32), ("lr_mult", torch.float32),
                            ("good_steps", torch.int32), ("skip", torch.int32),
                            ("norm", torch.float32), ("grad_mult", torch.float32)):
            f = getattr(StepControlC, name)
            setattr(self, name, self.buffer[f.offset:f.offset + f.size].view(dtype)[0])
        self._groups = None
        self._n_groups = 0

    def begin(self, groups, max_norm: float = 0.0, check: bool = True, scaler: "LossScaler" = None,
              stream=None):
        """zero_step_begin: decide the step from `sumsq` (check=False: take it
        unseen) with clipping to `max_norm` (0: none), and set the constants of
        `groups` (AdamHParams, one for each parameter group).  `scaler` gives
        the rule of a dynamic loss scale; its own scale is not used."""
        _on_current_device(self.device_index, "the control block")
        if max_norm and not ctypes.c_float(max_norm).value:
            raise ValueError("max_norm is below fp32's range (0 means no clipping)")
        n = len(groups)
        arr = (AdamHParams * max(1, n))(*groups)
        _check(lib.zero_step_begin(self._ptr, arr, n, max_norm, bool(check),
                                   None if scaler is None else _ref(scaler),
                                   _raw_stream(stream, self.device_index)))
        self._n_groups = n


def _raw_stream(stream, dev: int):
    """hipStream_t of a torch stream (None -> the device's current stream), as a
    number: looking the current one up this way takes a fortieth of the time
    that making a Stream object does."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _on_current_device(index: int, what: str):
    if index != _current_device():
        raise ValueError(f"{what} is on cuda:{index}, the current device is another")


def _dtype_of(tensors, what: str, kinds) -> int:
    """The one dtype of a list of tensors, as a ZERO_DTYPE number."""
    seen = {t.dtype for t in tensors}
    if len(seen) > 1:
        raise ValueError(f"{what}: the tensors have different dtypes")
    for d in seen:
        if d not in kinds:
            raise ValueError(f"{what}: dtype {d} is not supported")
        return kinds[d]
    return DTYPE_NONE


def _addresses(tensors, what: str, sizes, dev: int) -> list:
    """Device addresses of contiguous tensors of the given sizes on device `dev`.
    Lists run to tens of thousands: the checks pass over them whole, and only a
    failed one looks for its tensor."""
    if len(tensors) != len(sizes):
        raise ValueError(f"{what} has {len(tensors)} tensors, the set {len(sizes)}")
    for bad, why in (([t.get_device() != dev for t in tensors], f"is not on cuda:{dev}, the current device"),
                     ([not t.is_contiguous() for t in tensors], "must be contiguous"),
                     ([t.numel() != n for t, n in zip(tensors, sizes)], "has another size than the set's tensor needs")):
        if any(bad):
            raise ValueError(f"{what}[{bad.index(True)}] {why}")
    return [t.data_ptr() for t in tensors]


_BITS16 = {torch.float16: DTYPE_FP16, torch.int16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16}
_GRAD_DTYPES = {**_BITS16, torch.float32: DTYPE_FP32}
_SCALE_DTYPES = {torch.uint8: DTYPE_MXFP8, torch.float8_e8m0fnu: DTYPE_MXFP8}
_STATE_DTYPES = {torch.float32: DTYPE_FP32, torch.uint8: DTYPE_MXFP8, torch.float8_e4m3fn: DTYPE_MXFP8}


class TensorSet:
    """Owner of a zero_tensor_set: lists of device tensors, contiguous and of
    any size, one entry for each parameter (or each piece of one that a rank's
    shard holds, Layout.rank_segments).  A call writes p, out and states as an
    in-place operation does: autograd's version counters of p and out are raised
    (of m and v by a conversion), but not by a graph's replays.

      p        fp32 master values
      grads    fp16 (or int16 bit patterns), bf16 or fp32
      m, v     fp32 states, or e4m3 codes (float8_e4m3fn or uint8) with
               m_scale, v_scale: a scale byte for each 32 elements (uint8 or
               float8_e8m0fnu).  All zeros is the state to start from.
      out      fp16 (or int16) or bf16 copies that a step writes
      groups   each tensor's parameter group (default 0)
      seed     of the random rounding of 8-bit states
      m_rounding   of an 8-bit m: "auto" (to nearest up to beta1 = 0.9444, at
               random above, where to nearest it would not decay) or "random"
               (keeps the mean of m at any beta1: to nearest, under a steady
               gradient, m stops at 0.62 to 0.8 of it for beta1 = 0.9)
      grad_dtype   of gradients that bind_grads will bring, when grads is not given

    Lists that an operator does not need may be left out: grad_sumsq needs
    grads, adamw_step p, grads, m and v, states_from m and v.  The tensors'
    storage must not be moved or resized while the set is in use, and a graph
    that captured one of its calls needs the set as long as it is replayed."""

    def __init__(self, p=None, grads=None, m=None, v=None, m_scale=None, v_scale=None, out=None,
                 groups=None, seed: int = 0, grad_dtype=None, stream=None, m_rounding: str = "auto"):
        self._h = None
        if m_rounding not in ("auto", "random"):
            raise ValueError("m_rounding must be 'auto' or 'random'")
        lists = dict(p=p, grad=grads, m=m, v=v, m_scale=m_scale, v_scale=v_scale, out=out)
        lists = {k: list(x) for k, x in lists.items() if x is not None}
        if not lists:
            raise ValueError("a tensor set needs tensors")
        if ("m" in lists) != ("v" in lists):
            raise ValueError("m and v come together")
        self._numels = [t.numel() for t in lists.get("m", next(iter(lists.values())))]
        n = len(self._numels)
        self._dev = _current_device()
        self._grad_type = _dtype_of(lists.get("grad", []), "grads", _GRAD_DTYPES)
        if "grad" not in lists and grad_dtype is not None:
            if grad_dtype not in _GRAD_DTYPES:
                raise ValueError(f"grad_dtype {grad_dtype} is not supported")
            self._grad_type = _GRAD_DTYPES[grad_dtype]
        state_type = _dtype_of(lists.get("m", []), "m", _STATE_DTYPES)
        if state_type != _dtype_of(lists.get("v", []), "v", _STATE_DTYPES):
            raise ValueError("m and v have different dtypes")
        out_type = _dtype_of(lists.get("out", []), "out", _BITS16)
        _dtype_of(lists.get("p", []), "p", {torch.float32: DTYPE_FP32})
        mx = state_type == DTYPE_MXFP8
        if m_rounding != "auto" and not mx:
            raise ValueError("m_rounding is of states in 8 bits")
        if ("m_scale" in lists, "v_scale" in lists) != (mx, mx):
            raise ValueError("m_scale and v_scale come with states in 8 bits, and only with them")
        if groups is not None and len(groups) != n:
            raise ValueError(f"groups has {len(groups)} entries, the set {n} tensors")
        blocks = [-(-k // STATE_BLOCK) for k in self._numels]
        recs = np.zeros(max(1, n), dtype=np.dtype(TensorC))
        recs["numel"][:n] = self._numels
        if groups is not None:
            recs["group"][:n] = [int(g) for g in groups]
        for name, lst in lists.items():
            sizes = blocks if name in ("m_scale", "v_scale") else self._numels
            if name in ("m_scale", "v_scale"):
                _dtype_of(lst, name, _SCALE_DTYPES)
            recs[name][:n] = _addresses(lst, name, sizes, self._dev)
        h = ctypes.c_void_p()
        _check(lib.zero_tensor_set_create(recs.ctypes.data, n, self._grad_type, state_type, out_type,
                                          int(seed) & 0xFFFFFFFF, _raw_stream(stream, self._dev), _ref(h)))
        self._h = h
        if m_rounding == "random":
            _check(lib.zero_tensor_set_m_rounding(h, 1))
        TensorSet._free_late()
        self._keep = lists
        self._counted = {}   # lists written by a call -> their version counters' tensors
        self._work_elems = lib.zero_grad_sumsq_work_bytes(h) // 8

    _late = []   # handles that wait to be freed

    def close(self):
        """Free the set's tables.  Work that uses them must have finished.
        Freeing waits for the device, which a stream that is being captured
        cannot: a set that is closed, or collected, while its thread's current
        stream is, or that the runtime refuses to free, is freed with the next
        set that is made or closed.  Captures of other threads go on."""
        if self._h:
            TensorSet._late.append(self._h)
            self._h = None
        TensorSet._free_late()

    @staticmethod
    def _free_late():
        if not TensorSet._late or torch.cuda.is_current_stream_capturing():
            return
        for _ in range(len(TensorSet._late)):
            try:
                h = TensorSet._late.pop()
            except IndexError:      # another thread has freed the last
                return
            if lib.zero_tensor_set_destroy(h):
                TensorSet._late.append(h)
                return

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _wrote(self, *names):
        """Raise the version counters of lists that a call wrote, so that a
        backward pass that saved one of their tensors before reports it.  Views
        share their base's, so a flat buffer is counted once; which tensors
        these are is looked up at the first such call."""
        if names not in self._counted:
            tensors = [t for name in names for t in self._keep.get(name, ())]
            bases = [t._base for t in tensors]
            views = {id(b): b for b in bases if b is not None}
            self._counted[names] = list(views.values()) + [t for t, b in zip(tensors, bases) if b is None]
        torch.autograd.graph.increment_version(self._counted[names])

    def bind_grads(self, grads, stream=None):
        """Replace the gradient tensors (same sizes and dtype)."""
        grads = list(grads)
        kind = _dtype_of(grads, "grads", _GRAD_DTYPES)
        if grads and kind != self._grad_type:
            raise ValueError("the set's gradients have another dtype")
        ptrs = np.array(_addresses(grads, "grads", self._numels, self._dev) or [0], dtype=np.uint64)
        _check(lib.zero_tensor_set_bind_grads(self._h, ptrs.ctypes.data, _raw_stream(stream, self._dev)))
        self._keep["grad"] = grads

    def grad_sumsq(self, out, accumulate: bool = False, stream=None):
        """zero_grad_sumsq: the sum of squares of every gradient value into
        `out` (one float64 on the device, StepControl.sumsq); accumulate=True
        adds it to what is there."""
        if out.dtype != torch.float64 or out.numel() != 1 or out.get_device() != self._dev:
            raise ValueError(f"out must be one float64 on cuda:{self._dev}")
        work = None
        if self._work_elems:
            # workspace of this call alone, from the pool of its stream: calls
            # on other streams and captured graphs get their own
            if stream is None:
                work = torch.empty(self._work_elems, dtype=torch.float64, device=out.device)
            else:
                with torch.cuda.stream(stream):
                    work = torch.empty(self._work_elems, dtype=torch.float64, device=out.device)
        _check(lib.zero_grad_sumsq(self._h, out.data_ptr(), bool(accumulate),
                                   None if work is None else work.data_ptr(), _raw_stream(stream, self._dev)))

    def adamw_step(self, control: "StepControl", stream=None):
        """zero_adamw_step: the step that `control` began, on every tensor."""
        if control._n_groups == 0:
            raise ValueError("the step has not begun (StepControl.begin)")
        _on_current_device(control.device_index, "the control block")
        _check(lib.zero_adamw_step(self._h, control._ptr, control._n_groups, _raw_stream(stream, self._dev)))
        self._wrote("p", "out")

    def states_from(self, source: "TensorSet", stream=None):
        """zero_states_convert: write `source`'s states into this set's, fp32
        to 8 bits or back."""
        _check(lib.zero_states_convert(self._h, source._h, _raw_stream(stream, self._dev)))
        self._wrote("m", "v")


# ---------------------------------------------------------------------------
# activation checkpoints in 8 bits, and the gradients made from them
# ---------------------------------------------------------------------------

def _matrix(t, what: str, dev: int) -> MatrixC:
    """A tensor as a matrix: its last dimension's values neighbours, the others
    its rows, equally far apart."""
    if t.get_device() != dev:
        raise ValueError(f"{what} is not on cuda:{dev}, the current device")
    kind = _GRAD_DTYPES.get(t.dtype)
    if kind is None:
        raise ValueError(f"{what}: dtype {t.dtype} is not supported")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{what} must have a last dimension")
        try:
            t = t.view(math.prod(t.shape[:-1]), t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{what}: its rows are not equally far apart") from None
    rows, cols = t.shape
    stride, step = t.stride()
    if step != 1 and cols > 1 and rows > 0:
        raise ValueError(f"{what}: the values of a row must be neighbours")
    return MatrixC(t.data_ptr(), rows, cols, stride, kind, 0)


def _wrote(*tensors):
    """Raise autograd's version counters of what a call wrote."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def _workspace(nbytes: int, like, stream):
    """Memory of one call alone, from the pool of its stream: calls on other
    streams and captured graphs get their own."""
    if not nbytes:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _tokens(t, n: int, dev: int):
    """(address, bytes of one) of a contiguous tensor of n tokens."""
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"tokens: dtype {t.dtype} is not supported")
    if t.get_device() != dev:
        raise ValueError(f"tokens are not on cuda:{dev}, the current device")
    if t.numel() != n:
        raise ValueError(f"{t.numel()} tokens for {n} rows")
    if not t.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return t.data_ptr(), t.element_size()


class Checkpoint:
    """A matrix of activations kept in 8 bits (a zero_checkpoint, MXFP8): `code`
    holds rows of e4m3 codes, padded to whole blocks of 32, and `scale` a byte for
    each block.  Made empty from its sizes, or from tensors that hold one
    (`code` [rows, 32 ceil(cols / 32)], `scale` [rows, ceil(cols / 32)], uint8 or
    the float8 types, both contiguous, `code` 16-byte aligned; rows of a larger
    checkpoint are one)."""

    def __init__(self, rows: int = None, cols: int = None, code=None, scale=None, device=None):
        if cols is None or cols < 0 or (code is None) != (scale is None) or (code is None) == (rows is None):
            raise ValueError("a checkpoint takes rows and cols, or code, scale and cols")
        blocks = -(-int(cols) // STATE_BLOCK)
        if code is None:
            if rows < 0:
                raise ValueError("rows must not be negative")
            dev = torch.device("cuda", _current_device()) if device is None else torch.device(device)
            code = torch.empty(int(rows), STATE_BLOCK * blocks, dtype=torch.uint8, device=dev)
            scale = torch.empty(int(rows), blocks, dtype=torch.uint8, device=dev)
        if not code.is_cuda or code.device != scale.device:
            raise ValueError("code and scale live on one GPU")
        if code.dtype not in (torch.uint8, torch.float8_e4m3fn) or scale.dtype not in _SCALE_DTYPES:
            raise ValueError(f"code and scale: dtypes {code.dtype} and {scale.dtype} are not supported")
        if code.dim() != 2 or tuple(code.shape) != (code.shape[0], STATE_BLOCK * blocks) \
                or tuple(scale.shape) != (code.shape[0], blocks):
            raise ValueError(f"code and scale must have rows of {STATE_BLOCK * blocks} and {blocks}")
        if not (code.is_contiguous() and scale.is_contiguous()):
            raise ValueError("code and scale must be contiguous")
        self.rows, self.cols, self.code, self.scale = code.shape[0], int(cols), code, scale
        self.device_index = code.device.index
        self._c = CheckpointC(code.data_ptr(), scale.data_ptr(), self.rows, self.cols)

    def _on(self, dev: int):
        if self.device_index != dev:
            raise ValueError(f"a checkpoint is on cuda:{self.device_index}, the current device is another")
        return _ref(self._c)

    def store(self, x, stream=None):
        """zero_checkpoint_store: keep x (fp16, bf16 or fp32)."""
        dev = _current_device()
        _check(lib.zero_checkpoint_store(_ref(_matrix(x, "x", dev)), self._on(dev), _raw_stream(stream, dev)))
        _wrote(self.code, self.scale)

    def load(self, out, stream=None):
        """zero_checkpoint_load: read it back into `out`."""
        dev = _current_device()
        _check(lib.zero_checkpoint_load(self._on(dev), _ref(_matrix(out, "out", dev)), _raw_stream(stream, dev)))
        _wrote(out)


ACTIVATIONS = {"relu": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def _kind(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"unknown activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


def activation(kind: str, x, out, checkpoint: Checkpoint = None, up=None, up_checkpoint: Checkpoint = None,
               out_checkpoint: Checkpoint = None, stream=None):
    """zero_activation: out = act(x), or act(x) * up, with the checkpoints of x
    and up that activation_grad reads, and of out for weight_grad of the layer
    that comes next.  `kind`: "relu", "silu", "gelu" (erf) or "gelu_tanh".  out
    may be x or up."""
    dev = _current_device()
    kept = [None if c is None else c._on(dev) for c in (checkpoint, up_checkpoint, out_checkpoint)]
    _check(lib.zero_activation(_kind(kind), _ref(_matrix(x, "x", dev)), None if up is None else _ref(_matrix(up, "up", dev)),
                               _ref(_matrix(out, "out", dev)), *kept, _raw_stream(stream, dev)))
    _wrote(out, *(t for c in (checkpoint, up_checkpoint, out_checkpoint) if c is not None for t in (c.code, c.scale)))


def activation_grad(kind: str, dy, checkpoint: Checkpoint, dx, up_checkpoint: Checkpoint = None, dup=None, stream=None):
    """zero_activation_grad: the gradients of x (and up) from that of the
    activation's result, x and up being read from their checkpoints.  dx or dup
    may be dy."""
    dev = _current_device()
    _check(lib.zero_activation_grad(_kind(kind), _ref(_matrix(dy, "dy", dev)), checkpoint._on(dev),
                                    None if up_checkpoint is None else up_checkpoint._on(dev),
                                    _ref(_matrix(dx, "dx", dev)), None if dup is None else _ref(_matrix(dup, "dup", dev)),
                                    _raw_stream(stream, dev)))
    _wrote(dx, dup)


def weight_grad(dy, checkpoint: Checkpoint, dw, bias=None, accumulate: bool = False, stream=None):
    """zero_weight_grad: dw[n, k] = sum of dy[t, n] x[t, k] over the tokens t, x
    being read from its checkpoint, and bias[n] = sum of dy[t, n]; accumulate=True
    adds to what is there.  dw may be the transpose of a tensor (`w.grad.t()` for
    a weight that is kept as inputs by outputs)."""
    dev = _current_device()
    m = _matrix(dy, "dy", dev)
    if dw.dim() != 2 or tuple(dw.shape) != (m.cols, checkpoint.cols):
        raise ValueError(f"dw must be {m.cols} by {checkpoint.cols}")
    transposed = dw.stride(1) != 1 and dw.shape[1] > 1
    if bias is not None and (bias.dtype != dw.dtype or bias.get_device() != dev or not bias.is_contiguous()
                             or bias.numel() != m.cols):
        raise ValueError(f"bias must be {m.cols} neighbouring values of dw's dtype on cuda:{dev}")
    work = _workspace(lib.zero_weight_grad_work_bytes(m.rows, m.cols, checkpoint.cols, m.type), dw, stream)
    _check(lib.zero_weight_grad(_ref(m), checkpoint._on(dev), _ref(_matrix(dw.t() if transposed else dw, "dw", dev)),
                                transposed, None if bias is None else bias.data_ptr(), bool(accumulate),
                                None if work is None else work.data_ptr(), _raw_stream(stream, dev)))
    _wrote(dw, bias)


def embedding_lookup(table, tokens, out, scale: float = 1.0, first: int = 0, stream=None):
    """zero_embedding_lookup: out's rows are scale times the table's rows
    tokens - first; zeros where that is no row (padding, or another rank's)."""
    dev = _current_device()
    m = _matrix(out, "out", dev)
    at, size = _tokens(tokens, m.rows, dev)
    _check(lib.zero_embedding_lookup(_ref(_matrix(table, "table", dev)), at, size, first, scale, _ref(m),
                                     _raw_stream(stream, dev)))
    _wrote(out)


def embedding_grad(dy, tokens, dtable, scale: float = 1.0, first: int = 0, accumulate: bool = False, stream=None):
    """zero_embedding_grad: row r of dtable is scale times the sum of dy's rows
    whose token is first + r; accumulate=True adds that to what is there (other
    rows stay as they are)."""
    dev = _current_device()
    m, d = _matrix(dy, "dy", dev), _matrix(dtable, "dtable", dev)
    at, size = _tokens(tokens, m.rows, dev)
    work = _workspace(lib.zero_embedding_grad_work_bytes(m.rows, d.rows, d.cols), dtable, stream)
    _check(lib.zero_embedding_grad(_ref(m), at, size, first, scale, _ref(d), bool(accumulate),
                                   None if work is None else work.data_ptr(), _raw_stream(stream, dev)))
    _wrote(dtable)


def version() -> int:
    return lib.zero_version()


def device_info():
    arch, mem = ctypes.c_int32(), ctypes.c_int64()
    _check(lib.zero_device_info(_ref(arch), _ref(mem)))
    return arch.value, mem.value


def set_kernel_timing(enable: bool):
    """zero_set_kernel_timing for the calling thread."""
    _check(lib.zero_set_kernel_timing(1 if enable else 0))


def last_kernel_ms() -> float:
    """zero_last_kernel_ms: device time of the last timed call's kernels."""
    ms = ctypes.c_float()
    _check(lib.zero_last_kernel_ms(_ref(ms)))
    return ms.value


def kernel_times() -> list:
    """zero_kernel_times: device time (ms) of every call timed since timing
    was enabled on this thread (at most the last 4096), oldest first."""
    n = ctypes.c_int64()
    buf = (ctypes.c_float * 4096)()
    _check(lib.zero_kernel_times(buf, 4096, _ref(n)))
    return [buf[i] for i in range(n.value)]


def carve_arena(plan: ArenaPlan, device="cuda"):
    """Allocate plan.total_bytes once and return {kind: tensor view} (fp32
    kinds as float32, fp16 kinds as int16 bit patterns)."""
    import torch
    arena = torch.empty(plan.total_bytes, dtype=torch.uint8, device=device)
    views = {"_arena": arena}
    for kind, (off, nbytes) in plan.as_dict().items():
        dt = torch.float32 if kind in ("master", "momentum", "variance", "master_alt",
                                       "momentum_alt", "variance_alt") else torch.int16
        views[kind] = arena[off:off + nbytes].view(dt)
    return views

