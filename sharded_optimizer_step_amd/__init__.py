"""The per-rank ZeRO shard step for MI355X (gfx950): a thin ctypes binding
of the C ABI declared in ``include/zero_step.h``.

This module only marshals arguments (torch tensors -> device or host
pointers and the current HIP stream). Every step of the computation runs in
``libzero_step.so``: its HIP kernels, and for the CPU-offloaded step (whose
optimizer state lives in host memory by design) the host optimizer built
into the same library. There is no CPU fallback: if the library is missing
the first call raises.

Functions keep the C names:

* ``zero_shard_reduce(grads, grad_scale, g_out)``
* ``zero_grad_check_norm_workspace_bytes(n)``
* ``zero_grad_check_norm(g, hp, external_sumsq, ws, res)``
* ``zero_adamw_step(master, exp_avg, exp_avg_sq, g, param_out, hp, res=None)``
* ``zero_step_workspace_bytes(tensors, M, hp)``
* ``zero_step(tensors, hp, external_sumsq, ws, res)``; ``StepRunner(tensors, ws, res).step(hp, external_sumsq)``
  (and ``.step_amp``): the same calls with the tensor list marshalled once
* ``zero_step_noalloc(tensors, hp, external_sumsq, res)``: the same step with the library's static device scratch
  as its workspace, for callers that cannot allocate
* ``zero_loss_scale_init(cfg, ls)``, ``zero_loss_scale_update(cfg, res, ls)``
* ``zero_step_amp_workspace_bytes(tensors, M, hp)``, ``zero_step_amp(tensors, hp, cfg, ls, external_sumsq, ws, res)``
* ``zero_bucket_reduce_workspace_bytes(shards, M)``,
  ``zero_bucket_reduce(shards, flags, grad_scale, stamp, partial, ws)``
* ``zero_step_accumulated_workspace_bytes(tensors)``,
  ``zero_step_accumulated(tensors, hp, partials, nbuckets, stamp, external_sumsq, ws, res)``,
  ``BucketReducer(shards, partial, ws=None, ls=None).reduce(flags, grad_scale, stamp)``
* ``zero_bucket_step_workspace_bytes(tensors, M)``, ``zero_bucket_step(tensors, flags, hp, stamp, partial, ws)``,
  ``BucketStepper(tensors, partial, ws=None).step(flags, hp, stamp)``: a bucket's final micro-batch folded and
  applied in one pass (no clipping, no skipping); then ``zero_step_accumulated([], ...)`` writes the record
* ``zero_offload_workspace_bytes(tensors, M)``, ``zero_offload_host_workspace_bytes(tensors)``,
  ``zero_offload_step(tensors, hp, external_sumsq, ws, host_ws, threads)``,
  ``zero_offload_adamw_host(master, exp_avg, exp_avg_sq, g, param_out, hp, clip_coef, threads)``
* ``zero_bucket_reduce_amp``, ``zero_step_accumulated_amp``, ``zero_offload_step_amp``: the same under the
  dynamic loss scale
* ``zero_act8_save(x, ckpt)``, ``zero_act8_load(ckpt, out)``: activation rows to and from an 8-bit checkpoint
  (``Act8``, made by ``new_act8(rows, cols, format)``)
* ``zero_act8_wgrad_workspace_bytes(rows, outs, cols)``, ``zero_act8_wgrad(dy, ckpt, dw, flags, ws, col_scale=None)``:
  a linear layer's weight gradient from its 8-bit input, as a bf16 replica or into an fp32 accumulator
* ``zero_block_norm(BlockNorm(...))``, ``zero_block_norm_grad_workspace_bytes(rows, cols, gate_rows)``,
  ``zero_block_norm_grad(BlockNormGrad(...), flags, ws)``: the norms after a block and before the next one, fused
  with the block's gate, the residual scale and the residual add, forward and backward
* ``zero_layer_norm(LayerNorm(...))``, ``zero_layer_norm_grad_workspace_bytes(rows, cols)``,
  ``zero_layer_norm_grad(LayerNormGrad(...), flags, ws)``: the residual add and the layer norm before a block, forward
  and backward
* ``zero_block_ffn_workspace_bytes(rows, cols, hidden)``, ``zero_block_ffn(BlockFfn(...), ws)``,
  ``zero_block_ffn_grad_workspace_bytes(rows, cols, hidden)``, ``zero_block_ffn_grad(BlockFfnGrad(...), flags, ws)``:
  the gated feed-forward block's two projections, activation and product in one kernel, and all gradients of it
* ``zero_workspace_forget(ws)``, ``zero_status_string(status)``
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
import weakref
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero_step.so")

ZERO_OK = 0
ZERO_ERR_INVALID_ARGUMENT = 1
ZERO_ERR_WORKSPACE_TOO_SMALL = 2
ZERO_ERR_HIP = 3
ZERO_ERR_STALE_WORKSPACE = 4
ZERO_ERR_BUCKET_PARTIALS = 5
ZERO_ERR_SCRATCH_TOO_SMALL = 6
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
RESULT_BYTES = 32
BUCKET_ACCUMULATE = 1
BUCKET_FINAL = 2
BUCKET_STREAM_STORES = 4
# steps above this many parameters write more than the 256 MiB Infinity Cache holds
STREAM_STORES_MIN_PARAMS = (256 << 20) // 14
BUCKET_PARTIAL_BYTES = 32
ACT8_E4M3 = 1
ACT8_INT8 = 2
GRAD_ACCUMULATE = 1
BLOCK_NORM_MAX_COLS = 16384
FFN_SILU = 1
FFN_GELU = 2
FFN_GELU_TANH = 3

# Every symbol the C ABI exports (include/zero_step.h).
EXPORTS = ("zero_shard_reduce", "zero_grad_check_norm_workspace_bytes", "zero_grad_check_norm", "zero_adamw_step",
           "zero_step_workspace_bytes", "zero_step", "zero_loss_scale_init", "zero_loss_scale_update",
           "zero_step_amp_workspace_bytes", "zero_step_amp", "zero_bucket_reduce_workspace_bytes",
           "zero_bucket_reduce", "zero_step_accumulated_workspace_bytes", "zero_step_accumulated",
           "zero_offload_workspace_bytes", "zero_offload_host_workspace_bytes", "zero_offload_step",
           "zero_offload_adamw_host", "zero_bucket_reduce_amp", "zero_step_accumulated_amp",
           "zero_offload_step_amp", "zero_workspace_forget", "zero_status_string", "zero_step_noalloc",
           "zero_bucket_step_workspace_bytes", "zero_bucket_step", "zero_act8_bytes", "zero_act8_save",
           "zero_act8_load", "zero_act8_wgrad_workspace_bytes", "zero_act8_wgrad", "zero_block_norm",
           "zero_block_norm_grad_workspace_bytes", "zero_block_norm_grad", "zero_layer_norm",
           "zero_layer_norm_grad_workspace_bytes", "zero_layer_norm_grad", "zero_block_ffn_workspace_bytes",
           "zero_block_ffn", "zero_block_ffn_grad_workspace_bytes", "zero_block_ffn_grad")
LOSS_SCALE_BYTES = 16


class _CHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("max_grad_norm", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("skip_on_nonfinite", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _CTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grads", ctypes.POINTER(ctypes.c_void_p)), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("param_out", ctypes.c_void_p)]


class _CGradShard(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grads", ctypes.POINTER(ctypes.c_void_p)), ("grad_acc", ctypes.c_void_p)]


class _CAccTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grad_acc", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("param_out", ctypes.c_void_p)]


class _CBucketTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grads", ctypes.POINTER(ctypes.c_void_p)), ("grad_acc", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("param_out", ctypes.c_void_p)]


class _COffloadTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grads", ctypes.POINTER(ctypes.c_void_p)), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("param_out", ctypes.c_void_p)]


class _CResult(ctypes.Structure):
    _fields_ = [("sumsq", ctypes.c_double), ("clip_coef", ctypes.c_double), ("grad_norm", ctypes.c_float),
                ("found_inf", ctypes.c_int32), ("skipped", ctypes.c_int32), ("status", ctypes.c_int32)]


class _CLossScaleConfig(ctypes.Structure):
    _fields_ = [("initial_scale_power", ctypes.c_int32), ("window", ctypes.c_int32), ("hysteresis", ctypes.c_int32),
                ("min_scale", ctypes.c_float)]


class _CRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _CBlockNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_double), ("eps", ctypes.c_double), ("x", _CRows), ("y", _CRows),
                ("w_post", _CRows), ("gate", _CRows), ("w_pre", _CRows), ("x_out", _CRows), ("h", _CRows),
                ("rstd_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p), ("ckpt_post", ctypes.c_void_p),
                ("ckpt_pre", ctypes.c_void_p), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _CBlockNormGrad(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
                ("residual_scale", ctypes.c_double), ("dh", _CRows), ("dx_out", _CRows), ("w_post", _CRows),
                ("gate", _CRows), ("w_pre", _CRows), ("x_out", _CRows), ("y", _CRows), ("ckpt_pre", ctypes.c_void_p),
                ("ckpt_post", ctypes.c_void_p), ("rstd_pre", ctypes.c_void_p), ("rstd_post", ctypes.c_void_p),
                ("dx", _CRows), ("dy", _CRows), ("dw_pre", _CRows), ("dw_post", _CRows), ("dgate", _CRows),
                ("format", ctypes.c_int32), ("flags", ctypes.c_int32)]


class _CLayerNorm(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("eps", ctypes.c_double), ("x", _CRows),
                ("y", _CRows), ("w", _CRows), ("b", _CRows), ("x_out", _CRows), ("h", _CRows),
                ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("ckpt_xn", ctypes.c_void_p),
                ("ckpt_h", ctypes.c_void_p), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _CLayerNormGrad(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("dh", _CRows), ("dx_out", _CRows), ("w", _CRows),
                ("x_out", _CRows), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("ckpt_xn", ctypes.c_void_p),
                ("dx", _CRows), ("dy", _CRows), ("dw", _CRows), ("db", _CRows), ("format", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class _CBlockFfn(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("hidden", ctypes.c_int64), ("h", _CRows),
                ("w_gate", _CRows), ("w_up", _CRows), ("a", _CRows), ("gate", _CRows), ("up", _CRows),
                ("ckpt_gate", ctypes.c_void_p), ("ckpt_up", ctypes.c_void_p), ("format", ctypes.c_int32),
                ("act", ctypes.c_int32)]


class _CBlockFfnGrad(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("hidden", ctypes.c_int64), ("da", _CRows),
                ("gate", _CRows), ("up", _CRows), ("ckpt_gate", ctypes.c_void_p), ("ckpt_up", ctypes.c_void_p),
                ("w_gate", _CRows), ("w_up", _CRows), ("h", _CRows), ("ckpt_h", ctypes.c_void_p),
                ("col_scale", _CRows), ("dgate", _CRows), ("dup", _CRows), ("dh", _CRows), ("dw_gate", _CRows),
                ("dw_up", _CRows), ("ckpt_a", ctypes.c_void_p), ("format", ctypes.c_int32), ("act", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ZeroError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {zero_status_string(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, dbl, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_size_t
        L.zero_shard_reduce.argtypes = [ctypes.POINTER(vp), i32, i64, dbl, vp, vp]
        L.zero_shard_reduce.restype = ctypes.c_int
        L.zero_grad_check_norm_workspace_bytes.argtypes = [i64]
        L.zero_grad_check_norm_workspace_bytes.restype = sz
        L.zero_grad_check_norm.argtypes = [vp, i64, ctypes.POINTER(_CHparams), dbl, vp, sz, vp, vp]
        L.zero_grad_check_norm.restype = ctypes.c_int
        L.zero_adamw_step.argtypes = [vp, vp, vp, vp, vp, i64, ctypes.POINTER(_CHparams), vp, vp]
        L.zero_adamw_step.restype = ctypes.c_int
        L.zero_step_workspace_bytes.argtypes = [ctypes.POINTER(_CTensor), i32, i32, ctypes.POINTER(_CHparams)]
        L.zero_step_workspace_bytes.restype = sz
        L.zero_step.argtypes = [ctypes.POINTER(_CTensor), i32, i32, ctypes.POINTER(_CHparams), dbl, vp, sz, vp, vp]
        L.zero_step.restype = ctypes.c_int
        L.zero_step_noalloc.argtypes = [ctypes.POINTER(_CTensor), i32, i32, ctypes.POINTER(_CHparams), dbl, vp, vp]
        L.zero_step_noalloc.restype = ctypes.c_int
        L.zero_loss_scale_init.argtypes = [ctypes.POINTER(_CLossScaleConfig), vp, vp]
        L.zero_loss_scale_init.restype = ctypes.c_int
        L.zero_loss_scale_update.argtypes = [ctypes.POINTER(_CLossScaleConfig), vp, vp, vp]
        L.zero_loss_scale_update.restype = ctypes.c_int
        L.zero_step_amp_workspace_bytes.argtypes = [ctypes.POINTER(_CTensor), i32, i32, ctypes.POINTER(_CHparams)]
        L.zero_step_amp_workspace_bytes.restype = sz
        L.zero_step_amp.argtypes = [ctypes.POINTER(_CTensor), i32, i32, ctypes.POINTER(_CHparams),
                                    ctypes.POINTER(_CLossScaleConfig), vp, dbl, vp, sz, vp, vp]
        L.zero_step_amp.restype = ctypes.c_int
        u64 = ctypes.c_uint64
        L.zero_bucket_reduce_workspace_bytes.argtypes = [ctypes.POINTER(_CGradShard), i32, i32]
        L.zero_bucket_reduce_workspace_bytes.restype = sz
        L.zero_bucket_reduce.argtypes = [ctypes.POINTER(_CGradShard), i32, i32, i32, dbl, u64, vp, vp, sz, vp]
        L.zero_bucket_reduce.restype = ctypes.c_int
        L.zero_step_accumulated_workspace_bytes.argtypes = [ctypes.POINTER(_CAccTensor), i32]
        L.zero_step_accumulated_workspace_bytes.restype = sz
        L.zero_step_accumulated.argtypes = [ctypes.POINTER(_CAccTensor), i32, ctypes.POINTER(_CHparams), vp, i32,
                                            u64, dbl, vp, sz, vp, vp]
        L.zero_step_accumulated.restype = ctypes.c_int
        L.zero_bucket_step_workspace_bytes.argtypes = [ctypes.POINTER(_CBucketTensor), i32, i32]
        L.zero_bucket_step_workspace_bytes.restype = sz
        L.zero_bucket_step.argtypes = [ctypes.POINTER(_CBucketTensor), i32, i32, i32, ctypes.POINTER(_CHparams), u64,
                                       vp, vp, sz, vp]
        L.zero_bucket_step.restype = ctypes.c_int
        L.zero_offload_workspace_bytes.argtypes = [ctypes.POINTER(_COffloadTensor), i32, i32]
        L.zero_offload_workspace_bytes.restype = sz
        L.zero_offload_host_workspace_bytes.argtypes = [ctypes.POINTER(_COffloadTensor), i32]
        L.zero_offload_host_workspace_bytes.restype = sz
        L.zero_offload_step.argtypes = [ctypes.POINTER(_COffloadTensor), i32, i32, ctypes.POINTER(_CHparams), dbl, vp,
                                        sz, vp, sz, ctypes.POINTER(_CResult), i32, vp]
        L.zero_offload_step.restype = ctypes.c_int
        L.zero_offload_adamw_host.argtypes = [vp, vp, vp, vp, vp, i64, ctypes.POINTER(_CHparams), dbl, i32]
        L.zero_offload_adamw_host.restype = ctypes.c_int
        lsc = ctypes.POINTER(_CLossScaleConfig)
        L.zero_bucket_reduce_amp.argtypes = [ctypes.POINTER(_CGradShard), i32, i32, i32, dbl, vp, u64, vp, vp, sz, vp]
        L.zero_bucket_reduce_amp.restype = ctypes.c_int
        L.zero_step_accumulated_amp.argtypes = [ctypes.POINTER(_CAccTensor), i32, ctypes.POINTER(_CHparams), lsc, vp,
                                                vp, i32, u64, dbl, vp, sz, vp, vp]
        L.zero_step_accumulated_amp.restype = ctypes.c_int
        L.zero_offload_step_amp.argtypes = [ctypes.POINTER(_COffloadTensor), i32, i32, ctypes.POINTER(_CHparams), lsc,
                                            vp, dbl, vp, sz, vp, sz, ctypes.POINTER(_CResult), i32, vp]
        L.zero_offload_step_amp.restype = ctypes.c_int
        rows = vp  # a zero_rows, as packed bytes or by reference
        L.zero_act8_bytes.argtypes = [i64, i64]
        L.zero_act8_bytes.restype = sz
        L.zero_act8_save.argtypes = [rows, i64, i64, i32, vp, vp]
        L.zero_act8_save.restype = ctypes.c_int
        L.zero_act8_load.argtypes = [vp, i64, i64, i32, rows, vp]
        L.zero_act8_load.restype = ctypes.c_int
        L.zero_act8_wgrad_workspace_bytes.argtypes = [i64, i64, i64]
        L.zero_act8_wgrad_workspace_bytes.restype = sz
        L.zero_act8_wgrad.argtypes = [rows, vp, i64, i64, i64, i32, rows, rows, i32, vp, sz, vp]
        L.zero_act8_wgrad.restype = ctypes.c_int
        L.zero_block_norm.argtypes = [vp, vp]
        L.zero_block_norm.restype = ctypes.c_int
        L.zero_block_norm_grad_workspace_bytes.argtypes = [i64, i64, i64]
        L.zero_block_norm_grad_workspace_bytes.restype = sz
        L.zero_block_norm_grad.argtypes = [vp, vp, sz, vp]
        L.zero_block_norm_grad.restype = ctypes.c_int
        L.zero_layer_norm.argtypes = [vp, vp]
        L.zero_layer_norm.restype = ctypes.c_int
        L.zero_layer_norm_grad_workspace_bytes.argtypes = [i64, i64]
        L.zero_layer_norm_grad_workspace_bytes.restype = sz
        L.zero_layer_norm_grad.argtypes = [vp, vp, sz, vp]
        L.zero_layer_norm_grad.restype = ctypes.c_int
        L.zero_block_ffn_workspace_bytes.argtypes = [i64, i64, i64]
        L.zero_block_ffn_workspace_bytes.restype = sz
        L.zero_block_ffn.argtypes = [vp, vp, sz, vp]
        L.zero_block_ffn.restype = ctypes.c_int
        L.zero_block_ffn_grad_workspace_bytes.argtypes = [i64, i64, i64]
        L.zero_block_ffn_grad_workspace_bytes.restype = sz
        L.zero_block_ffn_grad.argtypes = [vp, vp, sz, vp]
        L.zero_block_ffn_grad.restype = ctypes.c_int
        L.zero_workspace_forget.argtypes = [vp]
        L.zero_workspace_forget.restype = ctypes.c_int
        L.zero_status_string.argtypes = [ctypes.c_int]
        L.zero_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


@dataclasses.dataclass
class HParams:
    """AdamW knobs of one step (names of a deepspeed_config.json optimizer
    block), the step index t >= 1, the clip threshold (<= 0: off), the
    multiplier of the fp32 gradient sum, and the skip switch."""
    lr: float = 1e-3
    beta1: float = 0.9
    beta2: float = 0.95
    eps: float = 1e-8
    weight_decay: float = 0.1
    step: int = 1
    max_grad_norm: float = 0.0
    grad_scale: float = 1.0
    skip_on_nonfinite: int = 0

    def _c(self) -> _CHparams:
        return _CHparams(float(self.lr), float(self.beta1), float(self.beta2), float(self.eps),
                         float(self.weight_decay), int(self.step), float(self.max_grad_norm), float(self.grad_scale),
                         int(bool(self.skip_on_nonfinite)), 0)


@dataclasses.dataclass
class ZeroTensor:
    """One tensor's shard: M bf16 gradient replicas, fp32 master/exp_avg/
    exp_avg_sq (updated in place) and the bf16 output shard."""
    grads: List[torch.Tensor]
    master: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    param_out: torch.Tensor


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str, n: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")


def _need_ws(ws: Optional[torch.Tensor], name: str = "ws") -> int:
    """A device workspace (any dtype, contiguous) or None; returns its bytes.
    The library writes through it from kernels: a host tensor here would be a
    host address on the GPU."""
    if ws is None:
        return 0
    if not isinstance(ws, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not ws.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if not ws.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return ws.numel() * ws.element_size()


def _check(status: int, where: str):
    if status != ZERO_OK:
        raise ZeroError(status, where)


def zero_status_string(status: int) -> str:
    return lib().zero_status_string(int(status)).decode()


def new_result(device=None) -> torch.Tensor:
    """A 32-byte device buffer for the zero_result record."""
    return torch.zeros(RESULT_BYTES, dtype=torch.uint8, device=device or "cuda")


def read_result(res: torch.Tensor) -> dict:
    """Copy the record to the host (synchronizes with its stream)."""
    b = bytes(res.cpu().numpy().tobytes())
    sumsq, coef, norm, found_inf, skipped, status = struct.unpack("<ddfiii", b)
    return dict(sumsq=sumsq, grad_norm=norm, clip_coef=coef, found_inf=found_inf, skipped=skipped, status=status)


def zero_shard_reduce(grads: Sequence[torch.Tensor], grad_scale: float, g_out: torch.Tensor, stream=None) -> None:
    n = g_out.numel()
    _need(g_out, torch.float32, "g_out")
    for r, g in enumerate(grads):
        _need(g, torch.bfloat16, f"grads[{r}]", n)
    arr = (ctypes.c_void_p * max(len(grads), 1))(*[g.data_ptr() for g in grads])
    _check(lib().zero_shard_reduce(arr, len(grads), n, float(grad_scale), g_out.data_ptr(), _stream(stream)),
           "zero_shard_reduce")


def zero_grad_check_norm_workspace_bytes(n: int) -> int:
    return int(lib().zero_grad_check_norm_workspace_bytes(int(n)))


def zero_grad_check_norm(g: torch.Tensor, hp: Optional[HParams], external_sumsq: float, ws: Optional[torch.Tensor],
                         res: torch.Tensor, stream=None) -> None:
    _need(g, torch.float32, "g")
    _need(res, torch.uint8, "res", RESULT_BYTES)
    h = hp._c() if hp is not None else None
    wsb = _need_ws(ws)
    _check(lib().zero_grad_check_norm(g.data_ptr(), g.numel(), ctypes.byref(h) if h is not None else None,
                                      float(external_sumsq), _ptr(ws), wsb, res.data_ptr(), _stream(stream)),
           "zero_grad_check_norm")


def zero_adamw_step(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, g: torch.Tensor,
                    param_out: torch.Tensor, hp: HParams, res: Optional[torch.Tensor] = None, stream=None) -> None:
    n = master.numel()
    for t, nm in ((master, "master"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (g, "g")):
        _need(t, torch.float32, nm, n)
    _need(param_out, torch.bfloat16, "param_out", n)
    if res is not None:
        _need(res, torch.uint8, "res", RESULT_BYTES)
    h = hp._c()
    _check(lib().zero_adamw_step(master.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), g.data_ptr(),
                                 param_out.data_ptr(), n, ctypes.byref(h), _ptr(res), _stream(stream)),
           "zero_adamw_step")


def _ctensors(tensors: Sequence[ZeroTensor], check: bool):
    M = len(tensors[0].grads) if tensors else 1
    keep = []
    arr = (_CTensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        n = t.master.numel()
        if check:
            if len(t.grads) != M:
                raise ValueError(f"tensor {i}: {len(t.grads)} replicas, expected {M}")
            for r, g in enumerate(t.grads):
                _need(g, torch.bfloat16, f"tensors[{i}].grads[{r}]", n)
            for x, nm in ((t.master, "master"), (t.exp_avg, "exp_avg"), (t.exp_avg_sq, "exp_avg_sq")):
                _need(x, torch.float32, f"tensors[{i}].{nm}", n)
            _need(t.param_out, torch.bfloat16, f"tensors[{i}].param_out", n)
        ptrs = (ctypes.c_void_p * max(M, 1))(*[g.data_ptr() for g in t.grads])
        keep.append(ptrs)
        arr[i] = _CTensor(n, ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), t.master.data_ptr(),
                          t.exp_avg.data_ptr(), t.exp_avg_sq.data_ptr(), t.param_out.data_ptr())
    return arr, keep, M


def zero_step_workspace_bytes(tensors: Sequence[ZeroTensor], M: int, hp: HParams) -> int:
    arr, keep, _ = _ctensors(tensors, check=False)
    h = hp._c()
    return int(lib().zero_step_workspace_bytes(arr, len(tensors), int(M), ctypes.byref(h)))


def zero_step(tensors: Sequence[ZeroTensor], hp: HParams, external_sumsq: float, ws: Optional[torch.Tensor],
              res: torch.Tensor, stream=None) -> None:
    _need(res, torch.uint8, "res", RESULT_BYTES)
    arr, keep, M = _ctensors(tensors, check=True)
    h = hp._c()
    wsb = _need_ws(ws)
    _check(lib().zero_step(arr, len(tensors), M, ctypes.byref(h), float(external_sumsq), _ptr(ws), wsb,
                           res.data_ptr(), _stream(stream)), "zero_step")


class StepRunner:
    """A tensor list marshalled once, for a training loop that steps it every
    iteration: step() and step_amp() call zero_step and zero_step_amp with
    the pointer tables prepared here, so a call costs one small structure of
    hyperparameters instead of checking every replica of every tensor again
    (about 2 ms of host time per call on a 288-tensor list with 8 replicas).
    The tensors, the workspace and the result record must stay alive and at
    the same addresses."""

    def __init__(self, tensors: Sequence[ZeroTensor], ws: Optional[torch.Tensor], res: torch.Tensor):
        _need(res, torch.uint8, "res", RESULT_BYTES)
        self._arr, self._keep, self.M = _ctensors(tensors, check=True)
        self._tensors = list(tensors)
        self.T = len(self._tensors)
        self.ws, self.res = ws, res
        self._wsp, self._wsb = _ptr(ws), _need_ws(ws)

    def step(self, hp: HParams, external_sumsq: float = 0.0, stream=None) -> None:
        h = hp._c()
        st = lib().zero_step(self._arr, self.T, self.M, ctypes.byref(h), float(external_sumsq), self._wsp, self._wsb,
                             self.res.data_ptr(), _stream(stream))
        if st != ZERO_OK:
            raise ZeroError(st, "zero_step")

    def step_amp(self, hp: HParams, cfg: "LossScaleConfig", ls: torch.Tensor, external_sumsq: float = 0.0,
                 stream=None) -> None:
        h, c = hp._c(), cfg._c()
        st = lib().zero_step_amp(self._arr, self.T, self.M, ctypes.byref(h), ctypes.byref(c), ls.data_ptr(),
                                 float(external_sumsq), self._wsp, self._wsb, self.res.data_ptr(), _stream(stream))
        if st != ZERO_OK:
            raise ZeroError(st, "zero_step_amp")


def zero_step_noalloc(tensors: Sequence[ZeroTensor], hp: HParams, external_sumsq: float, res: torch.Tensor,
                      stream=None) -> None:
    """zero_step with the library's static device scratch as its workspace
    (NOALLOC_SCRATCH_BYTES per GPU): the call allocates nothing. Calls on one
    GPU share the scratch and must be ordered."""
    _need(res, torch.uint8, "res", RESULT_BYTES)
    arr, keep, M = _ctensors(tensors, check=True)
    h = hp._c()
    _check(lib().zero_step_noalloc(arr, len(tensors), M, ctypes.byref(h), float(external_sumsq), res.data_ptr(),
                                   _stream(stream)), "zero_step_noalloc")


@dataclasses.dataclass
class LossScaleConfig:
    """Dynamic loss-scale knobs (names of the fp16 block of a
    deepspeed_config.json; defaults are the values printed there)."""
    initial_scale_power: int = 12
    window: int = 1000
    hysteresis: int = 2
    min_scale: float = 1.0

    def _c(self) -> _CLossScaleConfig:
        return _CLossScaleConfig(int(self.initial_scale_power), int(self.window), int(self.hysteresis),
                                 float(self.min_scale))


def new_loss_scale(device=None) -> torch.Tensor:
    """A 16-byte device buffer for the zero_loss_scale state."""
    return torch.zeros(LOSS_SCALE_BYTES, dtype=torch.uint8, device=device or "cuda")


def read_loss_scale(ls: torch.Tensor) -> dict:
    """Copy the state to the host (synchronizes with its stream)."""
    scale, inv_scale, good_steps, overflows = struct.unpack("<ffii", bytes(ls.cpu().numpy().tobytes()))
    return dict(scale=scale, inv_scale=inv_scale, good_steps=good_steps, overflows=overflows)


def zero_loss_scale_init(cfg: LossScaleConfig, ls: torch.Tensor, stream=None) -> None:
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    c = cfg._c()
    _check(lib().zero_loss_scale_init(ctypes.byref(c), ls.data_ptr(), _stream(stream)), "zero_loss_scale_init")


def zero_loss_scale_update(cfg: LossScaleConfig, res: torch.Tensor, ls: torch.Tensor, stream=None) -> None:
    _need(res, torch.uint8, "res", RESULT_BYTES)
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    c = cfg._c()
    _check(lib().zero_loss_scale_update(ctypes.byref(c), res.data_ptr(), ls.data_ptr(), _stream(stream)),
           "zero_loss_scale_update")


def zero_step_amp_workspace_bytes(tensors: Sequence[ZeroTensor], M: int, hp: HParams) -> int:
    arr, keep, _ = _ctensors(tensors, check=False)
    h = hp._c()
    return int(lib().zero_step_amp_workspace_bytes(arr, len(tensors), int(M), ctypes.byref(h)))


def zero_step_amp(tensors: Sequence[ZeroTensor], hp: HParams, cfg: LossScaleConfig, ls: torch.Tensor,
                  external_sumsq: float, ws: Optional[torch.Tensor], res: torch.Tensor, stream=None) -> None:
    _need(res, torch.uint8, "res", RESULT_BYTES)
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    arr, keep, M = _ctensors(tensors, check=True)
    h = hp._c()
    c = cfg._c()
    wsb = _need_ws(ws)
    _check(lib().zero_step_amp(arr, len(tensors), M, ctypes.byref(h), ctypes.byref(c), ls.data_ptr(),
                               float(external_sumsq), _ptr(ws), wsb, res.data_ptr(), _stream(stream)),
           "zero_step_amp")


# ---------------------------------------------------------------- ZeRO-2 streaming

@dataclasses.dataclass
class GradShard:
    """One tensor shard of a gradient bucket: M bf16 replicas of this
    micro-batch and the shard's fp32 gradient accumulator."""
    grads: List[torch.Tensor]
    grad_acc: torch.Tensor


@dataclasses.dataclass
class AccTensor:
    """One tensor shard of the step from accumulated gradients."""
    grad_acc: torch.Tensor
    master: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    param_out: torch.Tensor


def new_bucket_partials(nbuckets: int, device=None) -> torch.Tensor:
    """Device storage for nbuckets zero_bucket_partial records (32 bytes each)."""
    return torch.zeros(max(nbuckets, 1) * BUCKET_PARTIAL_BYTES, dtype=torch.uint8, device=device or "cuda")


def read_bucket_partial(partials: torch.Tensor, index: int = 0) -> dict:
    """Copy one bucket partial to the host (synchronizes with its stream)."""
    b = bytes(partials[index * BUCKET_PARTIAL_BYTES:(index + 1) * BUCKET_PARTIAL_BYTES].cpu().numpy().tobytes())
    sumsq, stamp, found_inf, scale, reserved = struct.unpack("<dQifq", b)
    return dict(sumsq=sumsq, stamp=stamp, found_inf=found_inf, grad_scale=scale, reserved=reserved)


def _cshards(shards: Sequence[GradShard], check: bool):
    M = len(shards[0].grads) if shards else 1
    keep = []
    arr = (_CGradShard * max(len(shards), 1))()
    for i, t in enumerate(shards):
        n = t.grad_acc.numel()
        if check:
            if len(t.grads) != M:
                raise ValueError(f"shard {i}: {len(t.grads)} replicas, expected {M}")
            for r, g in enumerate(t.grads):
                _need(g, torch.bfloat16, f"shards[{i}].grads[{r}]", n)
            _need(t.grad_acc, torch.float32, f"shards[{i}].grad_acc", n)
        ptrs = (ctypes.c_void_p * max(M, 1))(*[g.data_ptr() for g in t.grads])
        keep.append(ptrs)
        arr[i] = _CGradShard(n, ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), t.grad_acc.data_ptr())
    return arr, keep, M


def zero_bucket_reduce_workspace_bytes(shards: Sequence[GradShard], M: int) -> int:
    arr, keep, _ = _cshards(shards, check=False)
    return int(lib().zero_bucket_reduce_workspace_bytes(arr, len(shards), int(M)))


def zero_bucket_reduce(shards: Sequence[GradShard], flags: int, grad_scale: float, stamp: int,
                       partial: Optional[torch.Tensor], ws: Optional[torch.Tensor], stream=None) -> None:
    """partial: a 32-byte slice of new_bucket_partials(...) (this bucket's
    record), required with BUCKET_FINAL."""
    if partial is not None:
        _need(partial, torch.uint8, "partial", BUCKET_PARTIAL_BYTES)
    arr, keep, M = _cshards(shards, check=True)
    wsb = _need_ws(ws)
    _check(lib().zero_bucket_reduce(arr, len(shards), M, int(flags), float(grad_scale), int(stamp) & (2**64 - 1),
                                    _ptr(partial), _ptr(ws), wsb, _stream(stream)), "zero_bucket_reduce")


class BucketReducer:
    """One gradient bucket marshalled once, for a training loop that reduces
    it every micro-batch: reduce() calls zero_bucket_reduce with the arguments
    prepared here and no per-call Python checks. The shards' tensors, the
    partial and the workspace must stay alive and at the same addresses."""

    def __init__(self, shards: Sequence[GradShard], partial: Optional[torch.Tensor], ws: Optional[torch.Tensor] = None,
                 ls: Optional[torch.Tensor] = None):
        self._arr, self._keep, self.M = _cshards(shards, check=True)
        self._shards = list(shards)
        self.T = len(self._shards)
        if partial is not None:
            _need(partial, torch.uint8, "partial", BUCKET_PARTIAL_BYTES)
        self._partial = partial
        if ws is None:
            ws = workspace(zero_bucket_reduce_workspace_bytes(self._shards, self.M))
        self.ws = ws
        self._wsp = _ptr(ws)
        self._wsb = _need_ws(ws)
        self._pp = _ptr(partial)
        if ls is not None:
            _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
        self._ls = ls  # AMP: the dynamic loss scale the final pass reads
        self._fn = lib().zero_bucket_reduce if ls is None else lib().zero_bucket_reduce_amp

    def reduce(self, flags: int, grad_scale: float, stamp: int, stream=None) -> None:
        if self._ls is None:
            st = self._fn(self._arr, self.T, self.M, flags, grad_scale, stamp & 0xFFFFFFFFFFFFFFFF, self._pp,
                          self._wsp, self._wsb, _stream(stream))
        else:
            st = self._fn(self._arr, self.T, self.M, flags, grad_scale, self._ls.data_ptr(),
                          stamp & 0xFFFFFFFFFFFFFFFF, self._pp, self._wsp, self._wsb, _stream(stream))
        if st != ZERO_OK:
            raise ZeroError(st, "zero_bucket_reduce")


def zero_bucket_reduce_amp(shards: Sequence[GradShard], flags: int, grad_scale: float, ls: torch.Tensor, stamp: int,
                           partial: Optional[torch.Tensor], ws: Optional[torch.Tensor], stream=None) -> None:
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    if partial is not None:
        _need(partial, torch.uint8, "partial", BUCKET_PARTIAL_BYTES)
    arr, keep, M = _cshards(shards, check=True)
    wsb = _need_ws(ws)
    _check(lib().zero_bucket_reduce_amp(arr, len(shards), M, int(flags), float(grad_scale), ls.data_ptr(),
                                        int(stamp) & (2**64 - 1), _ptr(partial), _ptr(ws), wsb, _stream(stream)),
           "zero_bucket_reduce_amp")


def _cacc(tensors: Sequence[AccTensor], check: bool):
    arr = (_CAccTensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        n = t.master.numel()
        if check:
            for x, nm in ((t.grad_acc, "grad_acc"), (t.master, "master"), (t.exp_avg, "exp_avg"),
                          (t.exp_avg_sq, "exp_avg_sq")):
                _need(x, torch.float32, f"tensors[{i}].{nm}", n)
            _need(t.param_out, torch.bfloat16, f"tensors[{i}].param_out", n)
        arr[i] = _CAccTensor(n, t.grad_acc.data_ptr(), t.master.data_ptr(), t.exp_avg.data_ptr(),
                             t.exp_avg_sq.data_ptr(), t.param_out.data_ptr())
    return arr


def zero_step_accumulated_workspace_bytes(tensors: Sequence[AccTensor]) -> int:
    return int(lib().zero_step_accumulated_workspace_bytes(_cacc(tensors, check=False), len(tensors)))


def zero_step_accumulated(tensors: Sequence[AccTensor], hp: HParams, partials: Optional[torch.Tensor], nbuckets: int,
                          stamp: int, external_sumsq: float, ws: Optional[torch.Tensor], res: torch.Tensor,
                          stream=None) -> None:
    _need(res, torch.uint8, "res", RESULT_BYTES)
    if nbuckets > 0:
        _need(partials, torch.uint8, "partials")
        if partials.numel() < nbuckets * BUCKET_PARTIAL_BYTES:
            raise ValueError(f"partials: {partials.numel()} bytes for {nbuckets} buckets")
    arr = _cacc(tensors, check=True)
    h = hp._c()
    wsb = _need_ws(ws)
    _check(lib().zero_step_accumulated(arr, len(tensors), ctypes.byref(h), _ptr(partials), int(nbuckets),
                                       int(stamp) & (2**64 - 1), float(external_sumsq), _ptr(ws), wsb,
                                       res.data_ptr(), _stream(stream)), "zero_step_accumulated")


# ---------------------------------------------------------------- ZeRO-2, fused final pass

@dataclasses.dataclass
class BucketTensor:
    """One tensor shard of a bucket's fused final pass: this micro-batch's M
    bf16 replicas, the fp32 accumulator of the earlier micro-batches (read
    with BUCKET_ACCUMULATE; may be None otherwise), the fp32 state (updated in
    place) and the bf16 output shard."""
    grads: List[torch.Tensor]
    grad_acc: Optional[torch.Tensor]
    master: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    param_out: torch.Tensor


def _cbucket(tensors: Sequence[BucketTensor], check: bool):
    M = len(tensors[0].grads) if tensors else 1
    keep = []
    arr = (_CBucketTensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        n = t.master.numel()
        if check:
            if len(t.grads) != M:
                raise ValueError(f"tensor {i}: {len(t.grads)} replicas, expected {M}")
            for r, g in enumerate(t.grads):
                _need(g, torch.bfloat16, f"tensors[{i}].grads[{r}]", n)
            for x, nm in ((t.master, "master"), (t.exp_avg, "exp_avg"), (t.exp_avg_sq, "exp_avg_sq")):
                _need(x, torch.float32, f"tensors[{i}].{nm}", n)
            if t.grad_acc is not None:
                _need(t.grad_acc, torch.float32, f"tensors[{i}].grad_acc", n)
            _need(t.param_out, torch.bfloat16, f"tensors[{i}].param_out", n)
        ptrs = (ctypes.c_void_p * max(M, 1))(*[g.data_ptr() for g in t.grads])
        keep.append(ptrs)
        arr[i] = _CBucketTensor(n, ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), _ptr(t.grad_acc),
                                t.master.data_ptr(), t.exp_avg.data_ptr(), t.exp_avg_sq.data_ptr(),
                                t.param_out.data_ptr())
    return arr, keep, M


def zero_bucket_step_workspace_bytes(tensors: Sequence[BucketTensor], M: int) -> int:
    arr, keep, _ = _cbucket(tensors, check=False)
    return int(lib().zero_bucket_step_workspace_bytes(arr, len(tensors), int(M)))


def zero_bucket_step(tensors: Sequence[BucketTensor], flags: int, hp: HParams, stamp: int, partial: torch.Tensor,
                     ws: Optional[torch.Tensor], stream=None) -> None:
    """The final micro-batch of one bucket, folded and applied in one pass
    (no clipping, no skipping); partial: this bucket's 32-byte record."""
    _need(partial, torch.uint8, "partial", BUCKET_PARTIAL_BYTES)
    arr, keep, M = _cbucket(tensors, check=True)
    h = hp._c()
    wsb = _need_ws(ws)
    _check(lib().zero_bucket_step(arr, len(tensors), M, int(flags), ctypes.byref(h), int(stamp) & (2**64 - 1),
                                  partial.data_ptr(), _ptr(ws), wsb, _stream(stream)), "zero_bucket_step")


class BucketStepper:
    """One bucket's fused final pass marshalled once (for a loop that runs it
    every step): step() calls zero_bucket_step with the arguments prepared
    here. The tensors, the partial and the workspace must stay alive and at
    the same addresses."""

    def __init__(self, tensors: Sequence[BucketTensor], partial: torch.Tensor, ws: Optional[torch.Tensor] = None):
        self._arr, self._keep, self.M = _cbucket(tensors, check=True)
        self._tensors = list(tensors)
        self.T = len(self._tensors)
        _need(partial, torch.uint8, "partial", BUCKET_PARTIAL_BYTES)
        self._partial = partial
        if ws is None:
            ws = workspace(zero_bucket_step_workspace_bytes(self._tensors, self.M))
        self.ws = ws
        self._wsp, self._wsb = _ptr(ws), _need_ws(ws)

    def step(self, flags: int, hp: HParams, stamp: int, stream=None) -> None:
        h = hp._c()
        st = lib().zero_bucket_step(self._arr, self.T, self.M, flags, ctypes.byref(h), stamp & 0xFFFFFFFFFFFFFFFF,
                                    self._partial.data_ptr(), self._wsp, self._wsb, _stream(stream))
        if st != ZERO_OK:
            raise ZeroError(st, "zero_bucket_step")


# ---------------------------------------------------------------- CPU-offloaded step

@dataclasses.dataclass
class OffloadTensor:
    """One tensor shard of an offloaded step: M bf16 replicas (device), the
    fp32 master/exp_avg/exp_avg_sq in host memory (updated in place) and the
    bf16 output shard (device)."""
    grads: List[torch.Tensor]
    master: torch.Tensor
    exp_avg: torch.Tensor
    exp_avg_sq: torch.Tensor
    param_out: torch.Tensor


def _need_host(t: torch.Tensor, dtype, name: str, n: Optional[int] = None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device.type != "cpu":
        raise ValueError(f"{name}: must be a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")


def _coffload(tensors: Sequence[OffloadTensor], check: bool):
    M = len(tensors[0].grads) if tensors else 1
    keep = []
    arr = (_COffloadTensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        n = t.master.numel()
        if check:
            if len(t.grads) != M:
                raise ValueError(f"tensor {i}: {len(t.grads)} replicas, expected {M}")
            for r, g in enumerate(t.grads):
                _need(g, torch.bfloat16, f"tensors[{i}].grads[{r}]", n)
            for x, nm in ((t.master, "master"), (t.exp_avg, "exp_avg"), (t.exp_avg_sq, "exp_avg_sq")):
                _need_host(x, torch.float32, f"tensors[{i}].{nm}", n)
            _need(t.param_out, torch.bfloat16, f"tensors[{i}].param_out", n)
        ptrs = (ctypes.c_void_p * max(M, 1))(*[g.data_ptr() for g in t.grads])
        keep.append(ptrs)
        arr[i] = _COffloadTensor(n, ctypes.cast(ptrs, ctypes.POINTER(ctypes.c_void_p)), t.master.data_ptr(),
                                 t.exp_avg.data_ptr(), t.exp_avg_sq.data_ptr(), t.param_out.data_ptr())
    return arr, keep, M


def zero_offload_workspace_bytes(tensors: Sequence[OffloadTensor], M: int) -> int:
    arr, keep, _ = _coffload(tensors, check=False)
    return int(lib().zero_offload_workspace_bytes(arr, len(tensors), int(M)))


def zero_offload_host_workspace_bytes(tensors: Sequence[OffloadTensor]) -> int:
    arr, keep, _ = _coffload(tensors, check=False)
    return int(lib().zero_offload_host_workspace_bytes(arr, len(tensors)))


def host_workspace(nbytes: int) -> torch.Tensor:
    """Pinned host memory of nbytes (page-aligned), for zero_offload_step."""
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, pin_memory=True)


def zero_offload_step(tensors: Sequence[OffloadTensor], hp: HParams, external_sumsq: float, ws: torch.Tensor,
                      host_ws: torch.Tensor, threads: int = 0, stream=None) -> dict:
    """Returns the result record (the call reads it on the host)."""
    _need(ws, torch.uint8, "ws")
    _need_host(host_ws, torch.uint8, "host_ws")
    if not host_ws.is_pinned():
        raise ValueError("host_ws: must be pinned host memory (host_workspace())")
    arr, keep, M = _coffload(tensors, check=True)
    h = hp._c()
    r = _CResult()
    _check(lib().zero_offload_step(arr, len(tensors), M, ctypes.byref(h), float(external_sumsq), ws.data_ptr(),
                                   ws.numel(), host_ws.data_ptr(), host_ws.numel(), ctypes.byref(r), int(threads),
                                   _stream(stream)), "zero_offload_step")
    return dict(sumsq=r.sumsq, grad_norm=r.grad_norm, clip_coef=r.clip_coef, found_inf=r.found_inf,
                skipped=r.skipped, status=r.status)


def zero_offload_adamw_host(master: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor, g: torch.Tensor,
                            param_out: torch.Tensor, hp: HParams, clip_coef: float = 1.0, threads: int = 0) -> None:
    """The host half of the offloaded step on host tensors (fp32 state and
    gradient, bf16 output)."""
    n = master.numel()
    for t, nm in ((master, "master"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq"), (g, "g")):
        _need_host(t, torch.float32, nm, n)
    _need_host(param_out, torch.bfloat16, "param_out", n)
    h = hp._c()
    _check(lib().zero_offload_adamw_host(master.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), g.data_ptr(),
                                         param_out.data_ptr(), n, ctypes.byref(h), float(clip_coef), int(threads)),
           "zero_offload_adamw_host")


def zero_step_accumulated_amp(tensors: Sequence[AccTensor], hp: HParams, cfg: "LossScaleConfig", ls: torch.Tensor,
                              partials: Optional[torch.Tensor], nbuckets: int, stamp: int, external_sumsq: float,
                              ws: Optional[torch.Tensor], res: torch.Tensor, stream=None) -> None:
    _need(res, torch.uint8, "res", RESULT_BYTES)
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    if nbuckets > 0:
        _need(partials, torch.uint8, "partials")
        if partials.numel() < nbuckets * BUCKET_PARTIAL_BYTES:
            raise ValueError(f"partials: {partials.numel()} bytes for {nbuckets} buckets")
    arr = _cacc(tensors, check=True)
    h = hp._c()
    c = cfg._c()
    wsb = _need_ws(ws)
    _check(lib().zero_step_accumulated_amp(arr, len(tensors), ctypes.byref(h), ctypes.byref(c), ls.data_ptr(),
                                           _ptr(partials), int(nbuckets), int(stamp) & (2**64 - 1),
                                           float(external_sumsq), _ptr(ws), wsb, res.data_ptr(), _stream(stream)),
           "zero_step_accumulated_amp")


def zero_offload_step_amp(tensors: Sequence[OffloadTensor], hp: HParams, cfg: "LossScaleConfig", ls: torch.Tensor,
                          external_sumsq: float, ws: torch.Tensor, host_ws: torch.Tensor, threads: int = 0,
                          stream=None) -> dict:
    _need(ws, torch.uint8, "ws")
    _need_host(host_ws, torch.uint8, "host_ws")
    if not host_ws.is_pinned():
        raise ValueError("host_ws: must be pinned host memory (host_workspace())")
    _need(ls, torch.uint8, "ls", LOSS_SCALE_BYTES)
    arr, keep, M = _coffload(tensors, check=True)
    h = hp._c()
    c = cfg._c()
    r = _CResult()
    _check(lib().zero_offload_step_amp(arr, len(tensors), M, ctypes.byref(h), ctypes.byref(c), ls.data_ptr(),
                                       float(external_sumsq), ws.data_ptr(), ws.numel(), host_ws.data_ptr(),
                                       host_ws.numel(), ctypes.byref(r), int(threads), _stream(stream)),
           "zero_offload_step_amp")
    return dict(sumsq=r.sumsq, grad_norm=r.grad_norm, clip_coef=r.clip_coef, found_inf=r.found_inf,
                skipped=r.skipped, status=r.status)


# ---------------------------------------------------------------- around a training block

_DTYPES = {torch.bfloat16: 1, torch.float32: 2}  # ZERO_BF16, ZERO_F32


@dataclasses.dataclass
class Act8:
    """Rows of activations in 8 bits: rows x cols codes (ACT8_E4M3 or
    ACT8_INT8) with a power-of-two scale for each 32 columns, in one device
    buffer of zero_act8_bytes(rows, cols) bytes whose layout
    include/zero_step.h gives."""
    rows: int
    cols: int
    format: int
    buf: torch.Tensor


def zero_act8_bytes(rows: int, cols: int) -> int:
    return int(lib().zero_act8_bytes(int(rows), int(cols)))


def new_act8(rows: int, cols: int, format: int = ACT8_E4M3, device=None) -> Act8:
    """An empty checkpoint of rows x cols."""
    n = zero_act8_bytes(rows, cols)
    if n == 0 and rows != 0 and cols != 0:
        raise ValueError(f"no checkpoint of {rows} x {cols}")
    return Act8(rows, cols, format, torch.empty(n, dtype=torch.uint8, device=device or "cuda"))


# Marshalling of these calls: their operands are many and some of their
# launches short, so it reads each tensor's attributes once and packs the C
# structures in one step (a zero_rows is data, ld, dtype, reserved).
_ROWS = struct.Struct("=QqiI")
_BLOCK_NORM = struct.Struct("=qqqdd" + "QqiI" * 7 + "QQQQii")
_BLOCK_NORM_GRAD = struct.Struct("=qqqd" + "QqiI" * 7 + "QQQQ" + "QqiI" * 5 + "ii")
_LAYER_NORM = struct.Struct("=qqd" + "QqiI" * 6 + "QQQQii")
_LAYER_NORM_GRAD = struct.Struct("=qq" + "QqiI" * 4 + "QQQ" + "QqiI" * 4 + "ii")
_BLOCK_FFN = struct.Struct("=qqq" + "QqiI" * 6 + "QQii")
_BLOCK_FFN_GRAD = struct.Struct("=qqq" + "QqiI" * 3 + "QQ" + "QqiI" * 3 + "Q" + "QqiI" * 6 + "Qiiii")
_ABSENT = (0, 0, 0, 0)


def _on(t, name: str, dev: int):
    """Refuses what is not a tensor on device dev."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on device {t.get_device()}, the current device is {dev}")


def _matrix(t, name: str):
    """The shape of a call's first operand, and the current device, which it has to be on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got {t.dim()} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    return *t.shape, torch.cuda.current_device()


def _row_major(t, name: str, rows: int, cols: int, dev: int, only=None):
    """A row-major matrix of any row stride (a vector is one row) as the
    fields of a zero_rows. None: absent."""
    if t is None:
        return _ABSENT
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    dtype = t.dtype
    if t.shape == (rows, cols) and t.is_contiguous() and (dtype is only if only is not None else dtype in _DTYPES):
        return t.data_ptr(), cols, _DTYPES[dtype], 0  # most operands, in fewer steps than the checks below
    if dtype not in _DTYPES or (only is not None and dtype is not only):
        raise TypeError(f"{name}: expected {only or 'torch.bfloat16 or torch.float32'}, got {dtype}")
    dim = t.dim()
    if dim == 2:
        r, c = t.shape
        ld, step = t.stride()
    elif dim == 1:
        r, (c,), ld, (step,) = 1, t.shape, 0, t.stride()
    else:
        r = c = -1
    if r != rows or c != cols:
        raise ValueError(f"{name}: expected {(rows, cols)}, got {tuple(t.shape)}")
    if step != 1 and c > 1:
        raise ValueError(f"{name}: the elements of a row must lie next to each other")
    if r <= 1:
        ld = c
    elif ld < c:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld, _DTYPES[dtype], 0


def _vector(t, name: str, cols: int, dev: int):
    """A row of cols elements, as one dimension or a matrix of one row."""
    if t is None:
        return _ABSENT
    if isinstance(t, torch.Tensor) and t.shape == (cols,) and t.get_device() == dev and t.is_contiguous():
        dtype = t.dtype
        if dtype in _DTYPES:
            return t.data_ptr(), cols, _DTYPES[dtype], 0
    return _row_major(t, name, 1, cols, dev)


def _per_row(t, name: str, rows: int, dev: int) -> int:
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    if t.shape != (rows,) or t.dtype is not torch.float32 or not t.is_contiguous():
        _need(t, torch.float32, name, rows)
    return t.data_ptr()


def _act8(c, name: str, rows: int, cols: int, dev: int) -> int:
    if c is None:
        return 0
    if not isinstance(c, Act8):
        raise TypeError(f"{name}: expected an Act8")
    if c.rows != rows or c.cols != cols:
        raise ValueError(f"{name}: holds {c.rows} x {c.cols}, expected {rows} x {cols}")
    t = c.buf
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _on(t, name, dev)
    if t.dtype is not torch.uint8 or not t.is_contiguous():
        _need(t, torch.uint8, name)
    if t.numel() < rows * -(-cols // 32) * 33:
        raise ValueError(f"{name}: {t.numel()} bytes for {rows} x {cols}")
    return t.data_ptr()


def _workspace_of(ws, dev: int):
    if ws is None:
        return None, 0
    n = _need_ws(ws)
    _on(ws, "ws", dev)
    return ws.data_ptr(), n


def _stream_of(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: of device {stream.device_index}, the current device is {dev}")
    return int(stream.cuda_stream)


def _checkpoint(c) -> Act8:
    if not isinstance(c, Act8):
        raise TypeError("ckpt: expected an Act8")
    return c


def zero_act8_save(x: torch.Tensor, ckpt: Act8, stream=None) -> None:
    rows, cols, dev = _matrix(x, "x")
    st = lib().zero_act8_save(_ROWS.pack(*_row_major(x, "x", rows, cols, dev)), rows, cols, int(_checkpoint(ckpt).format),
                              _act8(ckpt, "ckpt", rows, cols, dev), _stream_of(stream, dev))
    _check(st, "zero_act8_save")


def zero_act8_load(ckpt: Act8, out: torch.Tensor, stream=None) -> None:
    rows, cols, dev = _matrix(out, "out")
    st = lib().zero_act8_load(_act8(_checkpoint(ckpt), "ckpt", rows, cols, dev), rows, cols, int(ckpt.format),
                              _ROWS.pack(*_row_major(out, "out", rows, cols, dev)), _stream_of(stream, dev))
    _check(st, "zero_act8_load")


def zero_act8_wgrad_workspace_bytes(rows: int, outs: int, cols: int) -> int:
    return int(lib().zero_act8_wgrad_workspace_bytes(int(rows), int(outs), int(cols)))


def zero_act8_wgrad(dy: torch.Tensor, ckpt: Act8, dw: torch.Tensor, flags: int = 0, ws: Optional[torch.Tensor] = None,
                    col_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """dw (outs x cols, bf16 or fp32) = dy^T times the checkpoint's rows, its
    columns times col_scale; with GRAD_ACCUMULATE added to an fp32 dw."""
    rows, outs, dev = _matrix(dy, "dy")
    cols = int(_checkpoint(ckpt).cols)
    wsp, wsb = _workspace_of(ws, dev)
    scale = None if col_scale is None else _ROWS.pack(*_vector(col_scale, "col_scale", cols, dev))
    st = lib().zero_act8_wgrad(_ROWS.pack(*_row_major(dy, "dy", rows, outs, dev, torch.bfloat16)),
                               _act8(ckpt, "ckpt", rows, cols, dev), rows, outs, cols, int(ckpt.format), scale,
                               _ROWS.pack(*_row_major(dw, "dw", outs, cols, dev)), int(flags), wsp, wsb,
                               _stream_of(stream, dev))
    _check(st, "zero_act8_wgrad")


@dataclasses.dataclass
class BlockNorm:
    """The operands of zero_block_norm; None is an absent one. x and x_out:
    the residual stream (bf16 or fp32); y and h: bf16; w_post, gate and w_pre:
    bf16 or fp32; rstd_*: fp32; ckpt_*: Act8 of one format. gate has a row for
    every gate_rows rows."""
    x: torch.Tensor
    y: Optional[torch.Tensor] = None
    w_post: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    w_pre: Optional[torch.Tensor] = None
    x_out: Optional[torch.Tensor] = None
    h: Optional[torch.Tensor] = None
    rstd_post: Optional[torch.Tensor] = None
    rstd_pre: Optional[torch.Tensor] = None
    ckpt_post: Optional[Act8] = None
    ckpt_pre: Optional[Act8] = None
    gate_rows: int = 0
    residual_scale: float = 1.0
    eps: float = 1e-6


@dataclasses.dataclass
class BlockNormGrad:
    """The operands of zero_block_norm_grad; None is an absent one. Saved rows
    come from ckpt_* or, without one, from x_out and y."""
    dx: torch.Tensor
    dx_out: Optional[torch.Tensor] = None
    dh: Optional[torch.Tensor] = None
    w_post: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    w_pre: Optional[torch.Tensor] = None
    x_out: Optional[torch.Tensor] = None
    y: Optional[torch.Tensor] = None
    ckpt_pre: Optional[Act8] = None
    ckpt_post: Optional[Act8] = None
    rstd_pre: Optional[torch.Tensor] = None
    rstd_post: Optional[torch.Tensor] = None
    dy: Optional[torch.Tensor] = None
    dw_pre: Optional[torch.Tensor] = None
    dw_post: Optional[torch.Tensor] = None
    dgate: Optional[torch.Tensor] = None
    gate_rows: int = 0
    residual_scale: float = 1.0


def _act8_format(a: Optional[Act8], b: Optional[Act8]) -> int:
    if a is not None and b is not None and a.format != b.format:
        raise ValueError("ckpt_post and ckpt_pre have different formats")
    c = a if a is not None else b
    return 0 if c is None else int(c.format)


def _gates(rows: int, gate_rows: int) -> int:
    if gate_rows < 1:
        raise ValueError(f"gate_rows: {gate_rows} with a gate")
    return -(-rows // gate_rows)


def zero_block_norm(b: BlockNorm, stream=None) -> None:
    rows, cols, dev = _matrix(b.x, "x")
    bf16 = torch.bfloat16
    gate = _ABSENT if b.gate is None else _row_major(b.gate, "gate", _gates(rows, b.gate_rows), cols, dev)
    args = _BLOCK_NORM.pack(
        rows, cols, b.gate_rows, b.residual_scale, b.eps, *_row_major(b.x, "x", rows, cols, dev),
        *_row_major(b.y, "y", rows, cols, dev, bf16), *_vector(b.w_post, "w_post", cols, dev), *gate,
        *_vector(b.w_pre, "w_pre", cols, dev), *_row_major(b.x_out, "x_out", rows, cols, dev, b.x.dtype),
        *_row_major(b.h, "h", rows, cols, dev, bf16), _per_row(b.rstd_post, "rstd_post", rows, dev),
        _per_row(b.rstd_pre, "rstd_pre", rows, dev), _act8(b.ckpt_post, "ckpt_post", rows, cols, dev),
        _act8(b.ckpt_pre, "ckpt_pre", rows, cols, dev), _act8_format(b.ckpt_post, b.ckpt_pre), 0)
    _check(lib().zero_block_norm(args, _stream_of(stream, dev)), "zero_block_norm")


def zero_block_norm_grad_workspace_bytes(rows: int, cols: int, gate_rows: int) -> int:
    """gate_rows: 0 without a gate."""
    return int(lib().zero_block_norm_grad_workspace_bytes(int(rows), int(cols), int(gate_rows)))


def zero_block_norm_grad(b: BlockNormGrad, flags: int = 0, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    rows, cols, dev = _matrix(b.dx, "dx")
    bf16, like = torch.bfloat16, b.dx.dtype
    gates = 0 if b.gate is None else _gates(rows, b.gate_rows)
    wsp, wsb = _workspace_of(ws, dev)
    args = _BLOCK_NORM_GRAD.pack(
        rows, cols, b.gate_rows, b.residual_scale, *_row_major(b.dh, "dh", rows, cols, dev, bf16),
        *_row_major(b.dx_out, "dx_out", rows, cols, dev, like), *_vector(b.w_post, "w_post", cols, dev),
        *_row_major(b.gate, "gate", gates, cols, dev), *_vector(b.w_pre, "w_pre", cols, dev),
        *_row_major(b.x_out, "x_out", rows, cols, dev, like), *_row_major(b.y, "y", rows, cols, dev, bf16),
        _act8(b.ckpt_pre, "ckpt_pre", rows, cols, dev), _act8(b.ckpt_post, "ckpt_post", rows, cols, dev),
        _per_row(b.rstd_pre, "rstd_pre", rows, dev), _per_row(b.rstd_post, "rstd_post", rows, dev),
        *_row_major(b.dx, "dx", rows, cols, dev), *_row_major(b.dy, "dy", rows, cols, dev, bf16),
        *_vector(b.dw_pre, "dw_pre", cols, dev), *_vector(b.dw_post, "dw_post", cols, dev),
        *_row_major(b.dgate, "dgate", gates, cols, dev), _act8_format(b.ckpt_post, b.ckpt_pre), flags)
    _check(lib().zero_block_norm_grad(args, wsp, wsb, _stream_of(stream, dev)), "zero_block_norm_grad")


@dataclasses.dataclass
class LayerNorm:
    """The operands of zero_layer_norm; None is an absent one. x and x_out: the
    residual stream (bf16 or fp32); y and h: bf16; w and b: bf16 or fp32; mean
    and rstd: fp32; ckpt_*: Act8 of one format."""
    x: torch.Tensor
    h: torch.Tensor
    y: Optional[torch.Tensor] = None
    w: Optional[torch.Tensor] = None
    b: Optional[torch.Tensor] = None
    x_out: Optional[torch.Tensor] = None
    mean: Optional[torch.Tensor] = None
    rstd: Optional[torch.Tensor] = None
    ckpt_xn: Optional[Act8] = None
    ckpt_h: Optional[Act8] = None
    eps: float = 1e-5


@dataclasses.dataclass
class LayerNormGrad:
    """The operands of zero_layer_norm_grad; None is an absent one. The
    normalised rows come from ckpt_xn or, without it, from x_out and mean."""
    dx: torch.Tensor
    dh: torch.Tensor
    rstd: torch.Tensor
    dx_out: Optional[torch.Tensor] = None
    w: Optional[torch.Tensor] = None
    x_out: Optional[torch.Tensor] = None
    mean: Optional[torch.Tensor] = None
    ckpt_xn: Optional[Act8] = None
    dy: Optional[torch.Tensor] = None
    dw: Optional[torch.Tensor] = None
    db: Optional[torch.Tensor] = None


def zero_layer_norm(b: LayerNorm, stream=None) -> None:
    rows, cols, dev = _matrix(b.x, "x")
    bf16 = torch.bfloat16
    args = _LAYER_NORM.pack(
        rows, cols, b.eps, *_row_major(b.x, "x", rows, cols, dev), *_row_major(b.y, "y", rows, cols, dev, bf16),
        *_vector(b.w, "w", cols, dev), *_vector(b.b, "b", cols, dev),
        *_row_major(b.x_out, "x_out", rows, cols, dev, b.x.dtype), *_row_major(b.h, "h", rows, cols, dev, bf16),
        _per_row(b.mean, "mean", rows, dev), _per_row(b.rstd, "rstd", rows, dev),
        _act8(b.ckpt_xn, "ckpt_xn", rows, cols, dev), _act8(b.ckpt_h, "ckpt_h", rows, cols, dev),
        _act8_format(b.ckpt_xn, b.ckpt_h), 0)
    _check(lib().zero_layer_norm(args, _stream_of(stream, dev)), "zero_layer_norm")


def zero_layer_norm_grad_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().zero_layer_norm_grad_workspace_bytes(int(rows), int(cols)))


def zero_layer_norm_grad(b: LayerNormGrad, flags: int = 0, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    rows, cols, dev = _matrix(b.dx, "dx")
    bf16, like = torch.bfloat16, b.dx.dtype
    wsp, wsb = _workspace_of(ws, dev)
    args = _LAYER_NORM_GRAD.pack(
        rows, cols, *_row_major(b.dh, "dh", rows, cols, dev, bf16), *_row_major(b.dx_out, "dx_out", rows, cols, dev, like),
        *_vector(b.w, "w", cols, dev), *_row_major(b.x_out, "x_out", rows, cols, dev, like),
        _per_row(b.mean, "mean", rows, dev), _per_row(b.rstd, "rstd", rows, dev),
        _act8(b.ckpt_xn, "ckpt_xn", rows, cols, dev), *_row_major(b.dx, "dx", rows, cols, dev),
        *_row_major(b.dy, "dy", rows, cols, dev, bf16), *_vector(b.dw, "dw", cols, dev), *_vector(b.db, "db", cols, dev),
        _act8_format(b.ckpt_xn, None), flags)
    _check(lib().zero_layer_norm_grad(args, wsp, wsb, _stream_of(stream, dev)), "zero_layer_norm_grad")


@dataclasses.dataclass
class BlockFfn:
    """The operands of zero_block_ffn, all bf16; None is an absent one. gate
    and up, or ckpt_gate and ckpt_up (Act8 of one format): what the backward
    pass reads. act: FFN_SILU, FFN_GELU or FFN_GELU_TANH."""
    h: torch.Tensor
    w_gate: torch.Tensor
    w_up: torch.Tensor
    a: torch.Tensor
    gate: Optional[torch.Tensor] = None
    up: Optional[torch.Tensor] = None
    ckpt_gate: Optional[Act8] = None
    ckpt_up: Optional[Act8] = None
    act: int = FFN_SILU


@dataclasses.dataclass
class BlockFfnGrad:
    """The operands of zero_block_ffn_grad; None is an absent one. The saved
    gate and up come as bf16 rows or Act8, and so does the block's input (h, or
    ckpt_h with col_scale); all Act8 are of one format. dw_gate and dw_up: bf16
    or fp32."""
    da: torch.Tensor
    dgate: torch.Tensor
    dup: torch.Tensor
    gate: Optional[torch.Tensor] = None
    up: Optional[torch.Tensor] = None
    ckpt_gate: Optional[Act8] = None
    ckpt_up: Optional[Act8] = None
    w_gate: Optional[torch.Tensor] = None
    w_up: Optional[torch.Tensor] = None
    dh: Optional[torch.Tensor] = None
    h: Optional[torch.Tensor] = None
    ckpt_h: Optional[Act8] = None
    col_scale: Optional[torch.Tensor] = None
    dw_gate: Optional[torch.Tensor] = None
    dw_up: Optional[torch.Tensor] = None
    ckpt_a: Optional[Act8] = None
    act: int = FFN_SILU


def zero_block_ffn_workspace_bytes(rows: int, cols: int, hidden: int) -> int:
    return int(lib().zero_block_ffn_workspace_bytes(int(rows), int(cols), int(hidden)))


def zero_block_ffn(b: BlockFfn, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    rows, cols, dev = _matrix(b.h, "h")
    hidden = _matrix(b.w_gate, "w_gate")[0]
    bf16 = torch.bfloat16
    wsp, wsb = _workspace_of(ws, dev)
    args = _BLOCK_FFN.pack(
        rows, cols, hidden, *_row_major(b.h, "h", rows, cols, dev, bf16),
        *_row_major(b.w_gate, "w_gate", hidden, cols, dev, bf16), *_row_major(b.w_up, "w_up", hidden, cols, dev, bf16),
        *_row_major(b.a, "a", rows, hidden, dev, bf16), *_row_major(b.gate, "gate", rows, hidden, dev, bf16),
        *_row_major(b.up, "up", rows, hidden, dev, bf16), _act8(b.ckpt_gate, "ckpt_gate", rows, hidden, dev),
        _act8(b.ckpt_up, "ckpt_up", rows, hidden, dev), _act8_format(b.ckpt_gate, b.ckpt_up), b.act)
    _check(lib().zero_block_ffn(args, wsp, wsb, _stream_of(stream, dev)), "zero_block_ffn")


def zero_block_ffn_grad_workspace_bytes(rows: int, cols: int, hidden: int) -> int:
    return int(lib().zero_block_ffn_grad_workspace_bytes(int(rows), int(cols), int(hidden)))


def _ffn_cols(b: BlockFfnGrad) -> int:
    """The width of the block's input, from the operands that have it."""
    for t in (b.dh, b.dw_gate, b.dw_up):
        if t is not None:
            return _matrix(t, "dh, dw_gate or dw_up")[1]
    return 0


def zero_block_ffn_grad(b: BlockFfnGrad, flags: int = 0, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    rows, hidden, dev = _matrix(b.da, "da")
    cols = _ffn_cols(b)
    bf16 = torch.bfloat16
    wsp, wsb = _workspace_of(ws, dev)
    wide = lambda t, name: _row_major(t, name, rows, hidden, dev, bf16)  # noqa: E731
    args = _BLOCK_FFN_GRAD.pack(
        rows, cols, hidden, *wide(b.da, "da"), *wide(b.gate, "gate"), *wide(b.up, "up"),
        _act8(b.ckpt_gate, "ckpt_gate", rows, hidden, dev), _act8(b.ckpt_up, "ckpt_up", rows, hidden, dev),
        *_row_major(b.w_gate, "w_gate", hidden, cols, dev, bf16), *_row_major(b.w_up, "w_up", hidden, cols, dev, bf16),
        *_row_major(b.h, "h", rows, cols, dev, bf16), _act8(b.ckpt_h, "ckpt_h", rows, cols, dev),
        *_vector(b.col_scale, "col_scale", cols, dev), *wide(b.dgate, "dgate"), *wide(b.dup, "dup"),
        *_row_major(b.dh, "dh", rows, cols, dev, bf16), *_row_major(b.dw_gate, "dw_gate", hidden, cols, dev),
        *_row_major(b.dw_up, "dw_up", hidden, cols, dev), _act8(b.ckpt_a, "ckpt_a", rows, hidden, dev),
        _one_format(b.ckpt_gate, b.ckpt_up, b.ckpt_h, b.ckpt_a), b.act, flags, 0)
    _check(lib().zero_block_ffn_grad(args, wsp, wsb, _stream_of(stream, dev)), "zero_block_ffn_grad")


def _one_format(*checkpoints: Optional[Act8]) -> int:
    formats = {int(c.format) for c in checkpoints if c is not None}
    if len(formats) > 1:
        raise ValueError("the checkpoints have different formats")
    return formats.pop() if formats else 0


def zero_workspace_forget(ws: torch.Tensor) -> None:
    _check(lib().zero_workspace_forget(ws.data_ptr()), "zero_workspace_forget")


def workspace(nbytes: int, device=None) -> Optional[torch.Tensor]:
    """A device workspace of nbytes (torch allocations are 256-byte aligned).
    When the tensor is freed, the library forgets any plan it cached there:
    the allocator may hand the same memory out again for something else."""
    if nbytes <= 0:
        return None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device or "cuda")
    weakref.finalize(ws, _forget_ptr, ws.data_ptr())
    return ws


def _forget_ptr(ptr: int) -> None:
    if _lib is not None:
        _lib.zero_workspace_forget(ptr)


def zero_step_workspace_bytes_for_sizes(sizes: Sequence[int], M: int, hp: HParams) -> int:
    """Workspace size of a zero_step over shards of these lengths (no tensors needed)."""
    arr = (_CTensor * max(len(sizes), 1))()
    for i, n in enumerate(sizes):
        arr[i] = _CTensor(int(n), None, None, None, None, None)
    h = hp._c()
    return int(lib().zero_step_workspace_bytes(arr, len(sizes), int(M), ctypes.byref(h)))
