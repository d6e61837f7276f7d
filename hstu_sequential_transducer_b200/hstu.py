"""Thin Python binding of libhstu.so (include/hstu.h).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  If
the library is missing this module raises on first use; there is no
fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from ctypes import POINTER, Structure, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# HSTU_DEBUG_BUILD=1 loads the debug build (-DHSTU_DEBUG: index checks on the
# attention kernels' direct global accesses, reported as HSTU_DEVICE_BOUNDS)
DEBUG_BUILD = os.environ.get("HSTU_DEBUG_BUILD") == "1"
LIB_PATH = os.path.join(_HERE, "libhstu_debug.so" if DEBUG_BUILD else "libhstu.so")

HSTU_F32, HSTU_BF16 = 0, 1
SAVED_PRE, SAVED_G, SAVED_O, SAVED_Z, SAVED_MEAN, SAVED_RSTD, SAVED_XLOW, SAVED_COUNT = range(8)
K_PROJ_IN, K_ATTN_FWD, K_LN_FWD, K_PROJ_OUT, K_PROJ_OUT_BWD, K_LN_BWD, K_ATTN_BWD, \
    K_PROJ_IN_BWD, K_ATTN_CACHED, K_MISC, K_SOFTMAX, K_EMBED, K_BLOCK_NORM, K_CHECKPOINT, \
    K_COUNT = range(15)
KERNEL_NAMES = ["proj_in", "attn_fwd", "ln_fwd", "proj_out", "proj_out_bwd", "ln_bwd",
                "attn_bwd", "proj_in_bwd", "attn_cached", "misc", "softmax_fwd", "embed",
                "block_norm", "checkpoint"]
NORM_NONE, NORM_LAYER, NORM_RMS = range(3)
GATE_NONE, GATE_SIGMOID, GATE_SILU = range(3)
CKPT_INT8, CKPT_E4M3 = range(2)
CKPT_PRE, CKPT_DEV, CKPT_X, CKPT_PRE_SCALE, CKPT_DEV_SCALE, CKPT_X_SCALE, CKPT_MEAN, CKPT_RSTD, \
    CKPT_COUNT = range(9)

FLAG_OFFSETS_START, FLAG_OFFSETS_ORDER, FLAG_OFFSETS_END = 0x1, 0x2, 0x4
FLAG_SEQ_TOO_LONG, FLAG_TARGETS_RANGE, FLAG_TIME_ORDER = 0x8, 0x10, 0x20


class Config(Structure):
    _fields_ = [("d_model", c_int32), ("num_heads", c_int32), ("head_dim", c_int32),
                ("num_pos_buckets", c_int32), ("num_time_buckets", c_int32),
                ("max_seq_len", c_int32), ("norm_N", c_float), ("ln_eps", c_float),
                ("dtype", c_int32), ("io_dtype", c_int32)]


class Weights(Structure):
    _fields_ = [("W1", c_void_p), ("b1", c_void_p), ("W2", c_void_p), ("b2", c_void_p),
                ("ln_gamma", c_void_p), ("ln_beta", c_void_p), ("rab_pos", c_void_p),
                ("rab_time", c_void_p)]


class Grads(Structure):
    _fields_ = [("dW1", c_void_p), ("db1", c_void_p), ("dW2", c_void_p), ("db2", c_void_p),
                ("dgamma", c_void_p), ("dbeta", c_void_p), ("drab_pos", c_void_p),
                ("drab_time", c_void_p)]


class CBlockNorm(Structure):
    _fields_ = [("post_kind", c_int32), ("pre_kind", c_int32), ("gate_act", c_int32),
                ("reserved", c_int32), ("post_gamma", c_void_p), ("post_beta", c_void_p),
                ("res_scale", c_void_p), ("pre_gamma", c_void_p), ("pre_beta", c_void_p)]


class CBlockNormGrads(Structure):
    _fields_ = [("post_gamma", c_void_p), ("post_beta", c_void_p), ("res_scale", c_void_p),
                ("pre_gamma", c_void_p), ("pre_beta", c_void_p)]


class HSTUError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


_lib = None
V, S, I32, I64, P = c_void_p, c_size_t, c_int32, c_int64, c_void_p
_CP = POINTER(Config)
_WP = POINTER(Weights)
_GP = POINTER(Grads)

_SIGS = {
    "hstu_workspace_size": (I32, [_CP, I32, I64, POINTER(c_size_t), POINTER(c_size_t)]),
    "hstu_saved_layout": (I32, [_CP, I64, POINTER(c_size_t)]),
    "hstu_proj_in_fwd": (I32, [_CP, _WP, P, I64, P, P, P]),
    "hstu_attention_fwd": (I32, [_CP, P, P, P, P, I32, I64, P, P, P, P, S, P]),
    "hstu_attention_fwd_cached": (I32, [_CP, P, P, P, P, I32, I64, P, P, P, I64, P, P, P, S, P]),
    "hstu_attention_workspace_size": (S, [_CP, I32, I64]),
    "hstu_softmax_attention_fwd": (I32, [_CP, P, P, P, P, I32, I64, P, P, P, P, S, P]),
    "hstu_attention_fwd_noalloc": (I32, [_CP, P, P, P, P, I32, I64, P, P, P, P]),
    "hstu_ln_gate_fwd": (I32, [_CP, P, P, P, P, I64, P, P, P, P]),
    "hstu_proj_out_fwd": (I32, [_CP, P, P, P, P, I64, P, P]),
    "hstu_proj_out_bwd": (I32, [_CP, P, P, P, I64, P, P, P, P]),
    "hstu_ln_gate_bwd": (I32, [_CP, P, P, P, P, P, P, P, P, I64, P, P, P, P, P]),
    "hstu_attention_bwd": (I32, [_CP, P, P, P, P, P, P, I32, I64, P, P, P, P, P, P, S, P]),
    "hstu_attention_bwd_workspace_size": (S, [_CP, I32, I64]),
    "hstu_proj_in_bwd": (I32, [_CP, P, P, P, P, I64, P, P, P, P]),
    "hstu_fwd": (I32, [_CP, _WP, P, P, I32, I64, P, P, P, P, P, P, S, P]),
    "hstu_fwd_cached": (I32, [_CP, _WP, P, P, I32, I64, P, P, P, I64, P, P, P, S, P]),
    "hstu_bwd": (I32, [_CP, _WP, P, P, P, P, I32, I64, P, P, P, _GP, P, S, P]),
    "hstu_fwd_chain": (I32, [_CP, _WP, P, P, P, I32, I64, P, P, P, P, P, P, P, S, P]),
    "hstu_bwd_chain": (I32, [_CP, _WP, P, P, P, P, P, I32, I64, P, P, P, P, _GP, P, S, P]),
    "hstu_validate_inputs": (I32, [P, I32, I64, P, P, I32, P, P]),
    "hstu_sl_subsequence_length": (I64, [I64, c_double]),
    "hstu_stochastic_length": (I32, [P, P, I32, I64, I64, P, P, P, P, P]),
    "hstu_gather_rows": (I32, [P, I64, I64, P, P, I64, I64, P, I64, P]),
    "hstu_embedding_fwd": (I32, [P, I32, I64, I32, I64, P, I32, I64, c_float, P, I32, I32, I64, P,
                                 I64, P]),
    "hstu_embedding_bwd_workspace_size": (S, [I64, I64, I32]),
    "hstu_embedding_bwd": (I32, [P, I32, I64, P, I32, I64, I64, I32, c_float, P, I64, P, S, P]),
    "hstu_embedding_bwd_rows": (I32, [P, I32, I64, P, I32, I64, I64, I32, c_float, P, P, I64, P, P,
                                      S, P]),
    "hstu_block_norm_fwd": (I32, [_CP, POINTER(CBlockNorm), P, P, P, I64, I64, P, P, P, P]),
    "hstu_block_norm_bwd": (I32, [_CP, POINTER(CBlockNorm), P, P, P, I64, P, P, P, I64, P, P, P,
                                  I64, POINTER(CBlockNormGrads), P, S, P]),
    "hstu_block_norm_bwd_workspace_size": (S, [_CP, I64]),
    "hstu_checkpoint_layout": (I32, [_CP, I64, POINTER(c_size_t)]),
    "hstu_checkpoint_save": (I32, [_CP, I32, P, I64, P, P]),
    "hstu_checkpoint_restore": (I32, [_CP, I32, P, P, P, I64, P, P]),
    "hstu_profiler_enable": (None, [I32]),
    "hstu_nvtx_enable": (None, [I32]),
    "hstu_profiler_collect": (I32, [I32, POINTER(c_int64), POINTER(c_double)]),
    "hstu_profiler_reset": (None, []),
    "hstu_launch_count": (I64, []),
    "hstu_device_status": (I32, [POINTER(c_uint32), I32, P]),
    "hstu_selftest_wait_timeout": (I32, [ctypes.c_uint64, P, P]),
    "hstu_status_string": (c_char_p, [I32]),
    "hstu_version": (c_char_p, []),
}


def lib():
    """Loads libhstu.so (built by hstu_sequential_transducer_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m "
                               "hstu_sequential_transducer_b200.build"
                               f"{' --debug' if DEBUG_BUILD else ''}` first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols() -> Sequence[str]:
    return list(_SIGS)


def status_string(s: int) -> str:
    return lib().hstu_status_string(int(s)).decode()


def _check(s: int, where: str):
    if s != 0:
        raise HSTUError(s, where)


def ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return t.data_ptr()


# The current stream's handle: torch.cuda.current_stream() makes a Stream object
# of it at every call, which takes as long as the launch itself.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def stream_ptr(stream: Optional[torch.cuda.Stream] = None):
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def torch_dtype(dtype: int):
    return torch.bfloat16 if dtype == HSTU_BF16 else torch.float32


def make_config(d_model: int, num_heads: int, norm_N: float, dtype: int = HSTU_BF16,
                num_pos_buckets: int = 32, num_time_buckets: int = 32, max_seq_len: int = 8192,
                ln_eps: float = 1e-5, io_dtype: Optional[int] = None) -> Config:
    """io_dtype (x, y, dy, dx) defaults to fp32: a bf16 layer then keeps its
    residual stream in fp32 and only the contraction operands are bf16."""
    io = HSTU_F32 if io_dtype is None else io_dtype
    return Config(d_model, num_heads, d_model // num_heads, num_pos_buckets, num_time_buckets,
                  max_seq_len, float(norm_N), float(ln_eps), dtype, io)


@dataclass
class LayerWeights:
    """Device tensors of one layer (dtype of the config; rab tables fp32)."""
    W1: torch.Tensor
    W2: torch.Tensor
    rab_pos: Optional[torch.Tensor] = None
    rab_time: Optional[torch.Tensor] = None
    b1: Optional[torch.Tensor] = None
    b2: Optional[torch.Tensor] = None
    ln_gamma: Optional[torch.Tensor] = None
    ln_beta: Optional[torch.Tensor] = None

    def c(self) -> Weights:
        return Weights(ptr(self.W1), ptr(self.b1), ptr(self.W2), ptr(self.b2), ptr(self.ln_gamma),
                       ptr(self.ln_beta), ptr(self.rab_pos), ptr(self.rab_time))


@dataclass
class LayerGradBufs:
    dW1: Optional[torch.Tensor] = None
    dW2: Optional[torch.Tensor] = None
    db1: Optional[torch.Tensor] = None
    db2: Optional[torch.Tensor] = None
    dgamma: Optional[torch.Tensor] = None
    dbeta: Optional[torch.Tensor] = None
    drab_pos: Optional[torch.Tensor] = None
    drab_time: Optional[torch.Tensor] = None

    @staticmethod
    def zeros_like(w: LayerWeights, device) -> "LayerGradBufs":
        z = lambda t: None if t is None else torch.zeros(t.shape, dtype=torch.float32, device=device)
        return LayerGradBufs(z(w.W1), z(w.W2), z(w.b1), z(w.b2), z(w.ln_gamma), z(w.ln_beta),
                             z(w.rab_pos), z(w.rab_time))

    def c(self) -> Grads:
        return Grads(ptr(self.dW1), ptr(self.db1), ptr(self.dW2), ptr(self.db2), ptr(self.dgamma),
                     ptr(self.dbeta), ptr(self.drab_pos), ptr(self.drab_time))


# ----------------------------------------------------------------------------
# Sizes
# ----------------------------------------------------------------------------

def workspace_size(cfg: Config, B: int, T: int):
    ws, sv = c_size_t(0), c_size_t(0)
    _check(lib().hstu_workspace_size(ctypes.byref(cfg), B, T, ctypes.byref(ws), ctypes.byref(sv)),
           "hstu_workspace_size")
    return ws.value, sv.value


def attention_workspace_size(cfg: Config, B: int, T: int) -> int:
    return int(lib().hstu_attention_workspace_size(ctypes.byref(cfg), B, T))


def saved_layout(cfg: Config, T: int):
    off = (c_size_t * (SAVED_COUNT + 1))()
    _check(lib().hstu_saved_layout(ctypes.byref(cfg), T, off), "hstu_saved_layout")
    return list(off)


def saved_views(cfg: Config, saved: torch.Tensor, T: int):
    """Typed views of one layer's saved block: pre, g, o, z, mean, rstd."""
    off = saved_layout(cfg, T)
    d = cfg.d_model
    dt = torch_dtype(cfg.dtype)
    es = 2 if cfg.dtype == HSTU_BF16 else 4

    def view(i, n, dtype, shape):
        nbytes = n * (4 if dtype == torch.float32 else es)
        return saved[off[i]:off[i] + nbytes].view(dtype).view(*shape)
    out = {"pre": view(SAVED_PRE, T * 4 * d, dt, (T, 4 * d)),
            "g": view(SAVED_G, T * 4 * d, dt, (T, 4 * d)),
            "o": view(SAVED_O, T * d, torch.float32, (T, d)),
            "z": view(SAVED_Z, T * d, dt, (T, d)),
            "mean": view(SAVED_MEAN, T, torch.float32, (T,)),
            "rstd": view(SAVED_RSTD, T, torch.float32, (T,))}
    if cfg.io_dtype != cfg.dtype:
        out["xlow"] = view(SAVED_XLOW, T * d, dt, (T, d))
    return out


def _empty(shape, dtype, device, stream):
    """A buffer that kernels on this stream write (None: the current one): from the stream's own
    pool, whose memory nothing that is still queued on another stream uses."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _like(t, stream):
    """A contiguous buffer of t's shape and type for kernels on this stream."""
    return _empty(t.shape, t.dtype, t.device, stream)


def workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """Scratch of one call, at least nbytes: a new buffer each time, on the stream that the call's
    kernels run on, so that no two calls, streams or captured graphs share one."""
    return _empty((max(nbytes, 256),), torch.uint8, device, stream)


# ----------------------------------------------------------------------------
# Step-level calls
# ----------------------------------------------------------------------------

def proj_in_fwd(cfg, w: LayerWeights, x, pre_out, g_out, stream=None):
    _check(lib().hstu_proj_in_fwd(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(x), x.shape[0],
                                  ptr(pre_out), ptr(g_out), stream_ptr(stream)), "hstu_proj_in_fwd")


def attention_fwd(cfg, rab_pos, rab_time, g, offsets, timestamps, num_targets, o_out, stream=None,
                  ws_bytes=None):
    """ws_bytes: workspace bytes passed to the call (default: the full
    hstu_attention_workspace_size)."""
    B, T = offsets.numel() - 1, g.shape[0]
    n = lib().hstu_attention_workspace_size(ctypes.byref(cfg), B, T)
    ws = workspace(n, g.device, stream)
    nb = ws.numel() if ws_bytes is None else min(int(ws_bytes), ws.numel())
    _check(lib().hstu_attention_fwd(ctypes.byref(cfg), ptr(rab_pos), ptr(rab_time), ptr(g),
                                    ptr(offsets), B, T, ptr(timestamps), ptr(num_targets),
                                    ptr(o_out), ptr(ws), nb, stream_ptr(stream)),
           "hstu_attention_fwd")


def softmax_attention_fwd(cfg, rab_pos, rab_time, g, offsets, timestamps, num_targets, o_out,
                          stream=None):
    """The softmax comparison attention (same score and mask, softmax weights)."""
    B, T = offsets.numel() - 1, g.shape[0]
    n = lib().hstu_attention_workspace_size(ctypes.byref(cfg), B, T)
    ws = workspace(n, g.device, stream)
    _check(lib().hstu_softmax_attention_fwd(ctypes.byref(cfg), ptr(rab_pos), ptr(rab_time), ptr(g),
                                            ptr(offsets), B, T, ptr(timestamps), ptr(num_targets),
                                            ptr(o_out), ptr(ws), ws.numel(), stream_ptr(stream)),
           "hstu_softmax_attention_fwd")


def attention_fwd_noalloc(cfg, rab_pos, rab_time, g, offsets, timestamps, num_targets, o_out,
                          stream=None):
    """hstu_attention_fwd without a workspace (static device scratch)."""
    B, T = offsets.numel() - 1, g.shape[0]
    _check(lib().hstu_attention_fwd_noalloc(ctypes.byref(cfg), ptr(rab_pos), ptr(rab_time), ptr(g),
                                            ptr(offsets), B, T, ptr(timestamps), ptr(num_targets),
                                            ptr(o_out), stream_ptr(stream)),
           "hstu_attention_fwd_noalloc")


def attention_fwd_cached(cfg, rab_pos, rab_time, cand_g, cand_offsets, cand_ts, hist_kv,
                         hist_offsets, hist_ts, o_out, stream=None):
    B, Tc, Th = cand_offsets.numel() - 1, cand_g.shape[0], hist_kv.shape[0]
    n = lib().hstu_attention_workspace_size(ctypes.byref(cfg), B, Tc)
    ws = workspace(n, cand_g.device, stream)
    _check(lib().hstu_attention_fwd_cached(ctypes.byref(cfg), ptr(rab_pos), ptr(rab_time),
                                           ptr(cand_g), ptr(cand_offsets), B, Tc, ptr(cand_ts),
                                           ptr(hist_kv), ptr(hist_offsets), Th, ptr(hist_ts),
                                           ptr(o_out), ptr(ws), ws.numel(), stream_ptr(stream)),
           "hstu_attention_fwd_cached")


def ln_gate_fwd(cfg, gamma, beta, o, g, z_out, mean_out=None, rstd_out=None, stream=None):
    _check(lib().hstu_ln_gate_fwd(ctypes.byref(cfg), ptr(gamma), ptr(beta), ptr(o), ptr(g),
                                  o.shape[0], ptr(z_out), ptr(mean_out), ptr(rstd_out),
                                  stream_ptr(stream)), "hstu_ln_gate_fwd")


def proj_out_fwd(cfg, W2, b2, z, x, y_out, stream=None):
    _check(lib().hstu_proj_out_fwd(ctypes.byref(cfg), ptr(W2), ptr(b2), ptr(z), ptr(x), z.shape[0],
                                   ptr(y_out), stream_ptr(stream)), "hstu_proj_out_fwd")


def proj_out_bwd(cfg, W2, z, dy, dz_out, dW2=None, db2=None, stream=None):
    _check(lib().hstu_proj_out_bwd(ctypes.byref(cfg), ptr(W2), ptr(z), ptr(dy), dy.shape[0],
                                   ptr(dz_out), ptr(dW2), ptr(db2), stream_ptr(stream)),
           "hstu_proj_out_bwd")


def ln_gate_bwd(cfg, gamma, beta, dz, o, g, pre, mean, rstd, do_out, dpre, dgamma=None,
                dbeta=None, stream=None):
    _check(lib().hstu_ln_gate_bwd(ctypes.byref(cfg), ptr(gamma), ptr(beta), ptr(dz), ptr(o), ptr(g),
                                  ptr(pre), ptr(mean), ptr(rstd), dz.shape[0], ptr(do_out),
                                  ptr(dpre), ptr(dgamma), ptr(dbeta), stream_ptr(stream)),
           "hstu_ln_gate_bwd")


def attention_bwd(cfg, rab_pos, rab_time, g, pre, dout, offsets, timestamps, num_targets, dpre,
                  drab_pos=None, drab_time=None, stream=None):
    B, T = offsets.numel() - 1, g.shape[0]
    n = lib().hstu_attention_bwd_workspace_size(ctypes.byref(cfg), B, T)
    ws = workspace(n, g.device, stream)
    _check(lib().hstu_attention_bwd(ctypes.byref(cfg), ptr(rab_pos), ptr(rab_time), ptr(g), ptr(pre),
                                    ptr(dout), ptr(offsets), B, T, ptr(timestamps),
                                    ptr(num_targets), ptr(dpre), ptr(drab_pos), ptr(drab_time),
                                    ptr(ws), ws.numel(), stream_ptr(stream)), "hstu_attention_bwd")


def proj_in_bwd(cfg, W1, x, dpre, dy_resid, dx_out, dW1=None, db1=None, stream=None):
    _check(lib().hstu_proj_in_bwd(ctypes.byref(cfg), ptr(W1), ptr(x), ptr(dpre), ptr(dy_resid),
                                  dpre.shape[0], ptr(dx_out), ptr(dW1), ptr(db1),
                                  stream_ptr(stream)), "hstu_proj_in_bwd")


def validate_inputs(offsets, timestamps, num_targets, max_seq_len, stream=None) -> int:
    """Runs the device validator and returns its flag word (synchronises)."""
    B = offsets.numel() - 1
    T = timestamps.numel()
    with torch.cuda.stream(stream):            # the flags are cleared and read on the validator's stream
        flags = torch.zeros(1, dtype=torch.int32, device=offsets.device)
        _check(lib().hstu_validate_inputs(ptr(offsets), B, T, ptr(timestamps), ptr(num_targets),
                                          max_seq_len, ptr(flags), stream_ptr(stream)),
               "hstu_validate_inputs")
        return int(flags.item())


# ----------------------------------------------------------------------------
# Stochastic Length sampler
# ----------------------------------------------------------------------------

def sl_subsequence_length(max_len: int, alpha: float) -> int:
    """L = floor(N^(alpha/2)), computed by the library on the host."""
    v = int(lib().hstu_sl_subsequence_length(int(max_len), float(alpha)))
    if v < 0:
        raise HSTUError(1, "hstu_sl_subsequence_length")
    return v


def stochastic_length(offsets, num_targets, sub_len, keep_draw, keys, new_offsets=None,
                      gather_index=None, stream=None):
    """Samples the jagged batch; returns (new_offsets [B+1], gather_index [T])
    on the device.  new_offsets[B] is the sampled row count; entries of
    gather_index past it are not written."""
    B, T = offsets.numel() - 1, keys.numel()
    for name, t, sizes in (("offsets", offsets, (8,)), ("keep_draw", keep_draw, (4,)),
                           ("keys", keys, (4,)), ("num_targets", num_targets, (4,))):
        if t is not None and (t.element_size() not in sizes or not t.is_contiguous()):
            raise ValueError(f"stochastic_length: {name} must be contiguous with "
                             f"{sizes[0]}-byte elements")
    if keep_draw.numel() != B:
        raise ValueError("stochastic_length: keep_draw needs one entry per sequence")
    if new_offsets is None:
        new_offsets = _empty((B + 1,), torch.int64, offsets.device, stream)
    if gather_index is None:
        gather_index = _empty((max(T, 1),), torch.int64, offsets.device, stream)
    _check(lib().hstu_stochastic_length(ptr(offsets), ptr(num_targets), B, T, int(sub_len),
                                        ptr(keep_draw), ptr(keys), ptr(new_offsets),
                                        ptr(gather_index), stream_ptr(stream)),
           "hstu_stochastic_length")
    return new_offsets, gather_index


def gather_rows(src, gather_index, d_num_rows, out, stream=None):
    """out[r] = src[gather_index[r]] for r < d_num_rows (a device int64
    scalar view) and r < out.shape[0]; src and out are 1-D or 2-D tensors with
    contiguous rows of the same width and dtype."""
    src2 = src.reshape(src.shape[0], -1)
    out2 = out.reshape(out.shape[0], -1)
    if src2.dtype != out2.dtype or src2.shape[1] != out2.shape[1] or \
            src2.stride(1) != 1 or out2.stride(1) != 1:
        raise ValueError("gather_rows: src and out need the same dtype, width and unit inner stride")
    es = src2.element_size()
    _check(lib().hstu_gather_rows(ptr(src2), src2.stride(0) * es, src2.shape[0],
                                  ptr(gather_index), ptr(d_num_rows), out2.shape[0],
                                  src2.shape[1] * es, ptr(out2), out2.stride(0) * es,
                                  stream_ptr(stream)),
           "hstu_gather_rows")
    return out


# ----------------------------------------------------------------------------
# Shared by the calls below: checks of their tensors, the device they run on
# ----------------------------------------------------------------------------

_DTYPE_IDS = {torch.float32: HSTU_F32, torch.bfloat16: HSTU_BF16}


def _rows(where, name, t, rows, width, dtype, device):
    """Checks a [rows][width] tensor with unit inner stride; returns its row stride."""
    if t.dtype is dtype and t.shape == (rows, width) and t.device == device:
        st = t.stride()
        if st[1] == 1 or width == 1:
            return st[0] if rows > 1 or st[0] > width else width
    raise ValueError(f"{where}: {name} must be [{rows}][{width}] {dtype} on {device} with unit inner "
                     f"stride, got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")


def _flat(where, name, t, shape, dtype, device):
    """Checks a contiguous tensor of this shape; returns its address (None for a None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{where}: {name} must be contiguous {tuple(shape)} {dtype} on {device}, got "
                     f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")


def _launch(where, device, stream, f, *args, ws_bytes=None):
    """Calls the entry point f(*args[, workspace, bytes], stream) on the tensors' device, with
    a workspace of this call alone."""
    if device.type != "cuda":
        raise ValueError(f"{where}: needs CUDA tensors, got {device}")
    index = device.index
    if index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch(where, device, stream, f, *args, ws_bytes=ws_bytes)
    if stream is None:
        s = _raw_stream(index)
    else:
        if stream.device_index != index:
            raise ValueError(f"{where}: the stream belongs to cuda:{stream.device_index}, the tensors "
                             f"to {device}")
        s = stream.cuda_stream
    ws = _empty(ws_bytes, torch.uint8, device, stream) if ws_bytes else None
    if ws_bytes is None:
        status = f(*args, s)
    else:
        status = f(*args, None if ws is None else ws.data_ptr(), ws_bytes, s)
    if status:
        raise HSTUError(status, where)


# ----------------------------------------------------------------------------
# Embedding lookup and its gradient
# ----------------------------------------------------------------------------

def _ids(where, ids, device):
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 1 or ids.device != device or \
            not ids.is_contiguous():
        raise ValueError(f"{where}: ids must be contiguous [T] int32 or int64 on {device}, got "
                         f"{tuple(ids.shape)} {ids.dtype} on {ids.device}")
    return ids.shape[0], ids.element_size()


def embedding_fwd(table, ids, scale: float = 1.0, out=None, low=None, out_dtype=torch.float32,
                  stream=None):
    """out[t] = scale * table[ids[t]] (zero where the id is outside the table); returns out.  out
    [T][width] with width >= the table's (further columns are zeroed), fp32 or bf16; low: an
    optional bf16 copy of an fp32 out, as fwd's x_low takes it."""
    where = "embedding_fwd"
    dev = table.device
    T, ib = _ids(where, ids, dev)
    if table.dim() != 2 or table.dtype not in _DTYPE_IDS:
        raise ValueError(f"{where}: table must be [V][dim] fp32 or bf16")
    V, dim = table.shape
    ts = _rows(where, "table", table, V, dim, table.dtype, dev)
    if out is None:
        out = _empty((T, dim), out_dtype, dev, stream)
    if out.dtype not in _DTYPE_IDS or out.dim() != 2:
        raise ValueError(f"{where}: out must be [T][width] fp32 or bf16")
    width = out.shape[1]
    os_ = _rows(where, "out", out, T, width, out.dtype, dev)
    ls = 0 if low is None else _rows(where, "low", low, T, width, torch.bfloat16, dev)
    _launch(where, dev, stream, lib().hstu_embedding_fwd, table.data_ptr(), _DTYPE_IDS[table.dtype], V,
            dim, ts, ids.data_ptr(), ib, T, scale, out.data_ptr(), _DTYPE_IDS[out.dtype], width, os_,
            ptr(low), ls)
    return out


def _embedding_upstream(where, dout, ids, dim):
    dev = dout.device
    T, ib = _ids(where, ids, dev)
    if dout.dtype not in _DTYPE_IDS or dout.dim() != 2 or dout.shape[1] < dim:
        raise ValueError(f"{where}: dout must be [T][width] fp32 or bf16 with width >= {dim}")
    return T, ib, _rows(where, "dout", dout, T, dout.shape[1], dout.dtype, dev)


def embedding_bwd(dout, ids, dtable, scale: float = 1.0, stream=None):
    """dtable[v] += scale * the sum of dout's rows whose id is v (fp32 [V][dim]; dout may be
    wider, its further columns are not read); returns dtable."""
    where = "embedding_bwd"
    V, dim = dtable.shape
    T, ib, ds = _embedding_upstream(where, dout, ids, dim)
    gs = _rows(where, "dtable", dtable, V, dim, torch.float32, dout.device)
    L = lib()
    _launch(where, dout.device, stream, L.hstu_embedding_bwd, dout.data_ptr(), _DTYPE_IDS[dout.dtype],
            ds, ids.data_ptr(), ib, T, V, dim, scale, dtable.data_ptr(), gs,
            ws_bytes=L.hstu_embedding_bwd_workspace_size(T, V, dim))
    return dtable


def embedding_bwd_rows(dout, ids, num_items: int, row_ids, rows, count, scale: float = 1.0, stream=None):
    """The gradient of a table of num_items rows as its non-zero rows: row_ids [min(T, num_items)]
    int64 (ascending), rows [min(T, num_items)][dim] fp32 (written), count [1] int64, on the device.
    Entries past count are left as they were."""
    where = "embedding_bwd_rows"
    if rows.dim() != 2:
        raise ValueError(f"{where}: rows must be [min(T, num_items)][dim]")
    cap, dim = rows.shape
    T, ib, ds = _embedding_upstream(where, dout, ids, dim)
    dev = dout.device
    rs = _rows(where, "rows", rows, min(T, num_items), dim, torch.float32, dev)
    _flat(where, "row_ids", row_ids, (cap,), torch.int64, dev)
    _flat(where, "count", count, (1,), torch.int64, dev)
    L = lib()
    _launch(where, dev, stream, L.hstu_embedding_bwd_rows, dout.data_ptr(), _DTYPE_IDS[dout.dtype], ds,
            ids.data_ptr(), ib, T, num_items, dim, scale, row_ids.data_ptr(), rows.data_ptr(), rs,
            count.data_ptr(), ws_bytes=L.hstu_embedding_bwd_workspace_size(T, num_items, dim))
    return row_ids, rows, count


# ----------------------------------------------------------------------------
# Norms before and after a block
# ----------------------------------------------------------------------------

_NORMS = {None: NORM_NONE, "none": NORM_NONE, "layer": NORM_LAYER, "rms": NORM_RMS}
_GATES = {None: GATE_NONE, "none": GATE_NONE, "sigmoid": GATE_SIGMOID, "silu": GATE_SILU}
_PARAMS = ("post_gamma", "post_beta", "res_scale", "pre_gamma", "pre_beta")


@dataclass
class BlockNorm:
    """The joint of two blocks: kinds "layer", "rms" or None, the gate's activation "silu",
    "sigmoid" or None (the gate as it is), and [d] parameters in the config's dtype."""
    post: Optional[str] = "layer"
    pre: Optional[str] = "layer"
    gate_act: Optional[str] = None
    post_gamma: Optional[torch.Tensor] = None
    post_beta: Optional[torch.Tensor] = None
    res_scale: Optional[torch.Tensor] = None
    pre_gamma: Optional[torch.Tensor] = None
    pre_beta: Optional[torch.Tensor] = None

    def c(self, cfg, where, device) -> CBlockNorm:
        if self.post not in _NORMS or self.pre not in _NORMS or self.gate_act not in _GATES:
            raise ValueError(f"{where}: unknown norm or gate activation: {self.post}, {self.pre}, "
                             f"{self.gate_act}")
        shape, dt = (cfg.d_model,), torch_dtype(cfg.dtype)
        return CBlockNorm(_NORMS[self.post], _NORMS[self.pre], _GATES[self.gate_act], 0,
                          _flat(where, "post_gamma", self.post_gamma, shape, dt, device),
                          _flat(where, "post_beta", self.post_beta, shape, dt, device),
                          _flat(where, "res_scale", self.res_scale, shape, dt, device),
                          _flat(where, "pre_gamma", self.pre_gamma, shape, dt, device),
                          _flat(where, "pre_beta", self.pre_beta, shape, dt, device))


@dataclass
class BlockNormGrads:
    """fp32 [d] gradients of a BlockNorm's parameters, accumulated; None: not wanted.  Parameters that
    are one tensor may have one gradient, which takes the sum."""
    post_gamma: Optional[torch.Tensor] = None
    post_beta: Optional[torch.Tensor] = None
    res_scale: Optional[torch.Tensor] = None
    pre_gamma: Optional[torch.Tensor] = None
    pre_beta: Optional[torch.Tensor] = None

    @staticmethod
    def zeros_like(bn: BlockNorm) -> "BlockNormGrads":
        z = lambda t: None if t is None else torch.zeros(t.shape, dtype=torch.float32, device=t.device)
        return BlockNormGrads(*(z(getattr(bn, n)) for n in _PARAMS))

    def c(self, cfg, where, device) -> CBlockNormGrads:
        shape = (cfg.d_model,)
        return CBlockNormGrads(*[_flat(where, n, getattr(self, n), shape, torch.float32, device)
                                 for n in _PARAMS])


def block_norm_fwd(cfg, bn: BlockNorm, x, b=None, gate=None, y=None, h=None, stats=None, want_h=True,
                   stream=None):
    """y = x + res_scale * (Norm_post(b) * act(gate)), h = Norm_pre(y); returns (y, h).  Without b
    (the start of a stack) y is x; with want_h False (its end) h is None, and the backward has no dh.
    stats: fp32 [T][4], kept for block_norm_bwd."""
    where = "block_norm_fwd"
    dev, d, T = x.device, cfg.d_model, x.shape[0]
    io, dt = torch_dtype(cfg.io_dtype), torch_dtype(cfg.dtype)
    if b is None and (gate is not None or (y is not None and y is not x)):
        raise ValueError(f"{where}: gate and y need b (without it y is x)")
    if h is None and want_h:
        h = _empty((T, d), dt, dev, stream)
    if b is None:
        y = x
    elif y is None:
        y = _empty((T, d), io, dev, stream)
    shape = (T, d)
    gs = 0 if gate is None else _rows(where, "gate", gate, T, d, dt, dev)
    _launch(where, dev, stream, lib().hstu_block_norm_fwd, ctypes.byref(cfg),
            ctypes.byref(bn.c(cfg, where, dev)), _flat(where, "x", x, shape, io, dev),
            _flat(where, "b", b, shape, io, dev), ptr(gate), gs, T, _flat(where, "y", y, shape, io, dev),
            _flat(where, "h", h, shape, dt, dev), _flat(where, "stats", stats, (T, 4), torch.float32, dev))
    return y, h


def block_norm_bwd(cfg, bn: BlockNorm, y, b, gate, stats, dy=None, dh=None, dx=None, db=None, dgate=None,
                   grads: Optional[BlockNormGrads] = None, stream=None):
    """Backward of block_norm_fwd from dy (upstream of y along the residual stream; None: none) and
    dh (upstream of h; None: none).  Writes dx (may be dy), db and dgate where given, accumulates
    grads; returns dx."""
    where = "block_norm_bwd"
    dev, d, T = stats.device, cfg.d_model, stats.shape[0]
    io, dt = torch_dtype(cfg.io_dtype), torch_dtype(cfg.dtype)
    if dh is not None and y is None:
        raise ValueError(f"{where}: dh needs y")
    if b is None and (gate is not None or db is not None or dgate is not None):
        raise ValueError(f"{where}: gate, db and dgate need b")
    if dgate is not None and gate is None:
        raise ValueError(f"{where}: dgate needs gate")
    if dx is None:
        dx = _empty((T, d), io, dev, stream)
    shape = (T, d)
    gs = 0 if gate is None else _rows(where, "gate", gate, T, d, dt, dev)
    dgs = 0 if dgate is None else _rows(where, "dgate", dgate, T, d, dt, dev)
    L = lib()
    g = None if grads is None else ctypes.byref(grads.c(cfg, where, dev))
    _launch(where, dev, stream, L.hstu_block_norm_bwd, ctypes.byref(cfg),
            ctypes.byref(bn.c(cfg, where, dev)), _flat(where, "y", y, shape, io, dev),
            _flat(where, "b", b, shape, io, dev), ptr(gate), gs,
            _flat(where, "stats", stats, (T, 4), torch.float32, dev), _flat(where, "dy", dy, shape, io, dev),
            _flat(where, "dh", dh, shape, io, dev), T, _flat(where, "dx", dx, shape, io, dev),
            _flat(where, "db", db, shape, dt, dev), ptr(dgate), dgs, g,
            ws_bytes=0 if g is None else L.hstu_block_norm_bwd_workspace_size(ctypes.byref(cfg), T))
    return dx


# ----------------------------------------------------------------------------
# Activation checkpoints in 8 bits
# ----------------------------------------------------------------------------

def checkpoint_layout(cfg: Config, T: int):
    """Byte offsets of a checkpoint's parts and, last, its size."""
    off = (c_size_t * (CKPT_COUNT + 1))()
    _check(lib().hstu_checkpoint_layout(ctypes.byref(cfg), T, off), "hstu_checkpoint_layout")
    return list(off)


def checkpoint_bytes(cfg: Config, fmt: int, T: int) -> int:
    """Size of the checkpoint of one layer's saved block (the same for both formats)."""
    return checkpoint_layout(cfg, T)[CKPT_COUNT]


@functools.lru_cache(maxsize=256)
def _checkpoint_sizes(fields, T: int):
    """Bytes of a saved block and of its checkpoint for a config of these fields."""
    cfg = Config(*fields)
    return saved_layout(cfg, T)[SAVED_COUNT], checkpoint_layout(cfg, T)[CKPT_COUNT]


def _checkpoint_blocks(where, cfg, saved, ckpt, T):
    dev = saved.device
    # the sizes depend on these fields; the others are only checked to be valid
    sizes = _checkpoint_sizes((cfg.d_model, cfg.num_heads, cfg.head_dim, 1, 1, 1, 1.0, 0.0, cfg.dtype,
                               cfg.io_dtype), T)
    for n, t, need in (("saved", saved, sizes[0]), ("ckpt", ckpt, sizes[1])):
        if t.dtype is not torch.uint8 or t.device != dev or not t.is_contiguous() or t.numel() < need:
            raise ValueError(f"{where}: {n} must be at least {need} contiguous bytes on {dev}")
    return dev


def checkpoint_save(cfg: Config, fmt: int, saved, T: int, ckpt, stream=None):
    """Holds a layer's saved block (filled by fwd) in 8 bits (CKPT_INT8 or CKPT_E4M3); returns ckpt."""
    dev = _checkpoint_blocks("checkpoint_save", cfg, saved, ckpt, T)
    _launch("checkpoint_save", dev, stream, lib().hstu_checkpoint_save, ctypes.byref(cfg), fmt,
            saved.data_ptr(), T, ckpt.data_ptr())
    return ckpt


def checkpoint_restore(cfg: Config, fmt: int, ckpt, T: int, ln_gamma, ln_beta, saved, stream=None):
    """A saved block for bwd from a checkpoint and the layer's ln_gamma, ln_beta; returns saved."""
    where = "checkpoint_restore"
    dev = _checkpoint_blocks(where, cfg, saved, ckpt, T)
    shape, dt = (cfg.d_model,), torch_dtype(cfg.dtype)
    _launch(where, dev, stream, lib().hstu_checkpoint_restore, ctypes.byref(cfg), fmt, ckpt.data_ptr(),
            _flat(where, "ln_gamma", ln_gamma, shape, dt, dev),
            _flat(where, "ln_beta", ln_beta, shape, dt, dev), T, saved.data_ptr())
    return saved


# ----------------------------------------------------------------------------
# Layer-level calls
# ----------------------------------------------------------------------------

def fwd(cfg, w: LayerWeights, x, offsets, timestamps, num_targets=None, y=None, saved=None,
        kv_out=None, stream=None, x_low=None, y_low=None):
    """One layer forward; returns y.  `saved` (uint8, saved_bytes) is filled
    for a later bwd() when given.  x_low / y_low (bf16 [T][d] buffers, fp32
    io only): the bf16 copy of x from the previous layer, and where to write
    the bf16 copy of y for the next one (hstu_fwd_chain)."""
    B, T = offsets.numel() - 1, x.shape[0]
    ws_n, _ = workspace_size(cfg, B, T)
    ws = workspace(ws_n, x.device, stream)
    if y is None:
        y = _like(x, stream)
    if x_low is None and y_low is None:
        _check(lib().hstu_fwd(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(x), ptr(offsets), B, T,
                              ptr(timestamps), ptr(num_targets), ptr(y), ptr(saved), ptr(kv_out),
                              ptr(ws), ws.numel(), stream_ptr(stream)), "hstu_fwd")
    else:
        _check(lib().hstu_fwd_chain(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(x), ptr(x_low),
                                    ptr(offsets), B, T, ptr(timestamps), ptr(num_targets), ptr(y),
                                    ptr(y_low), ptr(saved), ptr(kv_out), ptr(ws), ws.numel(),
                                    stream_ptr(stream)), "hstu_fwd_chain")
    return y


def fwd_cached(cfg, w: LayerWeights, cand_x, cand_offsets, cand_ts, hist_kv, hist_offsets, hist_ts,
               y=None, stream=None):
    B, Tc = cand_offsets.numel() - 1, cand_x.shape[0]
    ws_n, _ = workspace_size(cfg, B, Tc)
    ws = workspace(ws_n, cand_x.device, stream)
    if y is None:
        y = _like(cand_x, stream)
    _check(lib().hstu_fwd_cached(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(cand_x),
                                 ptr(cand_offsets), B, Tc, ptr(cand_ts), ptr(hist_kv),
                                 ptr(hist_offsets), hist_kv.shape[0], ptr(hist_ts), ptr(y), ptr(ws),
                                 ws.numel(), stream_ptr(stream)), "hstu_fwd_cached")
    return y


def bwd(cfg, w: LayerWeights, x, dy, saved, offsets, timestamps, num_targets=None, dx=None,
        grads: Optional[LayerGradBufs] = None, stream=None, dy_low=None, dx_low=None):
    """One layer backward; returns dx.  dy_low / dx_low (bf16 [T][d], fp32 io
    only): the bf16 copy of dy from the layer above, and where to write the
    bf16 copy of dx for the layer below (hstu_bwd_chain)."""
    B, T = offsets.numel() - 1, x.shape[0]
    ws_n, _ = workspace_size(cfg, B, T)
    ws = workspace(ws_n, x.device, stream)
    if dx is None:
        dx = _like(x, stream)
    g = grads.c() if grads is not None else Grads()
    if dy_low is None and dx_low is None:
        _check(lib().hstu_bwd(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(x), ptr(dy), ptr(saved),
                              ptr(offsets), B, T, ptr(timestamps), ptr(num_targets), ptr(dx),
                              ctypes.byref(g), ptr(ws), ws.numel(), stream_ptr(stream)), "hstu_bwd")
    else:
        _check(lib().hstu_bwd_chain(ctypes.byref(cfg), ctypes.byref(w.c()), ptr(x), ptr(dy),
                                    ptr(dy_low), ptr(saved), ptr(offsets), B, T, ptr(timestamps),
                                    ptr(num_targets), ptr(dx), ptr(dx_low), ctypes.byref(g),
                                    ptr(ws), ws.numel(), stream_ptr(stream)), "hstu_bwd_chain")
    return dx


# ----------------------------------------------------------------------------
# Profiler
# ----------------------------------------------------------------------------

def profiler_enable(on: bool = True):
    lib().hstu_profiler_enable(1 if on else 0)


def nvtx_enable(on: bool = True):
    """NVTX ranges named after the kernel classes around the library's steps."""
    lib().hstu_nvtx_enable(1 if on else 0)


def profiler_reset():
    lib().hstu_profiler_reset()


def profiler_collect(kernel_id: int):
    n, ms = c_int64(0), c_double(0.0)
    _check(lib().hstu_profiler_collect(kernel_id, ctypes.byref(n), ctypes.byref(ms)),
           "hstu_profiler_collect")
    return n.value, ms.value


def launch_count() -> int:
    return int(lib().hstu_launch_count())


def device_status(clear: bool = True, stream=None) -> int:
    """The library's device status word (synchronises the stream)."""
    v = c_uint32(0)
    _check(lib().hstu_device_status(ctypes.byref(v), 1 if clear else 0, stream_ptr(stream)),
           "hstu_device_status")
    return v.value


def selftest_wait_timeout(limit_ns: int, result=None, stream=None):
    """Launches the library's bounded-wait diagnostic (a wait nothing ends
    but its limit); the device status word then carries HSTU_DEVICE_TIMEOUT."""
    _check(lib().hstu_selftest_wait_timeout(int(limit_ns), ptr(result), stream_ptr(stream)),
           "hstu_selftest_wait_timeout")


DEVICE_TIMEOUT, DEVICE_SMEM_ALIGN, DEVICE_BOUNDS = 0x100, 0x200, 0x400


def version() -> str:
    return lib().hstu_version().decode()
