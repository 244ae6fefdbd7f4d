"""Python binding of libdgsamp: argument marshalling only.

Every function here has the name of the C entry point it calls (include/dgsamp.h)
and does nothing but turn torch CUDA tensors into pointers, sizes and the current
stream, allocate outputs with torch when the caller gives none, and raise on a
non-zero status.  All arithmetic runs in the library's CUDA kernels; there is no
other path.  Importing this module fails if the library is missing.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdgsamp.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m denoising_sampler_step_gb300.build` "
        "(or __graft_entry__.build()); there is no fallback path")

lib = ctypes.CDLL(LIB_PATH)

_i64, _i32, _f32, _p, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_u32 = ctypes.c_uint32

# flags of the sampler-step calls (dg_step_flags)
DG_STEP_TWO_PASS = 1

lib.dg_version.restype = ctypes.c_int
lib.dg_last_error.restype = ctypes.c_char_p
lib.dg_row_stats.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p]
lib.dg_row_stats.restype = ctypes.c_int
lib.dg_soft_embed_workspace_size.argtypes = [_i64, _i64, _i64]
lib.dg_soft_embed_workspace_size.restype = _sz
lib.dg_soft_embed.argtypes = [_p, _i64, _p, _i64, _i64, _i64, _p, _i64, _i64, _i64, _f32, _p, _i64, _p, _sz, _p]
lib.dg_soft_embed.restype = ctypes.c_int
lib.dg_soft_embed_no_alloc.argtypes = [_p, _i64, _p, _i64, _i64, _i64, _p, _i64, _i64, _i64, _f32, _p, _i64, _p]
lib.dg_soft_embed_no_alloc.restype = ctypes.c_int
lib.dg_entropy_accept.argtypes = [_p, _p, _i32, _i32, _p, _i32, _p, _p, _p, _p]
lib.dg_entropy_accept.restype = ctypes.c_int
lib.dg_sum_partials.argtypes = [ctypes.POINTER(_p), _i32, _i64, _i64, _i64, _f32, _p, _i64, _p]
lib.dg_sum_partials.restype = ctypes.c_int
lib.dg_sampler_step.argtypes = [_p, _i32, _i32, _i64, _i64, _p, _i64, _i64, _i64, _i64, _i64, _f32, _p, _i32,
                                _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _u32, _p, _sz, _p]
lib.dg_sampler_step.restype = ctypes.c_int
lib.dg_get_device_status.argtypes = [_p]
lib.dg_get_device_status.restype = ctypes.c_int
lib.dg_row_sample.argtypes = [_p, _i64, _i64, _i64, _f32, ctypes.c_uint64, ctypes.c_uint64, _p, _p, _p]
lib.dg_row_sample.restype = ctypes.c_int
lib.dg_check_wait_timeout.argtypes = [ctypes.c_uint32, _p]
lib.dg_check_wait_timeout.restype = ctypes.c_int
lib.dg_entropy_accept_eligible.argtypes = [_p, _p, _p, _i32, _i32, _p, _i32, _p, _p, _p, _p]
lib.dg_entropy_accept_eligible.restype = ctypes.c_int
lib.dg_loop_update.argtypes = [_p, _p, _p, _p, _i32, _i32, _i32, _f32, _i32, _p, _p, _p, _p, _p, _p, _p]
lib.dg_loop_update.restype = ctypes.c_int
lib.dg_sampler_loop_step.argtypes = [_p, _i32, _i32, _i64, _i64, _p, _i64, _i64, _i64, _i64, _i64, _f32, _p, _i32,
                                     _i32, _f32, _i32, _f32, ctypes.c_uint64, ctypes.c_uint64,
                                     _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64,
                                     _p, _p, _p, _p, _p, _p, _u32, _p, _sz, _p]
lib.dg_row_stats_sample.argtypes = [_p, _i64, _i64, _i64, _f32, ctypes.c_uint64, ctypes.c_uint64,
                                    _p, _p, _p, _p, _p, _p, _p, _p]
lib.dg_row_stats_sample.restype = ctypes.c_int
lib.dg_row_stats_partial.argtypes = [_p, _i64, _i64, _i64, _i64, _p, _p]
lib.dg_row_stats_partial.restype = ctypes.c_int
lib.dg_row_stats_combine.argtypes = [_p, _i32, _i64, _p, _p, _p, _p, _p, _p]
lib.dg_row_stats_combine.restype = ctypes.c_int
lib.dg_sampler_loop_step.restype = ctypes.c_int
lib.dg_quantize_e4m3.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _p]
lib.dg_quantize_e4m3.restype = ctypes.c_int
lib.dg_soft_embed_workspace_size_e4m3.argtypes = [_i64, _i64, _i64]
lib.dg_soft_embed_workspace_size_e4m3.restype = _sz
lib.dg_soft_embed_e4m3.argtypes = [_p, _i64, _p, _i64, _i64, _i64, _p, _p, _i64, _i64, _i64, _f32, _p, _i64, _p,
                                   _sz, _p]
lib.dg_soft_embed_e4m3.restype = ctypes.c_int
lib.dg_sampler_step_e4m3.argtypes = [_p, _i32, _i32, _i64, _i64, _p, _p, _i64, _i64, _i64, _i64, _i64, _f32, _p,
                                     _i32, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, _u32, _p, _sz, _p]
lib.dg_sampler_step_e4m3.restype = ctypes.c_int
lib.dg_sampler_loop_step_e4m3.argtypes = [_p, _i32, _i32, _i64, _i64, _p, _p, _i64, _i64, _i64, _i64, _i64, _f32, _p,
                                          _i32, _i32, _f32, _i32, _f32, ctypes.c_uint64, ctypes.c_uint64,
                                          _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64,
                                          _p, _p, _p, _p, _p, _p, _u32, _p, _sz, _p]
lib.dg_sampler_loop_step_e4m3.restype = ctypes.c_int
lib.dg_soft_embed_shard_begin.argtypes = [_p, _i64, _i64, _i64, _i64, _p, _i64, _i64, _i64, _p, _p, _sz, _p]
lib.dg_soft_embed_shard_begin.restype = ctypes.c_int
lib.dg_soft_embed_shard_end.argtypes = [_p, _i64, _p, _i64, _i64, _p, _i64, _i64, _i64, _f32, _p, _i64, _p, _sz, _p]
lib.dg_soft_embed_shard_end.restype = ctypes.c_int
lib.dg_soft_embed_shard_begin_e4m3.argtypes = [_p, _i64, _i64, _i64, _i64, _p, _p, _i64, _i64, _i64, _p, _p, _sz, _p]
lib.dg_soft_embed_shard_begin_e4m3.restype = ctypes.c_int
lib.dg_soft_embed_shard_end_e4m3.argtypes = [_p, _i64, _p, _i64, _i64, _p, _p, _i64, _i64, _i64, _f32, _p, _i64, _p,
                                             _sz, _p]
lib.dg_soft_embed_shard_end_e4m3.restype = ctypes.c_int

_ROWS = [_p, _i32, _i64, _i64, _i64]  # logits, dtype, R, V, ldl
lib.dg_row_topk_workspace_size.argtypes = [_i64, _i64, _i32, _i32]
lib.dg_row_topk_workspace_size.restype = _sz
lib.dg_row_topk.argtypes = _ROWS + [_i32, _f32, _p, _p, _i64, _p, _p, _sz, _p]
lib.dg_row_topk.restype = ctypes.c_int
lib.dg_row_loss_workspace_size.argtypes = [_i64, _i64, _i32]
lib.dg_row_loss_workspace_size.restype = _sz
lib.dg_row_loss_needs_workspace.argtypes = [_i64, _i32]
lib.dg_row_loss_needs_workspace.restype = _i32
lib.dg_token_logp.argtypes = _ROWS + [_p, _f32, _p, _p, _p, _p, _sz, _p]
lib.dg_token_logp.restype = ctypes.c_int
lib.dg_token_logp_backward.argtypes = _ROWS + [_p, _f32, _p, _p, _p, _p, _i64, _p, _sz, _p]
lib.dg_token_logp_backward.restype = ctypes.c_int
lib.dg_distill_loss.argtypes = _ROWS + [_p, _p, _i32, _i64, _p, _f32, _p, _p, _p, _p, _p, _i64, _p, _sz, _p]
lib.dg_distill_loss.restype = ctypes.c_int
lib.dg_distill_loss_backward.argtypes = _ROWS + [_p, _p, _i32, _i64, _p, _f32, _p, _p, _p, _p, _i64, _p, _sz, _p]
lib.dg_distill_loss_backward.restype = ctypes.c_int
lib.dg_policy_loss.argtypes = _ROWS + [_p, _p, _p, _p, _f32, _f32, _f32, _f32] + [_p] * 8 + [_i64, _p, _sz, _p]
lib.dg_policy_loss.restype = ctypes.c_int
lib.dg_preference_loss.argtypes = _ROWS + [_p, _p, _p, _i32, _f32, _f32, _f32] + [_p] * 8 + [_i64, _p, _sz, _p]
lib.dg_preference_loss.restype = ctypes.c_int

lib.dg_token_embed.argtypes = [_p, _i32, _p, _i64, _i64, _i64, _i64, _i64, _i64, _p, _i64, _f32, _p, _i32, _i64, _p]
lib.dg_token_embed.restype = ctypes.c_int
lib.dg_token_embed_backward.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i64, _i64, _i64, _f32, _p, _i32, _i64, _i64,
                                        _i32, _p, _sz, _p]
lib.dg_token_embed_backward.restype = ctypes.c_int
lib.dg_token_embed_backward_workspace_size.argtypes = [_i64, _i64, _i64]
lib.dg_token_embed_backward_workspace_size.restype = _sz
lib.dg_rms_norm.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i32, _i64, _p, _i32, _f32, _f32, _p, _i32, _i64, _p, _i32,
                            _i64, _p, _p, _p]
lib.dg_rms_norm.restype = ctypes.c_int
lib.dg_rms_norm_backward.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _i32, _i64, _p, _p, _i32, _f32, _p, _i32, _i64, _p,
                                     _i64, _p, _p, _sz, _p]
lib.dg_rms_norm_backward.restype = ctypes.c_int
lib.dg_rms_norm_backward_workspace_size.argtypes = [_i64, _i64]
lib.dg_rms_norm_backward_workspace_size.restype = _sz
lib.dg_head_e4m3.argtypes = [_p, _i64, _p, _i64, _i64, _p, _p, _i64, _i64, _p, _i32, _i64, _p]
lib.dg_head_e4m3.restype = ctypes.c_int

# element types of logits, gradients and the hidden stream's matrices (dg_dtype)
DG_F32, DG_BF16, DG_E4M3 = 0, 1, 2
_DTYPE = {torch.float32: DG_F32, torch.bfloat16: DG_BF16}
_DTYPE_CODES = {**_DTYPE, torch.uint8: DG_E4M3}

STATUS = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED", 3: "DG_ERR_CUDA", 4: "DG_ERR_TIMEOUT"}


class DgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.dg_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS.get(status, status)}: {msg}")


def _check(status: int, where: str) -> None:
    if status != 0:
        raise DgError(status, where)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    # the current stream's handle without the Stream object, which costs a small call a tenth of its time
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _ld(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit column stride")
    return t.stride(0)


def _flags(two_pass: bool) -> int:
    return DG_STEP_TWO_PASS if two_pass else 0


def _new(shape, dtype, device):
    return torch.empty(shape, dtype=dtype, device=device)


def dg_row_stats(logits: torch.Tensor, V: int | None = None, stream=None, out: dict | None = None) -> dict:
    """Row statistics of fp32 logits [R, >=V] -> dict m, lse, H, kappa (fp32), argmax (int32)."""
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    dev = logits.device
    o = out
    if o is None:
        o = {k: _new(R, torch.float32, dev) for k in ("m", "lse", "H", "kappa")}
        o["argmax"] = _new(R, torch.int32, dev)
    _check(lib.dg_row_stats(_ptr(logits), R, V, _ld(logits), _ptr(o["m"]), _ptr(o["lse"]), _ptr(o["H"]),
                            _ptr(o["kappa"]), _ptr(o["argmax"]), _stream(stream)), "dg_row_stats")
    return o


def dg_row_sample(logits: torch.Tensor, temperature: float = 1.0, seed: int = 0, offset: int = 0,
                  V: int | None = None, stream=None, out: dict | None = None) -> dict:
    """Gumbel-max candidate per row of fp32 logits [R, >=V] at `temperature`, uniforms from
    Philox4x32-10 keyed by `seed` at step `offset` -> dict candidate (int32), log_p (fp32)."""
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    dev = logits.device
    o = out
    if o is None:
        o = {"candidate": _new(R, torch.int32, dev), "log_p": _new(R, torch.float32, dev)}
    _check(lib.dg_row_sample(_ptr(logits), R, V, _ld(logits), float(temperature), int(seed), int(offset),
                             _ptr(o["candidate"]), _ptr(o["log_p"]), _stream(stream)), "dg_row_sample")
    return o


def dg_row_stats_partial(shard: torch.Tensor, vocab_offset: int, n: int | None = None, stream=None,
                         out: torch.Tensor | None = None) -> torch.Tensor:
    """The shard's 16-byte summary per row: a [R, 4] float32 tensor whose column 1 holds the
    int32 bits of the global argmax (view it with .view(torch.int32))."""
    R = shard.shape[0]
    n = shard.shape[1] if n is None else n
    o = out if out is not None else _new((R, 4), torch.float32, shard.device)
    _check(lib.dg_row_stats_partial(_ptr(shard), R, n, _ld(shard), vocab_offset, _ptr(o), _stream(stream)),
           "dg_row_stats_partial")
    return o


def dg_soft_embed_shard_begin(shard: torch.Tensor, vocab_offset: int, W_shard, ws: torch.Tensor,
                              stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """First call of a shard's one-read soft embedding: the shard's [R, 4] row summaries (the
    format of dg_row_stats_partial); the split partials stay in `ws` for dg_soft_embed_shard_end.
    W_shard: bf16 [rows_pad, >= d], or an 8-bit table (codes, row scales)."""
    R, n = shard.shape
    o = out if out is not None else _new((R, 4), torch.float32, shard.device)
    if isinstance(W_shard, tuple):
        Q, scale = W_shard
        _check(lib.dg_soft_embed_shard_begin_e4m3(_ptr(shard), _ld(shard), R, n, vocab_offset, _ptr(Q), _ptr(scale),
                                                  Q.shape[0], _ld(Q), Q.shape[1], _ptr(o), _ptr(ws), ws.numel(),
                                                  _stream(stream)), "dg_soft_embed_shard_begin_e4m3")
    else:
        _check(lib.dg_soft_embed_shard_begin(_ptr(shard), _ld(shard), R, n, vocab_offset, _ptr(W_shard),
                                             W_shard.shape[0], _ld(W_shard), W_shard.shape[1], _ptr(o), _ptr(ws),
                                             ws.numel(), _stream(stream)), "dg_soft_embed_shard_begin")
    return o


def dg_soft_embed_shard_end(shard: torch.Tensor, lse: torch.Tensor, W_shard, gamma: float, ws: torch.Tensor,
                            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Second call: gamma * E_shard [R, d] from the partials the first call left in `ws`, scaled
    against the full-row lse."""
    R, n = shard.shape
    d = W_shard[0].shape[1] if isinstance(W_shard, tuple) else W_shard.shape[1]
    if out is None:
        out = _new((R, d), torch.float32, shard.device)
    if isinstance(W_shard, tuple):
        Q, scale = W_shard
        _check(lib.dg_soft_embed_shard_end_e4m3(_ptr(shard), _ld(shard), _ptr(lse), R, n, _ptr(Q), _ptr(scale),
                                                Q.shape[0], _ld(Q), d, gamma, _ptr(out), _ld(out), _ptr(ws),
                                                ws.numel(), _stream(stream)), "dg_soft_embed_shard_end_e4m3")
    else:
        _check(lib.dg_soft_embed_shard_end(_ptr(shard), _ld(shard), _ptr(lse), R, n, _ptr(W_shard),
                                           W_shard.shape[0], _ld(W_shard), d, gamma, _ptr(out), _ld(out), _ptr(ws),
                                           ws.numel(), _stream(stream)), "dg_soft_embed_shard_end")
    return out


def dg_soft_embed_shard_begin_e4m3(shard: torch.Tensor, vocab_offset: int, Q_shard: torch.Tensor,
                                   scale_shard: torch.Tensor, ws: torch.Tensor, stream=None,
                                   out: torch.Tensor | None = None) -> torch.Tensor:
    """dg_soft_embed_shard_begin over an 8-bit table shard (codes, row scales)."""
    return dg_soft_embed_shard_begin(shard, vocab_offset, (Q_shard, scale_shard), ws, stream=stream, out=out)


def dg_soft_embed_shard_end_e4m3(shard: torch.Tensor, lse: torch.Tensor, Q_shard: torch.Tensor,
                                 scale_shard: torch.Tensor, gamma: float, ws: torch.Tensor,
                                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dg_soft_embed_shard_end over an 8-bit table shard (codes, row scales)."""
    return dg_soft_embed_shard_end(shard, lse, (Q_shard, scale_shard), gamma, ws, out=out, stream=stream)


def dg_row_stats_combine(states: torch.Tensor, stream=None, out: dict | None = None) -> dict:
    """Full-row statistics from [T, R, 4] shard summaries in shard order."""
    T, R = states.shape[0], states.shape[1]
    dev = states.device
    o = out if out is not None else {"m": _new(R, torch.float32, dev), "lse": _new(R, torch.float32, dev),
                                     "H": _new(R, torch.float32, dev), "kappa": _new(R, torch.float32, dev),
                                     "argmax": _new(R, torch.int32, dev)}
    _check(lib.dg_row_stats_combine(_ptr(states), T, R, _ptr(o.get("m")), _ptr(o.get("lse")), _ptr(o.get("H")),
                                    _ptr(o.get("kappa")), _ptr(o.get("argmax")), _stream(stream)),
           "dg_row_stats_combine")
    return o


def dg_row_stats_sample(logits: torch.Tensor, temperature: float = 1.0, seed: int = 0, offset: int = 0,
                        V: int | None = None, stream=None, out: dict | None = None) -> dict:
    """Row statistics and a drawn candidate in one pass; kappa = -ln p(candidate)."""
    R = logits.shape[0]
    V = logits.shape[1] if V is None else V
    dev = logits.device
    o = out if out is not None else {
        "m": _new(R, torch.float32, dev), "lse": _new(R, torch.float32, dev), "H": _new(R, torch.float32, dev),
        "kappa": _new(R, torch.float32, dev), "argmax": _new(R, torch.int32, dev),
        "candidate": _new(R, torch.int32, dev), "log_p": _new(R, torch.float32, dev)}
    _check(lib.dg_row_stats_sample(_ptr(logits), R, V, _ld(logits), temperature, seed, offset, _ptr(o.get("m")),
                                   _ptr(o.get("lse")), _ptr(o.get("H")), _ptr(o.get("kappa")),
                                   _ptr(o.get("argmax")), _ptr(o["candidate"]), _ptr(o.get("log_p")),
                                   _stream(stream)), "dg_row_stats_sample")
    return o


def dg_soft_embed_workspace_size(R: int, vocab_len: int, d: int) -> int:
    return int(lib.dg_soft_embed_workspace_size(R, vocab_len, d))


def workspace(R: int, vocab_len: int, d: int, device) -> torch.Tensor:
    """A workspace tensor large enough for dg_soft_embed / dg_sampler_step."""
    n = max(16, dg_soft_embed_workspace_size(R, vocab_len, d))
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def dg_soft_embed(logits: torch.Tensor, lse: torch.Tensor, vocab_start: int, vocab_end: int,
                  W_shard: torch.Tensor, gamma: float, out: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None, R: int | None = None) -> torch.Tensor:
    """E = gamma * softmax(logits)[:, s:e] @ W_shard[0:e-s] (W_shard: bf16 [rows_pad, >=d])."""
    R = logits.shape[0] if R is None else R
    d = W_shard.shape[1]
    if W_shard.dtype not in (torch.bfloat16, torch.int16):
        raise TypeError("W_shard must hold bfloat16 values")
    if out is None:
        out = _new((R, d), torch.float32, logits.device)
    if ws is None:
        ws = workspace(R, max(1, vocab_end - vocab_start), d, logits.device)
    _check(lib.dg_soft_embed(_ptr(logits), _ld(logits), _ptr(lse), R, vocab_start, vocab_end, _ptr(W_shard),
                             W_shard.shape[0], _ld(W_shard), d, gamma, _ptr(out), _ld(out), _ptr(ws), ws.numel(),
                             _stream(stream)), "dg_soft_embed")
    return out


def dg_soft_embed_no_alloc(logits: torch.Tensor, lse: torch.Tensor, vocab_start: int, vocab_end: int,
                           W_shard: torch.Tensor, gamma: float, out: torch.Tensor, stream=None,
                           R: int | None = None) -> torch.Tensor:
    """dg_soft_embed without a workspace: the library's fixed scratch array holds the
    partial tiles.  `out` [R, >=d] fp32 must be given; nothing is allocated."""
    R = logits.shape[0] if R is None else R
    d = W_shard.shape[1]
    _check(lib.dg_soft_embed_no_alloc(_ptr(logits), _ld(logits), _ptr(lse), R, vocab_start, vocab_end,
                                      _ptr(W_shard), W_shard.shape[0], _ld(W_shard), d, gamma, _ptr(out), _ld(out),
                                      _stream(stream)), "dg_soft_embed_no_alloc")
    return out


def dg_quantize_e4m3(W: torch.Tensor, stream=None) -> tuple:
    """Per-row E4M3 quantisation of a bf16 table [V, >=d] -> (Q, scale): Q a uint8 [V, d] view
    of a buffer whose rows are padded to a multiple of 16 bytes, scale fp32 [V]."""
    if W.dtype not in (torch.bfloat16, torch.int16):
        raise TypeError("W must hold bfloat16 values")
    V, d = W.shape
    ldq = (d + 15) // 16 * 16
    Q = _new((V, ldq), torch.uint8, W.device)
    scale = _new(V, torch.float32, W.device)
    _check(lib.dg_quantize_e4m3(_ptr(W), V, d, _ld(W), _ptr(Q), ldq, _ptr(scale), _stream(stream)),
           "dg_quantize_e4m3")
    return Q[:, :d], scale


def dg_soft_embed_workspace_size_e4m3(R: int, vocab_len: int, d: int) -> int:
    return int(lib.dg_soft_embed_workspace_size_e4m3(R, vocab_len, d))


def workspace_e4m3(R: int, vocab_len: int, d: int, device) -> torch.Tensor:
    """A workspace tensor large enough for dg_soft_embed_e4m3 / dg_sampler_step_e4m3."""
    n = max(16, dg_soft_embed_workspace_size_e4m3(R, vocab_len, d))
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def dg_soft_embed_e4m3(logits: torch.Tensor, lse: torch.Tensor, vocab_start: int, vocab_end: int,
                       Q_shard: torch.Tensor, scale_shard: torch.Tensor, gamma: float, out: torch.Tensor | None = None,
                       ws: torch.Tensor | None = None, stream=None, R: int | None = None) -> torch.Tensor:
    """E = gamma * softmax(logits)[:, s:e] @ (scale * e4m3(Q_shard))[0:e-s] (Q_shard uint8 [rows_pad, d])."""
    R = logits.shape[0] if R is None else R
    d = Q_shard.shape[1]
    if Q_shard.dtype != torch.uint8 or scale_shard.dtype != torch.float32:
        raise TypeError("Q_shard must be uint8 codes and scale_shard fp32")
    if out is None:
        out = _new((R, d), torch.float32, logits.device)
    if ws is None:
        ws = workspace_e4m3(R, max(1, vocab_end - vocab_start), d, logits.device)
    _check(lib.dg_soft_embed_e4m3(_ptr(logits), _ld(logits), _ptr(lse), R, vocab_start, vocab_end, _ptr(Q_shard),
                                  _ptr(scale_shard), Q_shard.shape[0], _ld(Q_shard), d, gamma, _ptr(out), _ld(out),
                                  _ptr(ws), ws.numel(), _stream(stream)), "dg_soft_embed_e4m3")
    return out


def dg_sampler_step_e4m3(logits: torch.Tensor, n_req: int, L_c: int, Q: torch.Tensor, scale: torch.Tensor,
                         gamma: float, budgets: torch.Tensor, min_accept: int = 0, vocab_start: int = 0,
                         vocab_end: int | None = None, V: int | None = None, out: dict | None = None,
                         ws: torch.Tensor | None = None, stream=None, two_pass: bool = False) -> dict:
    """dg_sampler_step with the 8-bit table (Q uint8 [rows_pad, d], scale fp32 [rows_pad])."""
    R = n_req * L_c
    V = logits.shape[1] if V is None else V
    vocab_end = V if vocab_end is None else vocab_end
    d = Q.shape[1]
    dev = logits.device
    o = out
    if o is None:
        o = {k: _new(R, torch.float32, dev) for k in ("m", "lse", "H", "kappa")}
        o.update(argmax=_new(R, torch.int32, dev), order=_new(R, torch.int32, dev), mask=_new(R, torch.uint8, dev),
                 n_accepted=_new(n_req, torch.int32, dev), E=_new((R, d), torch.float32, dev))
    if ws is None:
        ws = workspace_e4m3(R, max(1, vocab_end - vocab_start), d, dev)
    _check(lib.dg_sampler_step_e4m3(_ptr(logits), n_req, L_c, V, _ld(logits), _ptr(Q), _ptr(scale), vocab_start,
                                    vocab_end, Q.shape[0], _ld(Q), d, gamma, _ptr(budgets), min_accept,
                                    _ptr(o["m"]), _ptr(o["lse"]), _ptr(o["H"]), _ptr(o["kappa"]), _ptr(o["argmax"]),
                                    _ptr(o["order"]), _ptr(o["mask"]), _ptr(o["n_accepted"]), _ptr(o["E"]),
                                    _ld(o["E"]), _flags(two_pass), _ptr(ws), ws.numel(), _stream(stream)),
           "dg_sampler_step_e4m3")
    return o


def dg_entropy_accept(H: torch.Tensor, kappa: torch.Tensor, n_req: int, L_c: int, budgets: torch.Tensor,
                      min_accept: int = 0, stream=None, out: dict | None = None) -> dict:
    dev = H.device
    R = n_req * L_c
    o = out if out is not None else {"order": _new(R, torch.int32, dev), "mask": _new(R, torch.uint8, dev),
                                     "n_accepted": _new(n_req, torch.int32, dev)}
    _check(lib.dg_entropy_accept(_ptr(H), _ptr(kappa), n_req, L_c, _ptr(budgets), min_accept, _ptr(o["order"]),
                                 _ptr(o["mask"]), _ptr(o["n_accepted"]), _stream(stream)), "dg_entropy_accept")
    return o


def dg_sum_partials(partials: list, gamma: float, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    R, d = partials[0].shape
    ldp = _ld(partials[0])
    if any(tuple(p.shape) != (R, d) or _ld(p) != ldp for p in partials):
        raise ValueError("partials must share shape and leading dimension")
    if out is None:
        out = _new((R, d), torch.float32, partials[0].device)
    arr = (_p * len(partials))(*[p.data_ptr() for p in partials])
    _check(lib.dg_sum_partials(arr, len(partials), R, d, ldp, gamma, _ptr(out), _ld(out), _stream(stream)),
           "dg_sum_partials")
    return out


def dg_sampler_step(logits: torch.Tensor, n_req: int, L_c: int, W: torch.Tensor, gamma: float,
                    budgets: torch.Tensor, min_accept: int = 0, vocab_start: int = 0, vocab_end: int | None = None,
                    V: int | None = None, out: dict | None = None, ws: torch.Tensor | None = None,
                    stream=None, two_pass: bool = False) -> dict:
    """One fused sampler step; returns dict m, lse, H, kappa, argmax, order, mask, n_accepted, E.
    two_pass: statistics before the product even over the whole vocabulary (DG_STEP_TWO_PASS)."""
    R = n_req * L_c
    V = logits.shape[1] if V is None else V
    vocab_end = V if vocab_end is None else vocab_end
    d = W.shape[1]
    dev = logits.device
    o = out
    if o is None:
        o = {k: _new(R, torch.float32, dev) for k in ("m", "lse", "H", "kappa")}
        o.update(argmax=_new(R, torch.int32, dev), order=_new(R, torch.int32, dev), mask=_new(R, torch.uint8, dev),
                 n_accepted=_new(n_req, torch.int32, dev), E=_new((R, d), torch.float32, dev))
    if ws is None:
        ws = workspace(R, max(1, vocab_end - vocab_start), d, dev)
    _check(lib.dg_sampler_step(_ptr(logits), n_req, L_c, V, _ld(logits), _ptr(W), vocab_start, vocab_end,
                               W.shape[0], _ld(W), d, gamma, _ptr(budgets), min_accept, _ptr(o["m"]), _ptr(o["lse"]),
                               _ptr(o["H"]), _ptr(o["kappa"]), _ptr(o["argmax"]), _ptr(o["order"]), _ptr(o["mask"]),
                               _ptr(o["n_accepted"]), _ptr(o["E"]), _ld(o["E"]), _flags(two_pass), _ptr(ws),
                               ws.numel(), _stream(stream)), "dg_sampler_step")
    return o


def dg_entropy_accept_eligible(H: torch.Tensor, kappa: torch.Tensor, eligible: torch.Tensor, n_req: int, L_c: int,
                               budgets: torch.Tensor, min_accept: int = 0, stream=None, out: dict | None = None) -> dict:
    dev = H.device
    R = n_req * L_c
    o = out if out is not None else {"order": _new(R, torch.int32, dev), "mask": _new(R, torch.uint8, dev),
                                     "n_accepted": _new(n_req, torch.int32, dev)}
    _check(lib.dg_entropy_accept_eligible(_ptr(H), _ptr(kappa), _ptr(eligible), n_req, L_c, _ptr(budgets), min_accept,
                                          _ptr(o["order"]), _ptr(o["mask"]), _ptr(o["n_accepted"]), _stream(stream)),
           "dg_entropy_accept_eligible")
    return o


LOOP_STATE_KEYS = ("canvas", "eligible", "prev_argmax", "stable", "steps", "converged")


def new_loop_state(n_req: int, L_c: int, device, canvas0: torch.Tensor | None = None) -> dict:
    """The state buffers a denoising loop starts from, as the C API documents them:
    prev_argmax -1, stable and steps 0, every position eligible, the canvas as given."""
    R = n_req * L_c
    canvas = torch.zeros(R, dtype=torch.int32, device=device) if canvas0 is None else \
        canvas0.to(device=device, dtype=torch.int32).reshape(R).clone()
    return {"canvas": canvas, "eligible": torch.ones(R, dtype=torch.uint8, device=device),
            "prev_argmax": torch.full((R,), -1, dtype=torch.int32, device=device),
            "stable": torch.zeros(n_req, dtype=torch.int32, device=device),
            "steps": torch.zeros(n_req, dtype=torch.int32, device=device),
            "converged": torch.zeros(n_req, dtype=torch.uint8, device=device)}


def dg_loop_update(candidate: torch.Tensor, H: torch.Tensor, mask: torch.Tensor, n_req: int, L_c: int,
                   state: dict, stable_steps: int, entropy_threshold: float, step_limit: int,
                   argmax: torch.Tensor | None = None, stream=None) -> dict:
    """Updates `state` (see new_loop_state) in place after one step; returns it.  The
    canvas takes `candidate`; stability is judged on `argmax` (default: the candidates)."""
    am = candidate if argmax is None else argmax
    _check(lib.dg_loop_update(_ptr(candidate), _ptr(am), _ptr(H), _ptr(mask), n_req, L_c, stable_steps,
                              entropy_threshold,
                              step_limit, *[_ptr(state[k]) for k in LOOP_STATE_KEYS], _stream(stream)),
           "dg_loop_update")
    return state


def dg_sampler_loop_step(logits: torch.Tensor, n_req: int, L_c: int, W: torch.Tensor, gamma: float,
                         budgets: torch.Tensor, state: dict, stable_steps: int, entropy_threshold: float,
                         step_limit: int, min_accept: int = 0, vocab_start: int = 0, vocab_end: int | None = None,
                         V: int | None = None, out: dict | None = None, ws: torch.Tensor | None = None,
                         temperature: float = 0.0, seed: int = 0, offset: int = 0, stream=None,
                         two_pass: bool = False) -> dict:
    """One denoising-loop step: the fused step over the eligible positions, then the loop
    update of `state` in place.  Returns the step outputs as dg_sampler_step does, plus
    `candidate` (the drawn tokens) when temperature > 0."""
    R = n_req * L_c
    V = logits.shape[1] if V is None else V
    vocab_end = V if vocab_end is None else vocab_end
    d = W.shape[1]
    dev = logits.device
    o = out
    if o is None:
        o = {k: _new(R, torch.float32, dev) for k in ("m", "lse", "H", "kappa")}
        o.update(argmax=_new(R, torch.int32, dev), order=_new(R, torch.int32, dev), mask=_new(R, torch.uint8, dev),
                 n_accepted=_new(n_req, torch.int32, dev), E=_new((R, d), torch.float32, dev))
    if temperature != 0.0 and "candidate" not in o:
        o["candidate"] = _new(R, torch.int32, dev)
    if ws is None:
        ws = workspace(R, max(1, vocab_end - vocab_start), d, dev)
    _check(lib.dg_sampler_loop_step(_ptr(logits), n_req, L_c, V, _ld(logits), _ptr(W), vocab_start, vocab_end,
                                    W.shape[0], _ld(W), d, gamma, _ptr(budgets), min_accept, stable_steps,
                                    entropy_threshold, step_limit, temperature, seed, offset, _ptr(o["m"]),
                                    _ptr(o["lse"]), _ptr(o["H"]), _ptr(o["kappa"]), _ptr(o["argmax"]),
                                    _ptr(o.get("candidate")), _ptr(o["order"]), _ptr(o["mask"]),
                                    _ptr(o["n_accepted"]), _ptr(o["E"]), _ld(o["E"]),
                                    *[_ptr(state[k]) for k in LOOP_STATE_KEYS], _flags(two_pass), _ptr(ws),
                                    ws.numel(), _stream(stream)), "dg_sampler_loop_step")
    return o


def dg_sampler_loop_step_e4m3(logits: torch.Tensor, n_req: int, L_c: int, Q: torch.Tensor, scale: torch.Tensor,
                              gamma: float, budgets: torch.Tensor, state: dict, stable_steps: int,
                              entropy_threshold: float, step_limit: int, min_accept: int = 0, vocab_start: int = 0,
                              vocab_end: int | None = None, V: int | None = None, out: dict | None = None,
                              ws: torch.Tensor | None = None, temperature: float = 0.0, seed: int = 0, offset: int = 0,
                              stream=None, two_pass: bool = False) -> dict:
    """dg_sampler_loop_step with the 8-bit table (Q uint8 [rows_pad, d], scale fp32 [rows_pad])."""
    R = n_req * L_c
    V = logits.shape[1] if V is None else V
    vocab_end = V if vocab_end is None else vocab_end
    d = Q.shape[1]
    dev = logits.device
    o = out
    if o is None:
        o = {k: _new(R, torch.float32, dev) for k in ("m", "lse", "H", "kappa")}
        o.update(argmax=_new(R, torch.int32, dev), order=_new(R, torch.int32, dev), mask=_new(R, torch.uint8, dev),
                 n_accepted=_new(n_req, torch.int32, dev), E=_new((R, d), torch.float32, dev))
    if temperature != 0.0 and "candidate" not in o:
        o["candidate"] = _new(R, torch.int32, dev)
    if ws is None:
        ws = workspace_e4m3(R, max(1, vocab_end - vocab_start), d, dev)
    _check(lib.dg_sampler_loop_step_e4m3(_ptr(logits), n_req, L_c, V, _ld(logits), _ptr(Q), _ptr(scale), vocab_start,
                                         vocab_end, Q.shape[0], _ld(Q), d, gamma, _ptr(budgets), min_accept,
                                         stable_steps, entropy_threshold, step_limit, temperature, seed, offset,
                                         _ptr(o["m"]), _ptr(o["lse"]), _ptr(o["H"]), _ptr(o["kappa"]),
                                         _ptr(o["argmax"]), _ptr(o.get("candidate")), _ptr(o["order"]),
                                         _ptr(o["mask"]), _ptr(o["n_accepted"]), _ptr(o["E"]), _ld(o["E"]),
                                         *[_ptr(state[k]) for k in LOOP_STATE_KEYS], _flags(two_pass), _ptr(ws),
                                         ws.numel(), _stream(stream)), "dg_sampler_loop_step_e4m3")
    return o


def dg_get_device_status(stream=None) -> None:
    _check(lib.dg_get_device_status(_stream(stream)), "dg_get_device_status")


def dg_check_wait_timeout(limit_us: int, stream=None) -> None:
    """Queues the diagnostic wait that gives up after limit_us; the next
    dg_get_device_status() raises DgError with DG_ERR_TIMEOUT."""
    _check(lib.dg_check_wait_timeout(int(limit_us), _stream(stream)), "dg_check_wait_timeout")


# --------------------------------------------------------------------------- training on the logits
#
# Common to the calls below: `logits` [R, V] in fp32 or bf16 with unit column stride, V taken from its
# shape (slice the padding off: logits[:, :V]); per-row vectors are contiguous, on the logits' device;
# `out` holds preallocated outputs by name, and an output it lacks is allocated.  `stream` is the
# stream the kernels run on; its tensors are the caller's to keep alive and ordered, as everywhere.

def _logits(t: torch.Tensor) -> tuple:
    """(pointer, dtype code, R, V, row stride) of a matrix of logits."""
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError("logits must be on the GPU")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"logits are on {t.device}, and the kernels would run on the current device, "
                         f"cuda:{torch._C._cuda_getDevice()}: use torch.cuda.device(logits.device)")
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("logits must be [R, V] with unit column stride")
    R, V = t.shape
    return t.data_ptr(), code, R, V, _row_stride(t)


def _row_stride(t: torch.Tensor) -> int:
    """Elements between rows.  The stride of a single row says nothing and is rounded up to 16 bytes."""
    if t.shape[0] > 1:
        return t.stride(0)
    per = 16 // t.element_size()
    return (t.shape[1] + per - 1) // per * per


def _vec(t, n: int, dtype, device, name: str):
    """Pointer of a contiguous vector of n elements (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _grad_like(grad: torch.Tensor, logits: torch.Tensor) -> tuple:
    """(pointer, row stride) of a gradient of these logits."""
    if grad.dtype is not logits.dtype or grad.shape != logits.shape or grad.device != logits.device:
        raise ValueError("grad must have the logits' type, shape and device")
    if grad.stride(1) != 1 and grad.shape[1] > 1:
        raise ValueError("grad must have unit column stride")
    return grad.data_ptr(), _row_stride(grad)


def _new_grad(logits: torch.Tensor, stream) -> torch.Tensor:
    """An uninitialised gradient [R, V] whose rows start on 16-byte boundaries."""
    R, V = logits.shape
    per = 16 // logits.element_size()
    with _on(stream):
        return _new((R, (V + per - 1) // per * per), logits.dtype, logits.device)[:, :V]


def _on(stream):
    """Allocations inside belong to the stream that writes them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _fill(out: dict | None, shapes: dict, device, stream) -> dict:
    """`out` with the missing outputs of {name: (shape, dtype)} allocated."""
    if out is not None and shapes.keys() <= out.keys():
        return out
    o = {} if out is None else out
    with _on(stream):
        for k in shapes:
            if k not in o:
                o[k] = _new(shapes[k][0], shapes[k][1], device)
    return o


def _table(t: torch.Tensor, R: int, K: int, dtype, device, name: str) -> int:
    """Row stride of an [R, K] table with unit column stride."""
    if t.dtype is not dtype or t.shape != (R, K) or t.device != device or (K > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be {dtype} [{R}, {K}] with unit column stride on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.stride(0) if R > 1 else K


def _entries(indices, teacher, R: int, device) -> tuple:
    """(K, row stride) of a teacher's entries."""
    if indices.dim() != 2:
        raise ValueError("indices must be [R, K]")
    K = indices.shape[1]
    ld = _table(indices, R, K, torch.int32, device, "indices")
    if _table(teacher, R, K, torch.float32, device, "teacher") != ld:
        raise ValueError("indices and teacher must have the same row stride")
    return K, ld


def dg_row_loss_workspace_size(R: int, V: int, dtype: int = DG_F32) -> int:
    return int(lib.dg_row_loss_workspace_size(R, V, dtype))


@functools.lru_cache(maxsize=256)
def dg_row_loss_needs_workspace(V: int, dtype: int = DG_F32) -> bool:
    """Whether the loss calls but dg_distill_loss_backward, which always does, need a workspace."""
    return bool(lib.dg_row_loss_needs_workspace(V, dtype))


def loss_workspace(R: int, V: int, device, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """A workspace tensor large enough for the loss calls."""
    n = max(16, dg_row_loss_workspace_size(R, V, _DTYPE[dtype]))
    return torch.empty(n, dtype=torch.uint8, device=device)


def _memory(ws: torch.Tensor, device) -> tuple:
    """(pointer, bytes) of a workspace tensor of any type."""
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous tensor on {device}, got strides {ws.stride()} on {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _loss_ws(ws, R: int, V: int, code: int, device, stream, always: bool = False) -> tuple:
    """(tensor, pointer, bytes) of the caller's workspace, of a new one (its memory stays with the stream
    that uses it), or of none where the call needs none."""
    if not always and not dg_row_loss_needs_workspace(V, code):
        return None, None, 0
    if ws is None:
        n = max(16, dg_row_loss_workspace_size(R, V, code))
        with _on(stream):
            ws = torch.empty(n, dtype=torch.uint8, device=device)
    return (ws, *_memory(ws, device))


def dg_row_topk_workspace_size(R: int, V: int, K: int, dtype: int = DG_F32) -> int:
    return int(lib.dg_row_topk_workspace_size(R, V, K, dtype))


def topk_workspace(R: int, V: int, K: int, device, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """A workspace tensor large enough for dg_row_topk."""
    n = max(16, dg_row_topk_workspace_size(R, V, K, _DTYPE[dtype]))
    return torch.empty((n + 15) // 16 * 16, dtype=torch.uint8, device=device)


def dg_row_topk(logits: torch.Tensor, K: int, temperature: float = 1.0, lse: bool = False,
                ws: torch.Tensor | None = None, stream=None, out: dict | None = None) -> dict:
    """The K largest logits per row, in order, ties to the lowest index -> dict values (fp32 [R, K]),
    indices (int32 [R, K]) and, with lse=True or an `lse` in `out`, the log-sum-exp of logits / T."""
    x, code, R, V, ld = _logits(logits)
    dev = logits.device
    shapes = {"values": ((R, K), torch.float32), "indices": ((R, K), torch.int32)}
    if lse:
        shapes["lse"] = (R, torch.float32)
    o = _fill(out, shapes, dev, stream)
    ldk = _table(o["values"], R, K, torch.float32, dev, "values")
    if _table(o["indices"], R, K, torch.int32, dev, "indices") != ldk:
        raise ValueError("values and indices must have the same row stride")
    if ws is None:
        with _on(stream):
            ws = topk_workspace(R, V, K, dev, logits.dtype)
    ws_ptr, ws_bytes = _memory(ws, dev)
    _check(lib.dg_row_topk(x, code, R, V, ld, K, temperature, o["values"].data_ptr(), o["indices"].data_ptr(), ldk,
                           _vec(o.get("lse"), R, torch.float32, dev, "lse"), ws_ptr, ws_bytes,
                           _stream(stream)), "dg_row_topk")
    return o


def dg_token_logp(logits: torch.Tensor, token: torch.Tensor, temperature: float = 1.0,
                  weight: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None,
                  out: dict | None = None) -> dict:
    """ln softmax(logits / T)[token] per row -> dict logp, lse (fp32 [R]).  Rows of weight 0 or with a
    negative token are left out (0)."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    o = _fill(out, {"logp": (R, f32), "lse": (R, f32)}, dev, stream)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream)
    _check(lib.dg_token_logp(x, code, R, V, ld, _vec(token, R, torch.int32, dev, "token"), temperature,
                             _vec(weight, R, f32, dev, "weight"), _vec(o["logp"], R, f32, dev, "logp"),
                             _vec(o["lse"], R, f32, dev, "lse"), ws_ptr, ws_bytes, _stream(stream)),
           "dg_token_logp")
    return o


def dg_token_logp_backward(logits: torch.Tensor, token: torch.Tensor, lse: torch.Tensor, dlogp: torch.Tensor,
                           scale: torch.Tensor | None = None, temperature: float = 1.0,
                           ws: torch.Tensor | None = None, stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient of sum_r scale_r dlogp_r logp_r from a forward call's lse (scale: the upstream
    gradient per row).  `out` may be the logits themselves."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    if out is None:
        out = _new_grad(logits, stream)
    g, ldg = _grad_like(out, logits)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream)
    _check(lib.dg_token_logp_backward(x, code, R, V, ld, _vec(token, R, torch.int32, dev, "token"), temperature,
                                      _vec(lse, R, f32, dev, "lse"), _vec(dlogp, R, f32, dev, "dlogp"),
                                      _vec(scale, R, f32, dev, "scale"), g, ldg, ws_ptr, ws_bytes,
                                      _stream(stream)),
           "dg_token_logp_backward")
    return out


def dg_distill_loss(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                    teacher_lse: torch.Tensor | None = None, temperature: float = 1.0,
                    weight: torch.Tensor | None = None, grad: bool = False,
                    ws: torch.Tensor | None = None, stream=None, out: dict | None = None) -> dict:
    """Distillation from a teacher's top logits (dg_row_topk's indices and values, with teacher_lse its lse
    for the bucket of the other entries) -> dict loss, lse (fp32 [R]), tail_logp (with teacher_lse) and,
    with grad=True or a `grad` in `out`, the logits' gradient of sum_r weight_r loss_r."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    K, ldk = _entries(indices, teacher, R, dev)
    shapes = {"loss": (R, f32), "lse": (R, f32)}
    if teacher_lse is not None:
        shapes["tail_logp"] = (R, f32)
    o = _fill(out, shapes, dev, stream)
    if grad and "grad" not in o:
        o["grad"] = _new_grad(logits, stream)
    g, ldg = _grad_like(o["grad"], logits) if "grad" in o else (None, 0)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream)
    _check(lib.dg_distill_loss(x, code, R, V, ld, indices.data_ptr(), teacher.data_ptr(), K, ldk,
                               _vec(teacher_lse, R, f32, dev, "teacher_lse"), temperature,
                               _vec(weight, R, f32, dev, "weight"), _vec(o["loss"], R, f32, dev, "loss"),
                               _vec(o["lse"], R, f32, dev, "lse"), _vec(o.get("tail_logp"), R, f32, dev, "tail_logp"),
                               g, ldg, ws_ptr, ws_bytes, _stream(stream)), "dg_distill_loss")
    return o


def dg_distill_loss_backward(logits: torch.Tensor, indices: torch.Tensor, teacher: torch.Tensor,
                             lse: torch.Tensor, dloss: torch.Tensor | None = None,
                             teacher_lse: torch.Tensor | None = None, tail_logp: torch.Tensor | None = None,
                             temperature: float = 1.0, ws: torch.Tensor | None = None, stream=None,
                             out: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient of sum_r dloss_r loss_r from a forward call's lse (and tail_logp).  `out` may be
    the logits themselves."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    K, ldk = _entries(indices, teacher, R, dev)
    if out is None:
        out = _new_grad(logits, stream)
    g, ldg = _grad_like(out, logits)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream, always=True)
    _check(lib.dg_distill_loss_backward(x, code, R, V, ld, indices.data_ptr(), teacher.data_ptr(), K, ldk,
                                        _vec(teacher_lse, R, f32, dev, "teacher_lse"), temperature,
                                        _vec(lse, R, f32, dev, "lse"), _vec(tail_logp, R, f32, dev, "tail_logp"),
                                        _vec(dloss, R, f32, dev, "dloss"), g, ldg, ws_ptr, ws_bytes,
                                        _stream(stream)),
           "dg_distill_loss_backward")
    return out


def dg_policy_loss(logits: torch.Tensor, token: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                   ref_logp: torch.Tensor | None = None, clip_low: float = 0.2, clip_high: float = 0.2,
                   kl_coef: float = 0.0, temperature: float = 1.0, weight: torch.Tensor | None = None,
                   grad: bool = False, ws: torch.Tensor | None = None, stream=None, out: dict | None = None) -> dict:
    """Clipped policy loss with a KL term against a reference -> dict loss, logp, lse, kl, dlogp (fp32 [R]),
    clipped (uint8 [R]) and, with grad=True or a `grad` in `out`, the logits' gradient of
    sum_r weight_r loss_r."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    o = _fill(out, {"loss": (R, f32), "logp": (R, f32), "lse": (R, f32), "kl": (R, f32), "dlogp": (R, f32),
                    "clipped": (R, torch.uint8)}, dev, stream)
    if grad and "grad" not in o:
        o["grad"] = _new_grad(logits, stream)
    g, ldg = _grad_like(o["grad"], logits) if "grad" in o else (None, 0)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream)
    _check(lib.dg_policy_loss(x, code, R, V, ld, _vec(token, R, torch.int32, dev, "token"),
                              _vec(old_logp, R, f32, dev, "old_logp"), _vec(ref_logp, R, f32, dev, "ref_logp"),
                              _vec(advantage, R, f32, dev, "advantage"), temperature, clip_low, clip_high, kl_coef,
                              _vec(weight, R, f32, dev, "weight"), _vec(o["loss"], R, f32, dev, "loss"),
                              _vec(o["logp"], R, f32, dev, "logp"), _vec(o["lse"], R, f32, dev, "lse"),
                              _vec(o["kl"], R, f32, dev, "kl"), _vec(o["clipped"], R, torch.uint8, dev, "clipped"),
                              _vec(o["dlogp"], R, f32, dev, "dlogp"), g, ldg, ws_ptr, ws_bytes, _stream(stream)),
           "dg_policy_loss")
    return o


def dg_preference_loss(logits: torch.Tensor, token: torch.Tensor, ref_logp: torch.Tensor | None,
                       seq_start: torch.Tensor, beta: float = 0.1, label_smoothing: float = 0.0,
                       temperature: float = 1.0, weight: torch.Tensor | None = None,
                       pair_weight: torch.Tensor | None = None, grad: bool = False,
                       ws: torch.Tensor | None = None, stream=None, out: dict | None = None) -> dict:
    """Preference loss on the log ratios of P pairs of packed sequences (rows [seq_start[j], seq_start[j+1]);
    pair i prefers sequence 2i over 2i + 1) -> dict loss [P], log_ratio [2P], logp, lse, dlogp [R] and, with
    grad=True or a `grad` in `out`, the logits' gradient of sum_i pair_weight_i loss_i."""
    x, code, R, V, ld = _logits(logits)
    dev, f32 = logits.device, torch.float32
    n = seq_start.numel()
    if n % 2 != 1:
        raise ValueError("seq_start must hold 2P + 1 offsets")
    P = n // 2
    o = _fill(out, {"loss": (P, f32), "log_ratio": (2 * P, f32), "logp": (R, f32), "lse": (R, f32),
                    "dlogp": (R, f32)}, dev, stream)
    if grad and "grad" not in o:
        o["grad"] = _new_grad(logits, stream)
    g, ldg = _grad_like(o["grad"], logits) if "grad" in o else (None, 0)
    ws, ws_ptr, ws_bytes = _loss_ws(ws, R, V, code, dev, stream)
    _check(lib.dg_preference_loss(x, code, R, V, ld, _vec(token, R, torch.int32, dev, "token"),
                                  _vec(ref_logp, R, f32, dev, "ref_logp"),
                                  _vec(seq_start, n, torch.int32, dev, "seq_start"), P, beta, label_smoothing,
                                  temperature, _vec(weight, R, f32, dev, "weight"),
                                  _vec(pair_weight, P, f32, dev, "pair_weight"), _vec(o["loss"], P, f32, dev, "loss"),
                                  _vec(o["log_ratio"], 2 * P, f32, dev, "log_ratio"),
                                  _vec(o["logp"], R, f32, dev, "logp"), _vec(o["lse"], R, f32, dev, "lse"),
                                  _vec(o["dlogp"], R, f32, dev, "dlogp"), g, ldg, ws_ptr, ws_bytes, _stream(stream)),
           "dg_preference_loss")
    return o


# --------------------------------------------------------------------------- the hidden stream
#
# Common to the calls below: matrices [R, d] in fp32 or bf16 with unit column stride and any row stride;
# E4M3 codes are uint8 and go with a contiguous fp32 vector of scales.  All tensors are on the current
# device; `out` holds preallocated outputs, and the ones it lacks are allocated.

def _matrix(t: torch.Tensor, R: int, d: int, name: str, device, types=_DTYPE) -> tuple:
    """(pointer, dtype code, row stride) of an [R, d] matrix on `device`."""
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} has type {t.dtype}: need one of {', '.join(map(str, types))}")
    strides = t.stride()        # (one call: each costs a small call a hundredth of its time)
    if t.shape != (R, d) or (strides[1] != 1 and d > 1) or t.device != device:
        raise ValueError(f"{name} must be [{R}, {d}] with unit column stride on {device}, "
                         f"got {list(t.shape)} with strides {list(strides)} on {t.device}")
    return t.data_ptr(), code, strides[0] if R > 1 else (d + 15) // 16 * 16


def _here(t: torch.Tensor, name: str):
    """The device of a matrix whose device the kernels will run on."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, and the kernels would run on the current device, "
                         f"cuda:{torch._C._cuda_getDevice()}: use torch.cuda.device({name}.device)")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return t.device


def _new_rows(R: int, d: int, dtype, device, stream) -> torch.Tensor:
    """An uninitialised [R, d] matrix whose rows start on 16-byte boundaries."""
    per = 16 // dtype.itemsize
    with _on(stream):
        return _new((R, (d + per - 1) // per * per), dtype, device)[:, :d]


def _scratch(n: int, device, stream) -> torch.Tensor:
    with _on(stream):
        return _new((max(16, n) + 15) // 16 * 16, torch.uint8, device)


def dg_token_embed_backward_workspace_size(R: int, vocab_len: int, d: int) -> int:
    return int(lib.dg_token_embed_backward_workspace_size(R, vocab_len, d))


def embed_workspace(R: int, vocab_len: int, d: int, device) -> torch.Tensor:
    """A workspace tensor large enough for dg_token_embed_backward, of these sizes or smaller ones."""
    return _scratch(dg_token_embed_backward_workspace_size(R, vocab_len, d), device, None)


def dg_token_embed(table: torch.Tensor, token: torch.Tensor, gamma: float = 1.0, scale: torch.Tensor | None = None,
                   vocab_start: int = 0, vocab_end: int | None = None, V: int | None = None,
                   out: torch.Tensor | None = None, dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """gamma times the table's rows at `token` [R] (int32; negative: padding, a row of zeros) -> [R, d].
    table: fp32 or bf16 [rows_pad, d], or E4M3 codes with the row scales `scale`; row j is vocabulary entry
    vocab_start + j (the whole table by default), and tokens outside [vocab_start, vocab_end) give zeros.
    V: the vocabulary's size, which a slice's caller gives too (default: vocab_end); a token at or past it is an
    error that dg_get_device_status reports.
    dtype: of a new output (default: the table's, bf16 for codes)."""
    device = _here(table, "table")
    rows, d = table.shape
    vocab_end = vocab_start + rows if vocab_end is None else vocab_end
    V = vocab_end if V is None else V
    R = token.shape[0] if token.dim() == 1 else -1
    tok = _vec(token, R, torch.int32, device, "token")
    tp, tc, ldw = _matrix(table, rows, d, "table", device, _DTYPE_CODES)
    if out is None:
        dtype = dtype if dtype is not None else torch.bfloat16 if tc == DG_E4M3 else table.dtype
        out = _new_rows(R, d, dtype, device, stream)
    op, oc, ldo = _matrix(out, R, d, "out", device)
    _check(lib.dg_token_embed(tp, tc, _vec(scale, rows, torch.float32, device, "scale"), V, vocab_start, vocab_end,
                              rows, ldw, d, tok, R, gamma, op, oc, ldo, _stream(stream)), "dg_token_embed")
    return out


def dg_token_embed_backward(grad: torch.Tensor, token: torch.Tensor, V: int, gamma: float = 1.0,
                            vocab_start: int = 0, vocab_end: int | None = None, accumulate: bool = False,
                            ws: torch.Tensor | None = None, out: torch.Tensor | None = None,
                            dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """The gradient [rows, d] of dg_token_embed's table (fp32 or bf16) from that of its rows [R, d]: every row
    of [vocab_start, vocab_end) is written, or with accumulate=True the sums are added to `out`.
    dtype: of a new gradient (default: grad's)."""
    device = _here(grad, "grad")
    R, d = grad.shape
    vocab_end = V if vocab_end is None else vocab_end
    gp, gc, ldg = _matrix(grad, R, d, "grad", device)
    tok = _vec(token, R, torch.int32, device, "token")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs `out`, the gradient to add to")
        out = _new_rows(max(0, vocab_end - vocab_start), d, grad.dtype if dtype is None else dtype, device, stream)
    rows = out.shape[0]
    tp, tc, ldt = _matrix(out, rows, d, "out", device)
    if ws is None and R > 0:
        ws = _scratch(dg_token_embed_backward_workspace_size(R, max(0, vocab_end - vocab_start), d), device, stream)
    wp, wn = (None, 0) if ws is None else _memory(ws, device)
    _check(lib.dg_token_embed_backward(gp, gc, R, d, ldg, tok, V, vocab_start, vocab_end, gamma, tp, tc, rows, ldt,
                                       bool(accumulate), wp, wn, _stream(stream)), "dg_token_embed_backward")
    return out


def dg_rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                eps: float = 1e-6, weight_offset: float = 0.0, dtype: torch.dtype | None = None,
                out: dict | None = None, stream=None) -> dict:
    """h = x + residual, y = h / rms(h) * (weight_offset + weight) -> dict out (y), rstd [R], with a residual
    hidden (h), with dtype=torch.uint8 scale [R] beside the E4M3 codes in out.
    dtype: of a new out (default: x's); hidden has the residual's type, and out={"hidden": None} leaves it out.
    `out` may hold x or residual themselves as hidden or as out: they are replaced."""
    device = _here(x, "x")
    R, d = x.shape
    xp, xc, ldx = _matrix(x, R, d, "x", device)
    o = {} if out is None else out
    y = o.get("out")
    if y is None:
        y = o["out"] = _new_rows(R, d, x.dtype if dtype is None else dtype, device, stream)
    yp, yc, ldy = _matrix(y, R, d, "out", device, _DTYPE_CODES)
    rp = hp = sp = wp = None
    rc = ldr = hc = ldh = wc = 0
    if residual is not None:
        rp, rc, ldr = _matrix(residual, R, d, "residual", device)
        if "hidden" not in o:
            o["hidden"] = _new_rows(R, d, residual.dtype, device, stream)
    if o.get("hidden") is not None:
        hp, hc, ldh = _matrix(o["hidden"], R, d, "hidden", device)
    if "rstd" not in o:
        with _on(stream):
            o["rstd"] = _new(R, torch.float32, device)
    if yc == DG_E4M3:
        if "scale" not in o:
            with _on(stream):
                o["scale"] = _new(R, torch.float32, device)
        sp = _vec(o["scale"], R, torch.float32, device, "scale")
    if weight is not None:
        wc = _DTYPE.get(weight.dtype, -1)
        wp = _vec(weight, d, weight.dtype, device, "weight")
    _check(lib.dg_rms_norm(xp, xc, R, d, ldx, rp, rc, ldr, wp, wc, weight_offset, eps, hp, hc, ldh, yp, yc, ldy, sp,
                           _vec(o["rstd"], R, torch.float32, device, "rstd"), _stream(stream)), "dg_rms_norm")
    return o


def dg_rms_norm_backward_workspace_size(R: int, d: int) -> int:
    return int(lib.dg_rms_norm_backward_workspace_size(R, d))


def norm_workspace(R: int, d: int, device) -> torch.Tensor:
    """A workspace tensor large enough for dg_rms_norm_backward, of these sizes or smaller ones."""
    return _scratch(dg_rms_norm_backward_workspace_size(R, d), device, None)


def dg_rms_norm_backward(grad: torch.Tensor, hidden: torch.Tensor, rstd: torch.Tensor,
                         weight: torch.Tensor | None = None, weight_offset: float = 0.0,
                         grad_hidden: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                         out: dict | None = None, stream=None) -> dict:
    """Gradients of dg_rms_norm from that of y (and of h: grad_hidden), the hidden and rstd it wrote (without a
    residual: x) -> dict grad (of x and of residual alike, in hidden's type) and, with a weight, grad_weight (in
    its type; out={"grad_weight": None} leaves it out).  grad may replace any of the three matrices."""
    device = _here(grad, "grad")
    R, d = grad.shape
    gp, gc, ldg = _matrix(grad, R, d, "grad", device)
    hp, hc, ldh = _matrix(hidden, R, d, "hidden", device)
    o = {} if out is None else out
    if "grad" not in o:
        o["grad"] = _new_rows(R, d, hidden.dtype, device, stream)
    if o["grad"].dtype is not hidden.dtype:
        raise TypeError(f"out['grad'] must have hidden's type, {hidden.dtype}")
    xp, _, ldx = _matrix(o["grad"], R, d, "out['grad']", device)
    up = wp = dp = wsp = None
    uc = ldu = wc = wn = 0
    if grad_hidden is not None:
        up, uc, ldu = _matrix(grad_hidden, R, d, "grad_hidden", device)
    if weight is not None:
        wc = _DTYPE.get(weight.dtype, -1)
        wp = _vec(weight, d, weight.dtype, device, "weight")
        if "grad_weight" not in o:
            with _on(stream):
                o["grad_weight"] = _new(d, weight.dtype, device)
    if o.get("grad_weight") is not None:
        if weight is None:
            raise ValueError("grad_weight needs a weight")
        dp = _vec(o["grad_weight"], d, weight.dtype, device, "grad_weight")
        if ws is None and R > 0:
            ws = _scratch(dg_rms_norm_backward_workspace_size(R, d), device, stream)
        wsp, wn = (None, 0) if ws is None else _memory(ws, device)
    _check(lib.dg_rms_norm_backward(gp, gc, R, d, ldg, hp, hc, ldh, _vec(rstd, R, torch.float32, device, "rstd"), wp,
                                    wc, weight_offset, up, uc, ldu, xp, ldx, dp, wsp, wn, _stream(stream)),
           "dg_rms_norm_backward")
    return o


def dg_head_e4m3(X: torch.Tensor, x_scale: torch.Tensor, Q: torch.Tensor, scale: torch.Tensor,
                 out: torch.Tensor | None = None, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """Logits [R, V] = x_scale scale (X Q^T) of E4M3 codes X [R, d] (dg_rms_norm's) and Q [V, d]
    (dg_quantize_e4m3's), in fp32 or bf16; rows of all three start on 16-byte boundaries."""
    device = _here(X, "X")
    R, d = X.shape
    V = Q.shape[0]
    codes = {torch.uint8: DG_E4M3}
    xp, _, ldx = _matrix(X, R, d, "X", device, codes)
    qp, _, ldq = _matrix(Q, V, d, "Q", device, codes)
    if out is None:
        out = _new_rows(R, V, dtype, device, stream)
    lp, lc, ldl = _matrix(out, R, V, "out", device)
    _check(lib.dg_head_e4m3(xp, ldx, _vec(x_scale, R, torch.float32, device, "x_scale"), R, d, qp,
                            _vec(scale, V, torch.float32, device, "scale"), V, ldq, lp, lc, ldl, _stream(stream)),
           "dg_head_e4m3")
    return out
