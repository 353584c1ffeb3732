"""The serving head in 8 bits: from hidden states to verified tokens.

  ce_quantize_fp8(x, block_rows=1 | 128)            -> (q, scale)
  ce_rms_norm_fp8(x, weight, residual=...)          -> (q, scale, residual_out)
  ce_gemm_fp8(A, a_scale, B, b_scale, ...)          -> D
  ce_verify_drafts(logits, draft_token, ...)        -> (accepted, tokens, logp)
and ``fp8_head_logits``, the norm and the product in one call. The formulas and
layouts are in include/ce.h. These calls are not differentiable: what they
return carries no graph.

8-bit matrices are ``torch.float8_e4m3fn`` tensors [rows, cols] whose rows start
at multiples of 16 bytes (new ones have such a row stride where cols is not
a multiple of 16), with contiguous fp32 scales: [rows, ceil(cols / 128)] for
activations, [ceil(rows / 128), ceil(cols / 128)] for weights. ``stream``
defaults to the current stream of the first tensor's device.
"""
from __future__ import annotations

import ctypes

import torch

from . import CE_DT, _check, _lib
from .logprob import _Call, _byref, _ptr, _workspace

_F32, _I32, _I64, _E4M3 = torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


class ce_norm_params(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_x", ctypes.c_int64),
                ("ld_residual", ctypes.c_int64), ("ld_residual_out", ctypes.c_int64), ("ld_q", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class ce_verify_params(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("n_drafts", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("seq_stride", ctypes.c_int64), ("ld", ctypes.c_int64), ("draft_seq_stride", ctypes.c_int64),
                ("ld_draft", ctypes.c_int64), ("dtype", ctypes.c_int32), ("token_is_int32", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("reserved", ctypes.c_int32)]


assert ctypes.sizeof(ce_norm_params) == 64 and ctypes.sizeof(ce_verify_params) == 72


def _sign():
    vp, i32, i64, sz, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
    for name, args in {
        "ce_rms_norm_fp8": [ctypes.POINTER(ce_norm_params)] + [vp] * 7,
        "ce_quantize_fp8": [i64, i64, vp, i64, i32, i32, vp, i64, vp, vp],
        "ce_gemm_fp8": [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i32, vp, i64, vp],
        "ce_verify_workspace_size": [ctypes.POINTER(ce_verify_params), ctypes.POINTER(sz)],
        "ce_verify_drafts": [ctypes.POINTER(ce_verify_params)] + [vp] * 10 + [sz, vp],
    }.items():
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = st, args


_sign()


# ---------------------------------------------------------------------- arguments
# (A call's host time is what the smallest calls take: sizes and strides are asked
# for once, and tensors made here are not checked.)
def _matrix(name, t):
    """(rows, columns, row stride) of a 2-D tensor with unit column stride."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or (strides[1] != 1 and shape[1] != 1):
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return shape[0], shape[1], strides[0] if shape[0] > 1 else shape[1]


def _like(name, t, n, cols, dtype):
    """The row stride of a matrix of the given size and type."""
    rows, columns, ld = _matrix(name, t)
    if rows != n or columns != cols:
        raise ValueError(f"{name} must have the shape ({n}, {cols})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    return ld


def _matrix8(name, t):
    """The same of an 8-bit matrix, whose rows start at multiples of 16 bytes."""
    if t.dtype is not _E4M3:
        raise TypeError(f"{name} must be {_E4M3}")
    rows, cols, ld = _matrix(name, t)
    if rows < 2:
        ld = (cols + 15) // 16 * 16
    if ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{name}'s rows must start at multiples of 16 bytes")
    return rows, cols, ld


def _out8(call, q, n, cols):
    """(an 8-bit matrix to write, its row stride): the given one, or a new one."""
    if q is None:
        ld = (cols + 15) // 16 * 16
        return call.empty(n, cols, dtype=_E4M3, strides=None if ld == cols else (ld, 1)), ld
    rows, columns, ld = _matrix8("q", q)
    if rows != n or columns != cols:
        raise ValueError(f"q must have the shape ({n}, {cols})")
    return q, ld


def _scales(name, t, rows, cols):
    if t.dtype is not _F32 or t.shape != (rows, cols) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 tensor [{rows}, {cols}]")
    return t


def _dtype(name, t):
    dt = CE_DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported {name} dtype {t.dtype}")
    return dt


# ---------------------------------------------------------------------- norm and quantising
def ce_rms_norm_fp8(x, weight, *, residual=None, eps=1e-6, with_residual_out=True, residual_out=None, q=None,
                    scale=None, stream=None):
    """(q [n, H], scale [n, ceil(H / 128)], residual_out or None): the
    root-mean-square norm of x + residual times weight, in 8 bits. The sum goes
    to ``residual_out`` (a new tensor of x's type unless one is given, which may
    be ``residual`` or ``x`` itself; not formed with ``with_residual_out=False``).
    x, residual: [n, H] bf16, fp16 or fp32; weight: [H] of x's type or fp32.
    One kernel, no workspace."""
    n, cols, ld = _matrix("x", x)
    dtype = x.dtype
    dt = _dtype("x", x)
    call = _Call(x, (weight, residual, residual_out, q, scale), stream)
    wt = weight.dtype
    if weight.shape != (cols,) or not weight.is_contiguous() or (wt is not dtype and wt is not _F32):
        raise ValueError("weight must be a contiguous tensor of H entries, of x's dtype or fp32")
    ldr = ldo = 0
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out given without residual")
    else:
        ldr = _like("residual", residual, n, cols, dtype)
        if residual_out is not None:
            if not with_residual_out:
                raise ValueError("residual_out given with with_residual_out=False")
            ldo = _like("residual_out", residual_out, n, cols, dtype)
        elif with_residual_out:
            residual_out = call.empty(n, cols, dtype=dtype)
            ldo = cols
    q, ldq = _out8(call, q, n, cols)
    blocks = (cols + 127) // 128
    scale = call.empty(n, blocks) if scale is None else _scales("scale", scale, n, blocks)
    p = ce_norm_params(n, cols, ld, ldr, ldo, ldq, dt, CE_DT[wt], eps, 0)
    call.run("ce_rms_norm_fp8", _byref(p), x.data_ptr(), _ptr(residual), weight.data_ptr(), _ptr(residual_out),
             q.data_ptr(), scale.data_ptr())
    return q, scale, residual_out


def ce_quantize_fp8(x, *, block_rows=1, q=None, scale=None, stream=None):
    """(q, scale) of a matrix in 8 bits: ``block_rows`` 1 for activations (a
    scale for every row and 128 columns), 128 for weights (for every 128 x 128)."""
    n, cols, ld = _matrix("x", x)
    dt = _dtype("x", x)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    call = _Call(x, (q, scale), stream)
    q, ldq = _out8(call, q, n, cols)
    up, blocks = -(-n // block_rows), (cols + 127) // 128
    scale = call.empty(up, blocks) if scale is None else _scales("scale", scale, up, blocks)
    call.run("ce_quantize_fp8", n, cols, x.data_ptr(), ld, dt, block_rows, q.data_ptr(), ldq, scale.data_ptr())
    return q, scale


# ---------------------------------------------------------------------- product
def ce_gemm_fp8(A, a_scale, B, b_scale, *, bias=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """A [M, K] times B^T, B [N, K], both in 8 bits (A in blocks of 1 x 128, B of
    128 x 128), plus bias [N] fp32: [M, N] of ``out_dtype`` or into ``out``."""
    (m, k, lda), (n, kb, ldb) = _matrix8("A", A), _matrix8("B", B)
    if kb != k:
        raise ValueError("inner dimensions differ")
    call = _Call(A, (a_scale, B, b_scale, bias, out), stream)
    blocks = (k + 127) // 128
    _scales("a_scale", a_scale, m, blocks)
    _scales("b_scale", b_scale, (n + 127) // 128, blocks)
    if bias is not None and (bias.dtype is not _F32 or bias.shape != (n,) or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous fp32 tensor of N entries")
    if out is None:
        dt = CE_DT.get(out_dtype)
        if dt is None:
            raise TypeError(f"unsupported out_dtype {out_dtype}")
        out, ldd = call.empty(m, n, dtype=out_dtype), n
    else:
        dt = _dtype("out", out)
        ldd = _like("out", out, m, n, out.dtype)
    call.run("ce_gemm_fp8", m, n, k, A.data_ptr(), lda, a_scale.data_ptr(), B.data_ptr(), ldb, b_scale.data_ptr(),
             _ptr(bias), dt, out.data_ptr(), ldd)
    return out


def fp8_head_logits(x, norm_weight, weight, weight_scale, *, residual=None, eps=1e-6, bias=None,
                    out_dtype=torch.bfloat16, stream=None):
    """Logits [..., V] of hidden states x [..., H]: the norm of x + residual in
    8 bits, times an 8-bit lm head (ce_quantize_fp8(W, block_rows=128)). For
    ce_verify_drafts, or for ce_token_logprob where rollouts are scored under the
    head that sampled them."""
    h = x.reshape(-1, x.shape[-1])
    r = None if residual is None else residual.reshape(-1, residual.shape[-1])
    if stream is not None:  # where reshape had to copy, nothing else holds the copies
        call = _Call(x, (residual,), stream)
        for given, rows in ((x, h), (residual, r)):
            if rows is not None and rows.data_ptr() != given.data_ptr():
                call.lend(rows)
    q, scale, _ = ce_rms_norm_fp8(h, norm_weight, residual=r, eps=eps, with_residual_out=False, stream=stream)
    out = ce_gemm_fp8(q, scale, weight, weight_scale, bias=bias, out_dtype=out_dtype, stream=stream)
    return out.view(*x.shape[:-1], weight.shape[0])


# ---------------------------------------------------------------------- verification
def _verify_ws_bytes(p) -> int:
    out = ctypes.c_size_t()
    _check(_lib.ce_verify_workspace_size(_byref(p), _byref(out)), "ce_verify_workspace_size")
    return out.value


def _given(name, t, call, shape, dtype):
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != call.index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on the logits' device")
    return t


def ce_verify_drafts(logits, draft_token, accept_uniform, sample_uniform, *, draft_logits=None, temperature=1.0,
                     accepted=None, tokens=None, logp=None, ws=None, stream=None):
    """(accepted [B] int32, tokens [B, K + 1], logp [B, K + 1]): how many of
    every sequence's K drafted tokens stay, the tokens it goes on with (those
    drafts, one drawn token, then -1) and their log-probabilities. logits
    [B, K + 1, V] (bf16, fp16 or fp32), draft_token [B, K] int64 or int32 (-1
    ends a shorter draft), accept_uniform [B, K] and sample_uniform [B] fp32 in
    [0, 1), draft_logits [B, K, V] of the logits' type, or None where the drafts
    were not sampled. ``temperature``: a number, or an fp32 tensor [B]; 0 is
    greedy. K = 0 draws one token a sequence."""
    shape = logits.shape
    if len(shape) != 3 or shape[1] < 1:
        raise ValueError("logits must be [B, K + 1, V]")
    B, rows, V = shape
    K = rows - 1
    dtype = logits.dtype
    dt = _dtype("logits", logits)
    tok = draft_token.dtype
    if tok is not _I64 and tok is not _I32:
        raise TypeError("draft_token must be int64 or int32")
    if draft_token.shape != (B, K) or not draft_token.is_contiguous():
        raise ValueError("draft_token must be a contiguous tensor [B, K]")
    if accept_uniform.dtype is not _F32 or accept_uniform.shape != (B, K) or not accept_uniform.is_contiguous():
        raise ValueError("accept_uniform must be a contiguous fp32 tensor [B, K]")
    if sample_uniform.dtype is not _F32 or sample_uniform.shape != (B,) or not sample_uniform.is_contiguous():
        raise ValueError("sample_uniform must be a contiguous fp32 tensor [B]")
    temps = None
    if isinstance(temperature, torch.Tensor):
        temps, temperature = temperature, 1.0
        if temps.dtype is not _F32 or temps.shape != (B,) or not temps.is_contiguous():
            raise ValueError("temperature must be a number or a contiguous fp32 tensor [B]")
    call = _Call(logits, (draft_token, accept_uniform, sample_uniform, draft_logits, temps), stream)
    xs, xr, unit = logits.stride()
    ys, yr = 0, V
    if draft_logits is not None:
        if draft_logits.shape != (B, K, V) or draft_logits.dtype is not dtype:
            raise ValueError("draft_logits must be [B, K, V] of the logits' dtype")
        ys, yr, unit_y = draft_logits.stride()
        if unit_y != 1 and V != 1:
            raise ValueError("draft_logits must have unit column stride")
        ys, yr = ys if B > 1 else 0, yr if K > 1 else V
    if unit != 1 and V != 1:
        raise ValueError("logits must have unit column stride")
    p = ce_verify_params(B, K, V, xs if B > 1 else 0, xr if K else V, ys, yr, dt, 1 if tok is _I32 else 0, temperature, 0)
    accepted = call.empty(B, dtype=_I32) if accepted is None else _given("accepted", accepted, call, (B,), _I32)
    tokens = call.empty(B, rows, dtype=tok) if tokens is None else _given("tokens", tokens, call, (B, rows), tok)
    logp = call.empty(B, rows) if logp is None else _given("logp", logp, call, (B, rows), _F32)
    ws, nbytes = _workspace(call, ws, _verify_ws_bytes(p))
    call.run("ce_verify_drafts", _byref(p), logits.data_ptr(), _ptr(draft_logits), draft_token.data_ptr(),
             accept_uniform.data_ptr(), sample_uniform.data_ptr(), _ptr(temps), accepted.data_ptr(),
             tokens.data_ptr(), logp.data_ptr(), _ptr(ws), nbytes)
    return accepted, tokens, logp
