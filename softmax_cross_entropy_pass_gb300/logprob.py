"""Token log-probabilities and the post-training losses made of them.

  ce_token_logprob(logits, target, ...)            -> (logp, entropy, stats)
  ce_token_logprob_backward(logits, target, stats, grad_logp, ...) -> grad
  ce_policy_fwd_bwd(logits, target, advantage, ...)    -> (loss, grad)
  ce_preference_fwd_bwd(logits, target, seq_offsets, ...) -> (loss, seq_logp, grad)
  flce_token_logprob(hidden, weight, target, ...)  -> (logp, entropy, stats)
  flce_token_logprob_backward(hidden, weight, target, stats, grad_logp, ...)
                                                   -> (grad_hidden, grad_weight, grad_bias)
and their torch.autograd entries ``token_logprob``, ``policy_loss``,
``preference_loss`` and ``linear_token_logprob``. The formulas, the layouts and what each call does with
ignored rows are in include/ce.h.

``logits`` is a 2-D CUDA tensor with unit column stride (bf16, fp16 or fp32).
Per-row and per-sequence inputs are contiguous fp32 tensors on its device.
``grad`` receives the gradient: a tensor of the logits' shape and dtype with
unit column stride, or None to write it over the logits. ``stream`` defaults
to the current stream of the logits' device.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import CE_DT, CE_RED, CEError, _check, _lib, ce_params, ce_scale_grad

_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream of a device as an integer
_current_device = torch._C._cuda_getDevice
_byref, _F32, _I64, _I32 = ctypes.byref, torch.float32, torch.int64, torch.int32

CE_FLAG_BAD_OFFSETS = 8
PREFERENCE_KINDS = {"sigmoid": 0, "hinge": 1, "squared": 2}


class ce_policy_params(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl_coef", ctypes.c_float), ("entropy_coef", ctypes.c_float), ("reserved", ctypes.c_int32)]


class ce_preference_params(ctypes.Structure):
    _fields_ = [("n_pairs", ctypes.c_int64), ("kind", ctypes.c_int32), ("offsets_are_int32", ctypes.c_int32),
                ("length_normalize", ctypes.c_int32), ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


assert ctypes.sizeof(ce_policy_params) == 24 and ctypes.sizeof(ce_preference_params) == 32


def _sign():
    P, vp, f, i64 = ctypes.POINTER(ce_params), ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
    sz, st = ctypes.c_size_t, ctypes.c_int
    for name, args in {
        "ce_token_logprob": [P, f, vp, vp, vp, vp, vp, vp],
        "ce_token_logprob_backward": [P, f, vp, vp, vp, vp, vp, vp, i64, vp],
        "ce_policy_fwd_bwd": [P, ctypes.POINTER(ce_policy_params)] + [vp] * 10 + [i64, vp, sz, vp],
        "ce_preference_workspace_size": [P, i64, ctypes.POINTER(sz)],
        "ce_preference_fwd_bwd": [P, ctypes.POINTER(ce_preference_params)] + [vp] * 8 + [i64, vp, sz, vp],
        "flce_token_logprob_workspace_size": [P, i64, i64, ctypes.POINTER(sz)],
        "flce_token_logprob": [P, i64, f] + [vp] * 8 + [sz, vp],
        "flce_token_logprob_backward": [P, i64, f] + [vp] * 9 + [ctypes.c_int32, vp, i64, vp, sz, vp],
    }.items():
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = st, args


_sign()


# ---------------------------------------------------------------------- arguments
def _ptr(t):
    return None if t is None else t.data_ptr()


def _check_target(target, n):
    dtype = target.dtype
    if dtype is not _I64 and dtype is not _I32:
        raise TypeError("target must be int64 or int32")
    if target.dim() != 1 or target.numel() != n or not target.is_contiguous():
        raise ValueError("target must be a contiguous 1-D tensor with one entry per row")
    return 1 if dtype is _I32 else 0


def _params(logits, target, ignore_index, reduction="mean") -> ce_params:
    if logits.dim() != 2:
        raise ValueError("logits must be a 2-D tensor with unit column stride")
    n, v = logits.shape
    ld, step = logits.stride()
    if step != 1 and v != 1:
        raise ValueError("logits must be a 2-D tensor with unit column stride")
    dtype = CE_DT.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}")
    if reduction not in CE_RED:
        raise ValueError(f"unknown reduction {reduction!r}")
    # n_rows, vocab, ld, ignore_index, class_weight, label_smoothing, dtype, reduction, target_is_int32
    return ce_params(n, v, ld if n > 1 else v, ignore_index, None, 0.0, dtype, CE_RED[reduction], _check_target(target, n))


def _vec(name, t, n, call):
    """A contiguous fp32 vector of n entries on the call's device (or None)."""
    if t is not None and (t.dtype is not _F32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous()
                          or t.get_device() != call.index):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of {n} entries on the logits' device")
    return t


def _rows4(name, t, n, call):
    if t is not None and (t.dtype is not _F32 or t.dim() != 2 or t.shape[1] != 4 or t.shape[0] != n
                          or not t.is_contiguous() or t.get_device() != call.index):
        raise ValueError(f"{name} must be a contiguous fp32 [n_rows, 4] tensor on the logits' device")
    return t


def _grad_buffer(logits, grad, p):
    """(the gradient's buffer, its row stride)."""
    if grad is None:
        return logits, p.ld
    if grad.shape != logits.shape or grad.dtype is not logits.dtype or grad.get_device() != logits.get_device() \
            or (grad.stride(1) != 1 and p.vocab != 1):
        raise ValueError("grad must have the logits' shape, dtype and device, and unit column stride")
    return grad, grad.stride(0) if p.n_rows > 1 else p.vocab


class _Call:
    """The device and the stream of one call. Memory that the call allocates
    comes from the current stream's pool: where the kernels run on another
    stream, that pool is told so before it may hand the memory out again."""
    __slots__ = ("device", "index", "stream", "other", "handle")

    def __init__(self, tensor, others, stream):
        index = self.index = tensor.get_device()
        if index < 0:
            raise ValueError("all tensors must live on the GPU")
        for t in others:
            if t is not None and t.get_device() != index:
                raise ValueError("all tensors must live on the logits' device")
        self.device, self.other, self.handle = tensor.device, None, _raw_stream(index)
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=self.device)
            if stream.device != self.device:
                raise ValueError("stream must be one of the logits' device")
            if stream.cuda_stream != self.handle:
                self.stream, self.other, self.handle = stream, torch.cuda.current_stream(self.device), stream.cuda_stream

    def empty(self, *shape, dtype=_F32, strides=None):
        t = torch.empty(shape, dtype=dtype, device=self.device) if strides is None else \
            torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        if self.other is not None:
            self.stream.wait_stream(self.other)  # the memory's last user may still be running there
            t.record_stream(self.stream)
        return t

    def lend(self, t):
        """A tensor that the current stream has made for this call alone: the kernels' stream waits for it, and the
        memory is not handed out again before that stream has read it."""
        if self.other is not None:
            self.stream.wait_stream(self.other)
            t.record_stream(self.stream)
        return t

    def run(self, name, *args):
        fn = getattr(_lib, name)
        if _current_device() == self.index:
            status = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, self.handle)
        if status:
            _check(status, name)


def _outputs(call, n, logp, entropy, stats, with_entropy):
    """The three outputs of a forward: those given, or new ones."""
    if not with_entropy and entropy is not None:
        raise ValueError("entropy given with with_entropy=False")
    logp = call.empty(n) if logp is None else _vec("logp", logp, n, call)
    if with_entropy:
        entropy = call.empty(n) if entropy is None else _vec("entropy", entropy, n, call)
    return logp, entropy, call.empty(n, 4) if stats is None else _rows4("stats", stats, n, call)


def _workspace(call, ws, nbytes):
    if ws is None:
        return call.empty(nbytes, dtype=torch.uint8), nbytes
    if ws.get_device() != call.index or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor on the logits' device")
    return ws, ws.numel() * ws.element_size()


# The sizes that ce_workspace_size and ce_preference_workspace_size stay within
# (include/ce.h), without the calls.
def _policy_ws_bytes(n) -> int:
    return 20 * n + 512


def _preference_ws_bytes(n, pairs) -> int:
    return 20 * n + 8 * pairs + 1024


# ---------------------------------------------------------------------- token log-probabilities
def ce_token_logprob(logits, target, *, temperature=1.0, ignore_index=-100, with_entropy=True, logp=None, entropy=None,
                     stats=None, stream=None):
    """(logp [n], entropy [n] or None, stats [n, 4]) of softmax(logits / temperature):
    the log-probability of every row's target and the entropy of its
    distribution. Ignored rows give 0, targets outside the vocabulary NaN.
    One kernel, no workspace."""
    p = _params(logits, target, ignore_index)
    n = p.n_rows
    call = _Call(logits, (target, logp, entropy, stats), stream)
    logp, entropy, stats = _outputs(call, n, logp, entropy, stats, with_entropy)
    call.run("ce_token_logprob", _byref(p), float(temperature), _ptr(logits), _ptr(target), _ptr(logp),
             _ptr(entropy), _ptr(stats))
    return logp, entropy, stats


def ce_token_logprob_backward(logits, target, stats, grad_logp, *, grad_entropy=None, temperature=1.0,
                              ignore_index=-100, grad=None, stream=None):
    """The gradient of sum(grad_logp logp + grad_entropy entropy), from the
    statistics ce_token_logprob returned for the same logits (with the
    entropy, if grad_entropy is given). Written over the logits unless
    ``grad`` is given; returned."""
    p = _params(logits, target, ignore_index)
    n = p.n_rows
    grad, ld = _grad_buffer(logits, grad, p)
    call = _Call(logits, (target, stats, grad_logp, grad_entropy, grad), stream)
    _vec("grad_logp", grad_logp, n, call)
    _vec("grad_entropy", grad_entropy, n, call)
    _rows4("stats", stats, n, call)
    call.run("ce_token_logprob_backward", _byref(p), float(temperature), _ptr(logits), _ptr(target), _ptr(stats),
             _ptr(grad_logp), _ptr(grad_entropy), _ptr(grad), ld)
    return grad


# ---------------------------------------------------------------------- policy loss
def ce_policy_fwd_bwd(logits, target, advantage, *, old_logp=None, ref_logp=None, row_weight=None, clip_low=0.2,
                      clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, temperature=1.0, ignore_index=-100,
                      reduction="mean", grad_output=None, grad=None, loss=None, row_stats=None, ws=None, stream=None):
    """(loss, grad) of the clipped policy loss with a KL term and an entropy
    bonus; ``grad`` (times grad_output, or 1) is written over the logits
    unless a buffer is given. ``row_stats``: an fp32 [n, 4] tensor that
    receives {logp, entropy, ratio, KL} of every row."""
    p = _params(logits, target, ignore_index, reduction)
    n = p.n_rows
    grad, ld = _grad_buffer(logits, grad, p)
    call = _Call(logits, (target, grad, loss), stream)
    _vec("advantage", advantage, n, call)
    _vec("old_logp", old_logp, n, call)
    _vec("ref_logp", ref_logp, n, call)
    _vec("row_weight", row_weight, n, call)
    _rows4("row_stats", row_stats, n, call)
    m = n if reduction == "none" else 1
    _vec("grad_output", grad_output, m, call)
    loss = call.empty(m) if loss is None else _vec("loss", loss, m, call)
    q = ce_policy_params(float(temperature), float(clip_low), float(clip_high), float(kl_coef), float(entropy_coef), 0)
    ws, nbytes = _workspace(call, ws, _policy_ws_bytes(n))
    call.run("ce_policy_fwd_bwd", _byref(p), _byref(q), _ptr(logits), _ptr(target), _ptr(advantage),
             _ptr(old_logp), _ptr(ref_logp), _ptr(row_weight), _ptr(grad_output), _ptr(loss), _ptr(row_stats),
             _ptr(grad), ld, _ptr(ws), nbytes)
    return loss, grad


# ---------------------------------------------------------------------- preference loss
def ce_preference_fwd_bwd(logits, target, seq_offsets, *, ref_logp=None, loss_kind="sigmoid", beta=0.1,
                          label_smoothing=0.0, length_normalize=False, ignore_index=-100, reduction="mean",
                          grad_output=None, grad=None, loss=None, seq_logp=None, ws=None, stream=None):
    """(loss, seq_logp [2 P], grad) of the paired preference loss. Sequence j
    is the rows seq_offsets[j] .. seq_offsets[j + 1] (2 P + 1 offsets); the
    first P sequences are the preferred ones, the last P their counterparts
    in the same order. ``seq_logp`` holds every sequence's log-probability
    (its mean per token with ``length_normalize``), ``ref_logp`` the
    reference model's values of the same kind. ``grad`` (times grad_output,
    or 1) is written over the logits unless a buffer is given."""
    p = _params(logits, target, ignore_index, reduction)
    n = p.n_rows
    if seq_offsets.dtype not in (torch.int64, torch.int32) or seq_offsets.dim() != 1 \
            or not seq_offsets.is_contiguous() or seq_offsets.shape[0] % 2 != 1:
        raise ValueError("seq_offsets must be a contiguous 1-D int64 or int32 tensor of 2 P + 1 entries")
    if loss_kind not in PREFERENCE_KINDS:
        raise ValueError(f"unknown loss_kind {loss_kind!r}")
    pairs = seq_offsets.shape[0] // 2
    grad, ld = _grad_buffer(logits, grad, p)
    call = _Call(logits, (target, seq_offsets, grad), stream)
    _vec("ref_logp", ref_logp, 2 * pairs, call)
    m = pairs if reduction == "none" else 1
    _vec("grad_output", grad_output, m, call)
    loss = call.empty(m) if loss is None else _vec("loss", loss, m, call)
    seq_logp = call.empty(2 * pairs) if seq_logp is None else _vec("seq_logp", seq_logp, 2 * pairs, call)
    q = ce_preference_params(pairs, PREFERENCE_KINDS[loss_kind], 1 if seq_offsets.dtype == torch.int32 else 0,
                             1 if length_normalize else 0, float(beta), float(label_smoothing), 0)
    ws, nbytes = _workspace(call, ws, _preference_ws_bytes(n, pairs))
    call.run("ce_preference_fwd_bwd", _byref(p), _byref(q), _ptr(logits), _ptr(target), _ptr(seq_offsets),
             _ptr(ref_logp), _ptr(grad_output), _ptr(loss), _ptr(seq_logp), _ptr(grad), ld, _ptr(ws), nbytes)
    return loss, seq_logp, grad


# ---------------------------------------------------------------------- autograd
def _once(ctx):
    """The backward passes here write or scale one buffer in place: a second
    run over the same graph would use it up again."""
    if getattr(ctx, "spent", False):
        raise CEError("the gradient of this call has been used up (its buffer was handed out by an earlier backward)")
    ctx.spent = True


class TokenLogprobFunction(torch.autograd.Function):
    """Forward reads the logits once and keeps 16 bytes a row; the backward
    reads them again and writes the gradient (over them with ``inplace``)."""

    @staticmethod
    def forward(ctx, logits, target, temperature, ignore_index, with_entropy, inplace):
        x = logits.detach()
        logp, entropy, stats = ce_token_logprob(x, target, temperature=temperature, ignore_index=ignore_index,
                                                with_entropy=with_entropy)
        ctx.save_for_backward(logits, target, stats)
        ctx.args = temperature, ignore_index, inplace
        ctx.set_materialize_grads(False)
        return (logp, entropy) if with_entropy else logp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp, grad_entropy=None):
        if grad_logp is None and grad_entropy is None:
            return None, None, None, None, None, None
        logits, target, stats = ctx.saved_tensors
        temperature, ignore_index, inplace = ctx.args
        x = logits.detach()
        if inplace:
            _once(ctx)
        g = None if grad_logp is None else grad_logp.detach().to(torch.float32).contiguous()
        h = None if grad_entropy is None else grad_entropy.detach().to(torch.float32).contiguous()
        out = ce_token_logprob_backward(x, target, stats, g, grad_entropy=h, temperature=temperature,
                                        ignore_index=ignore_index, grad=None if inplace else torch.empty_like(x))
        return out, None, None, None, None, None


def token_logprob(logits, target, *, temperature=1.0, ignore_index=-100, with_entropy=False, inplace=False):
    """Differentiable log-probabilities of the targets (and the entropies, as
    a pair, with ``with_entropy``). ``inplace``: the backward writes the
    gradient over the logits, which nothing else may use then."""
    return TokenLogprobFunction.apply(logits, target, temperature, ignore_index, with_entropy, inplace)


class _FormedGradientFunction(torch.autograd.Function):
    """A loss whose gradient the forward forms (one read and one write of the
    logits), times ``upstream`` where that is given; the backward multiplies it
    by grad_output over ``upstream``, skipped on the device where that is 1
    (otherwise the product is rounded a second time)."""

    @staticmethod
    def forward(ctx, logits, upstream, inplace, per_row, run):
        x = logits.detach()
        if upstream is not None:
            if not torch.is_tensor(upstream):
                raise TypeError("grad_output must be a tensor on the logits' device")
            upstream = upstream.detach().reshape(-1).contiguous()
        loss, grad = run(x, x if inplace else torch.empty_like(x), upstream)
        ctx.save_for_backward(grad, upstream)
        ctx.per_row = per_row
        return loss if per_row else loss.reshape(())

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        _once(ctx)
        grad, upstream = ctx.saved_tensors
        if grad.shape[0]:
            g = grad_out.detach().to(torch.float32).reshape(-1).contiguous()
            with torch.cuda.device(grad.device):
                if upstream is not None:
                    g = torch.where(g == upstream, 1.0, g / upstream)
                ce_scale_grad(grad, g, reduction="none" if ctx.per_row else "mean")
        return grad, None, None, None, None


def policy_loss(logits, target, advantage, *, old_logp=None, ref_logp=None, row_weight=None, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, temperature=1.0, ignore_index=-100, reduction="mean",
                grad_output=None, row_stats=None, inplace=False):
    """Differentiable ce_policy_fwd_bwd: the loss (a scalar, or [n] for
    reduction "none"). The gradient reaches the logits only; advantage,
    old_logp, ref_logp and row_weight are constants. ``inplace``: the
    gradient is formed over the logits, which nothing else may use then.
    ``grad_output``: what the backward will be given (an fp32 tensor of one
    element, or [n] for reduction "none"; not 0 where the latter is not): a
    loss scale, one over the accumulation steps. The forward has it in the
    gradient's one rounding then. Without it the gradient is rounded to the
    logits' type at 1 and scaled afterwards, so that in fp16 what lies below
    2^-25 at 1 is 0 whatever the loss scale."""
    def run(x, grad, upstream):
        return ce_policy_fwd_bwd(x, target, advantage, old_logp=old_logp, ref_logp=ref_logp, row_weight=row_weight,
                                 clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, entropy_coef=entropy_coef,
                                 temperature=temperature, ignore_index=ignore_index, reduction=reduction,
                                 grad_output=upstream, grad=grad, row_stats=row_stats)
    return _FormedGradientFunction.apply(logits, grad_output, inplace, reduction == "none", run)


def preference_loss(logits, target, seq_offsets, *, ref_logp=None, loss_kind="sigmoid", beta=0.1, label_smoothing=0.0,
                    length_normalize=False, ignore_index=-100, reduction="mean", grad_output=None, seq_logp=None,
                    inplace=False):
    """Differentiable ce_preference_fwd_bwd: the scalar loss ("mean" or
    "sum"). ``seq_logp``, if given, receives the sequences' values. The
    gradient reaches the logits only. ``grad_output`` (one element) and
    ``inplace`` as in policy_loss."""
    if reduction not in ("mean", "sum"):
        raise ValueError("preference_loss takes reduction 'mean' or 'sum'")

    def run(x, grad, upstream):
        loss, _, grad = ce_preference_fwd_bwd(x, target, seq_offsets, ref_logp=ref_logp, loss_kind=loss_kind, beta=beta,
                                              label_smoothing=label_smoothing, length_normalize=length_normalize,
                                              ignore_index=ignore_index, reduction=reduction, grad_output=upstream,
                                              grad=grad, seq_logp=seq_logp)
        return loss, grad
    return _FormedGradientFunction.apply(logits, grad_output, inplace, False, run)


# ---------------------------------------------------------------------- linear head
# dZ of all rows at once (bf16) up to this many bytes: grad_weight is then
# formed by one product, without a sum over chunks
DZ_BYTES = 16 << 30


def _linear_params(hidden, weight, target, ignore_index):
    if hidden.dim() != 2 or weight.dim() != 2 or not hidden.is_contiguous() or not weight.is_contiguous():
        raise ValueError("hidden and weight must be contiguous 2-D tensors")
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("hidden and weight must be bf16")
    if hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden and weight must have the same number of columns")
    n, V = hidden.shape[0], weight.shape[0]
    return ce_params(n, V, V, ignore_index, None, 0.0, CE_DT[torch.bfloat16], 0, _check_target(target, n))


def _linear_ws_bytes(p, hidden_dim, chunk_rows) -> int:
    out = ctypes.c_size_t()
    _check(_lib.flce_token_logprob_workspace_size(_byref(p), hidden_dim, chunk_rows, _byref(out)),
           "flce_token_logprob_workspace_size")
    return out.value


def flce_token_logprob(hidden, weight, target, *, bias=None, temperature=1.0, ignore_index=-100, with_entropy=True,
                       logp=None, entropy=None, stats=None, ws=None, stream=None):
    """(logp [n], entropy [n] or None, stats [n, 4]) of softmax((hidden
    weight^T + bias) / temperature) without the logits in memory: hidden
    [n, H] and weight [V, H] bf16, bias [V] fp32."""
    p = _linear_params(hidden, weight, target, ignore_index)
    n, H = hidden.shape
    call = _Call(hidden, (weight, target, bias, logp, entropy, stats), stream)
    _vec("bias", bias, weight.shape[0], call)
    logp, entropy, stats = _outputs(call, n, logp, entropy, stats, with_entropy)
    ws, nbytes = _workspace(call, ws, _linear_ws_bytes(p, H, 0))
    call.run("flce_token_logprob", _byref(p), H, float(temperature), _ptr(hidden), _ptr(weight), _ptr(bias),
             _ptr(target), _ptr(logp), _ptr(entropy), _ptr(stats), _ptr(ws), nbytes)
    return logp, entropy, stats


def flce_token_logprob_backward(hidden, weight, target, stats, grad_logp, *, grad_entropy=None, bias=None,
                                temperature=1.0, ignore_index=-100, chunk_rows=None, grad_hidden=None,
                                grad_weight=None, grad_bias=None, ws=None, stream=None):
    """(grad_hidden [n, H] bf16, grad_weight [V, H] fp32 or bf16, grad_bias
    [V] fp32 or None) of sum(grad_logp logp + grad_entropy entropy), from the
    statistics flce_token_logprob returned. ``chunk_rows`` rows of the logits'
    gradient (bf16) are held at a time: all of them by default where that
    takes at most 16 GB. ``grad_weight``: a buffer of either type; by
    default fp32. bf16 needs all rows in one chunk."""
    p = _linear_params(hidden, weight, target, ignore_index)
    (n, H), V = hidden.shape, weight.shape[0]
    call = _Call(hidden, (weight, target, stats, grad_logp, grad_entropy, bias, grad_hidden, grad_weight, grad_bias), stream)
    _vec("bias", bias, V, call)
    _vec("grad_logp", grad_logp, n, call)
    _vec("grad_entropy", grad_entropy, n, call)
    _rows4("stats", stats, n, call)
    if chunk_rows is None:
        chunk_rows = _chunk_rows(n, V)
    if grad_hidden is None:
        grad_hidden = call.empty(n, H, dtype=torch.bfloat16)
    elif grad_hidden.shape != hidden.shape or grad_hidden.dtype != torch.bfloat16 or not grad_hidden.is_contiguous():
        raise ValueError("grad_hidden must be a contiguous bf16 tensor of hidden's shape")
    if grad_weight is None:
        grad_weight = call.empty(V, H)
    elif grad_weight.shape != weight.shape or grad_weight.dtype not in (torch.float32, torch.bfloat16) \
            or not grad_weight.is_contiguous():
        raise ValueError("grad_weight must be a contiguous fp32 or bf16 tensor of weight's shape")
    if grad_bias is None and bias is not None:
        grad_bias = call.empty(V)
    _vec("grad_bias", grad_bias, V, call)
    ws, nbytes = _workspace(call, ws, _linear_ws_bytes(p, H, chunk_rows))
    call.run("flce_token_logprob_backward", _byref(p), H, float(temperature), _ptr(hidden), _ptr(weight), _ptr(bias),
             _ptr(target), _ptr(stats), _ptr(grad_logp), _ptr(grad_entropy), _ptr(grad_hidden), _ptr(grad_weight),
             CE_DT[grad_weight.dtype], _ptr(grad_bias), chunk_rows, _ptr(ws), nbytes)
    return grad_hidden, grad_weight, grad_bias


def _chunk_rows(n, V) -> int:
    fit = max(128, DZ_BYTES // (2 * V) // 128 * 128)
    return max(1, min(n, fit))


class LinearTokenLogprobFunction(torch.autograd.Function):
    """Forward: one product with the statistics in its epilogue. Backward: the
    logits formed again, their gradient in bf16, two products. grad_weight
    and grad_bias come in the parameters' types, as autograd has it."""

    @staticmethod
    def forward(ctx, hidden, weight, bias, target, temperature, ignore_index, with_entropy):
        logp, entropy, stats = flce_token_logprob(hidden.detach(), weight.detach(), target,
                                                  bias=None if bias is None else bias.detach(),
                                                  temperature=temperature, ignore_index=ignore_index,
                                                  with_entropy=with_entropy)
        ctx.save_for_backward(hidden, weight, bias, target, stats)
        ctx.args = temperature, ignore_index
        ctx.set_materialize_grads(False)
        return (logp, entropy) if with_entropy else logp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp, grad_entropy=None):
        hidden, weight, bias, target, stats = ctx.saved_tensors
        if grad_logp is None and grad_entropy is None:
            return None, None, None, None, None, None, None
        g = None if grad_logp is None else grad_logp.detach().to(torch.float32).contiguous()
        h = None if grad_entropy is None else grad_entropy.detach().to(torch.float32).contiguous()
        temperature, ignore_index = ctx.args
        n, V = hidden.shape[0], weight.shape[0]
        chunk = _chunk_rows(n, V)
        gw = torch.empty(weight.shape, dtype=torch.bfloat16 if chunk >= n else torch.float32, device=weight.device)
        gh, gw, gb = flce_token_logprob_backward(hidden.detach(), weight.detach(), target, stats, g, grad_entropy=h,
                                                 bias=None if bias is None else bias.detach(), temperature=temperature,
                                                 ignore_index=ignore_index, chunk_rows=chunk, grad_weight=gw)
        return gh, gw.to(weight.dtype), gb, None, None, None, None


def linear_token_logprob(hidden, weight, target, *, bias=None, temperature=1.0, ignore_index=-100, with_entropy=False):
    """Differentiable log-probabilities of a linear head's targets (and the
    entropies, as a pair, with ``with_entropy``), the logits never in memory:
    hidden [n, H] and weight [V, H] bf16, bias [V] fp32 or None."""
    return LinearTokenLogprobFunction.apply(hidden, weight, bias, target, temperature, ignore_index, with_entropy)
