"""Operators on a vocabulary's logits: log probabilities of given tokens with
entropy and top alternatives, distillation from a teacher's top alternatives,
and their gradients, as plain calls and as differentiable functions.

Logits are [rows, vocab], bf16 or float32, with unit column stride and any row
stride and alignment. With s = scale * logits (scale is 1 / temperature), a
column with s <= -1e8 is masked: probability and gradient 0. A token, label or
alternative < 0 is absent. include/nvfp4.h has the formulas and what rows with
nothing unmasked, NaN or indexes beyond the vocabulary give.

The recipe's runs are judged by their validation loss (gist.science summary of
"Pretraining Large Language Models with NVFP4", Resumen técnico §4). A linear
layer's logits go in, and the gradient that comes out is the dY that its
backward pass quantizes:

    teacher = token_logprobs(teacher_logits, top_k=64)
    r, dy = distill_step(student_logits, teacher.top_ids, teacher.top_logp,
                         d_loss=weights)

Every computation runs in the library's kernels on torch's current stream.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import _lib
from .autograd import once_differentiable


class TokenLogprobs(NamedTuple):
    """Per row, float32 (None: not asked for)."""

    logp: "object"      # of the given token
    entropy: "object"   # of the row's distribution, in nats
    lse: "object"       # ln of the sum of exponentials
    top_ids: "object"   # int32 [rows, top_k], falling probability; -1: no more unmasked
    top_logp: "object"  # [rows, top_k]


class Distilled(NamedTuple):
    """Per row, float32 (None: not asked for)."""

    loss: "object"      # divergence from the teacher, in nats
    logp: "object"      # of the label
    lse: "object"       # ln of the sum of exponentials
    lse_tail: "object"  # the same over the columns that are no alternative


def _rows(n, rows, device, apart=False):
    """n float32 vectors of a value per row, and their pointers: in one
    allocation (half the time of n), or each a tensor of its own, as an autograd
    function's outputs have to be (a view among several of one block may not be
    changed in place, and shares its version with them)."""
    if apart:
        out = [torch.empty(rows, dtype=torch.float32, device=device) for _ in range(n)]
        return out, [t.data_ptr() for t in out]
    block = torch.empty(n, rows, dtype=torch.float32, device=device)
    at = block.data_ptr()
    return block.unbind(0), [at + 4 * rows * i for i in range(n)]


def _workspace(matrix, k, device):
    """(workspace or None, its pointer, its size). The tensor has to live until
    the call has been enqueued."""
    n = _lib.nvfp4_logits_workspace(matrix[1], matrix[2], matrix[3], k)
    if n == 0:
        return None, None, 0
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), n


def _mode(tail):
    return _lib.DISTILL_TAIL if tail else _lib.DISTILL_RENORM


def token_logprobs(logits, tokens=None, top_k: int = 0, scale: float = 1.0, entropy: bool = True,
                   dev_status=None) -> TokenLogprobs:
    """Log probabilities of the tokens (int64 [rows], or None), the entropy and
    the top_k most probable tokens of each row (ties to the lowest id)."""
    return _token_logprobs(logits, tokens, top_k, scale, entropy, dev_status)


def _token_logprobs(logits, tokens, top_k, scale, entropy, dev_status, apart=False):
    matrix, stream = _lib._logits(logits)
    rows, device = matrix[2], logits.device
    given = _lib._vector(tokens, "tokens", torch.int64, (rows,), logits)
    out, at = _rows(1 + (given is not None) + bool(entropy), rows, device, apart)
    logp = h = p_logp = p_h = ids = top = p_ids = p_top = None
    if given is not None:
        logp, p_logp = out[1], at[1]
    if entropy:
        h, p_h = out[-1], at[-1]
    if top_k:
        ids = torch.empty(rows, top_k, dtype=torch.int32, device=device)
        top = torch.empty(rows, top_k, dtype=torch.float32, device=device)
        p_ids, p_top = ids.data_ptr(), top.data_ptr()
    ws, p_ws, n_ws = _workspace(matrix, top_k, device)
    _lib._check("nvfp4_token_logprobs", _lib.lib().nvfp4_token_logprobs(
        *matrix, given, scale, top_k, p_logp, p_h, at[0], p_ids, p_top, p_ws, n_ws,
        _lib._status_word(dev_status, logits), stream))
    return TokenLogprobs(logp, h, out[0], ids, top)


def token_logprobs_backward(logits, tokens, lse, entropy=None, d_logp=None, d_entropy=None,
                            scale: float = 1.0, out=None):
    """The logits' gradient from those of logp and entropy (float32 [rows], or
    None), with the lse and entropy of the forward call. ``out`` may be the
    logits themselves."""
    dz = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device) if out is None else out
    _lib.nvfp4_token_logprobs_backward(logits, tokens, scale, lse, entropy, d_logp, d_entropy, dz)
    return dz


def distill(logits, teacher_ids, teacher_logp, labels=None, tail: bool = True, scale: float = 1.0,
            dev_status=None) -> Distilled:
    """Divergence of the logits from a teacher known by its alternatives
    (int32 ids and float32 log probabilities, both [rows, k], as
    token_logprobs gives them; None: no teacher), and the labels' log
    probabilities (int64 [rows], or None). tail: the teacher's remaining mass
    is compared with the student's outside the alternatives; else the
    alternatives are renormalised to 1."""
    return _distill(logits, teacher_ids, teacher_logp, labels, tail, scale, dev_status)


def _distill(logits, teacher_ids, teacher_logp, labels, tail, scale, dev_status, apart=False):
    matrix, stream = _lib._logits(logits)
    teacher = _lib._teacher(logits, teacher_ids, teacher_logp, labels)
    out, at = _rows(3 + (labels is not None), matrix[2], logits.device, apart)
    ws, p_ws, n_ws = _workspace(matrix, teacher[2], logits.device)
    _lib._check("nvfp4_distill", _lib.lib().nvfp4_distill(
        *matrix, *teacher, _mode(tail), scale, at[0], None if labels is None else at[3], at[1],
        at[2], p_ws, n_ws, _lib._status_word(dev_status, logits), stream))
    return Distilled(out[0], None if labels is None else out[3], out[1], out[2])


def distill_backward(logits, teacher_ids, teacher_logp, labels, lse, lse_tail, d_loss=None,
                     d_logp=None, tail: bool = True, scale: float = 1.0, out=None):
    """The logits' gradient from those of the loss and of the labels' log
    probabilities (float32 [rows], or None), with the lse and lse_tail of the
    forward call. ``out`` may be the logits themselves."""
    dz = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device) if out is None else out
    _lib.nvfp4_distill_backward(logits, teacher_ids, teacher_logp, labels, _mode(tail), scale, lse,
                                lse_tail, d_loss, d_logp, dz)
    return dz


def distill_step(logits, teacher_ids, teacher_logp, labels=None, d_loss=None, d_logp=None,
                 tail: bool = True, scale: float = 1.0, out=None, dev_status=None):
    """distill and distill_backward in one call, for weights (d_loss, d_logp)
    that are known beforehand. Without a teacher it is the cross entropy of
    the labels. Returns (Distilled, the logits' gradient)."""
    matrix, stream = _lib._logits(logits)
    rows, device = matrix[2], logits.device
    teacher = _lib._teacher(logits, teacher_ids, teacher_logp, labels)
    gk = _lib._vector(d_loss, "d_loss", torch.float32, (rows,), logits)
    gl = _lib._vector(d_logp, "d_logp", torch.float32, (rows,), logits)
    dz = torch.empty(logits.shape, dtype=logits.dtype, device=device) if out is None else out
    gradient = _lib._gradient(dz, logits)
    r, at = _rows(3 + (labels is not None), rows, device)
    ws, p_ws, n_ws = _workspace(matrix, teacher[2], device)
    _lib._check("nvfp4_distill_step", _lib.lib().nvfp4_distill_step(
        *matrix, *teacher, _mode(tail), scale, gk, gl, at[0], None if labels is None else at[3],
        at[1], at[2], *gradient, p_ws, n_ws, _lib._status_word(dev_status, logits), stream))
    return Distilled(r[0], None if labels is None else r[3], r[1], r[2]), dz


# ---------------------------------------------------------------------------
# Differentiable forms (once: a second derivative raises)
# ---------------------------------------------------------------------------


class TokenLogprobsFunction(torch.autograd.Function):
    """(logp, entropy) of the logits; the gradient of both."""

    @staticmethod
    def forward(ctx, logits, tokens, scale: float):
        r = _token_logprobs(logits, tokens, 0, scale, True, None, apart=True)
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return r.logp, r.entropy

    @staticmethod
    @once_differentiable
    def backward(ctx, d_logp, d_entropy):
        logits, tokens, lse, entropy = ctx.saved_tensors
        if d_logp is None and d_entropy is None:
            return None, None, None
        dense = lambda t: None if t is None else t.contiguous()  # noqa: E731
        return token_logprobs_backward(logits, tokens, lse, entropy, dense(d_logp),
                                       dense(d_entropy), ctx.scale), None, None


class DistillFunction(torch.autograd.Function):
    """(loss, logp) of the logits against a teacher's alternatives and labels
    (both may be None); the gradient of both."""

    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logp, labels, tail: bool, scale: float):
        r = _distill(logits, teacher_ids, teacher_logp, labels, tail, scale, None, apart=True)
        ctx.save_for_backward(logits, teacher_ids, teacher_logp, labels, r.lse, r.lse_tail)
        ctx.how = (tail, scale)
        ctx.set_materialize_grads(False)
        return r.loss, r.logp

    @staticmethod
    @once_differentiable
    def backward(ctx, d_loss, d_logp):
        if d_loss is None and d_logp is None:
            return (None,) * 6
        dense = lambda t: None if t is None else t.contiguous()  # noqa: E731
        dz = distill_backward(*ctx.saved_tensors, dense(d_loss), dense(d_logp), *ctx.how)
        return dz, None, None, None, None, None
