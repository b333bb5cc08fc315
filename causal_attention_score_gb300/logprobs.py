"""Log probabilities of given tokens, with entropy, top alternatives and gradient: Python
binding of their C entry points (argument marshalling only, as in ops.py)."""
from __future__ import annotations

import torch

from . import _lib
from .ops import _allocate
from .serving import _ANY, _DTYPE, _device_of, _elsewhere, _stream_ptr


def _matrix(t: torch.Tensor, name: str, dtypes, dev: int, shape=None) -> int:
    """The row stride of a [rows, vocab] tensor on device ``dev``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise _elsewhere(t.device, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be [rows, vocab]")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    row, one = t.stride()
    rows, vocab = t.shape
    if one != 1 and vocab > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return row if rows > 1 else vocab  # the stride of one row means nothing


def _array(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: int) -> int:
    """Address of a contiguous tensor of this type and shape on device ``dev``."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise _elsewhere(t.device, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def token_logprobs_forward(logprob: torch.Tensor, entropy: torch.Tensor, stats: torch.Tensor,
                           logits: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0,
                           top_logprob: torch.Tensor | None = None,
                           top_token: torch.Tensor | None = None, stream=None) -> None:
    """For each row of ``logits`` [rows, vocab] (bf16, fp16 or fp32, any row stride) and its
    token in ``tokens`` (int32 [rows]; negative: the row is left out), with softmax(scale x):
    the token's log probability into ``logprob`` [rows], the distribution's entropy into
    ``entropy`` [rows], what the backward call needs into ``stats`` [rows, 2], and with
    ``top_logprob`` and ``top_token`` (fp32 and int32 [rows, top], top <= 32) the alternatives
    of the largest logits; see token_logprobs_forward in include/csa.h."""
    dev = _device_of(logits, "logits")
    stride = _matrix(logits, "logits", _ANY, dev)
    rows, vocab = logits.shape
    f32, top = torch.float32, 0
    if (top_logprob is None) != (top_token is None):
        raise ValueError("top_logprob and top_token go together")
    if top_token is not None:
        if not isinstance(top_token, torch.Tensor) or top_token.dim() != 2:
            raise ValueError("top_token must be [rows, top]")
        top = top_token.shape[1]
    p_log = _array(logprob, "logprob", f32, (rows,), dev)
    p_ent = _array(entropy, "entropy", f32, (rows,), dev)
    p_stats = _array(stats, "stats", f32, (rows, 2), dev)
    p_tok = _array(tokens, "tokens", torch.int32, (rows,), dev)
    p_top = p_index = None
    if top_token is not None:
        p_top = _array(top_logprob, "top_logprob", f32, (rows, top), dev)
        p_index = _array(top_token, "top_token", torch.int32, (rows, top), dev)
        n, k = 4 * rows, 4 * rows * top  # (what the library does not check)
        if k and (-k < p_top - p_index < k or -k < p_top - p_log < n or -k < p_index - p_log < n):
            raise ValueError("top_logprob, top_token and logprob must not overlap")
    rc = (_lib._lib or _lib.load()).token_logprobs_forward(
        p_log, p_ent, p_stats, logits.data_ptr(), _DTYPE[logits.dtype], rows, vocab, stride, p_tok,
        scale, top, p_top, p_index, _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "token_logprobs_forward")


def token_logprobs_backward(dlogits: torch.Tensor, logits: torch.Tensor, tokens: torch.Tensor,
                            stats: torch.Tensor, entropy: torch.Tensor,
                            d_logprob: torch.Tensor | None = None,
                            d_entropy: torch.Tensor | None = None,
                            d_top: torch.Tensor | None = None,
                            top_token: torch.Tensor | None = None, scale: float = 1.0,
                            stream=None) -> None:
    """The gradient by the logits into ``dlogits`` (of their type; ``logits`` itself is fine),
    from the gradients by the forward call's outputs (fp32, any of them None) and its ``stats``,
    ``entropy`` and, with ``d_top``, ``top_token``; see token_logprobs_backward in
    include/csa.h."""
    dev = _device_of(logits, "logits")
    stride = _matrix(logits, "logits", _ANY, dev)
    d_stride = _matrix(dlogits, "dlogits", (logits.dtype,), dev, logits.shape)
    rows, vocab = logits.shape
    f32, top = torch.float32, 0
    if d_top is not None:
        if top_token is None:
            raise ValueError("d_top needs top_token")
        if not isinstance(d_top, torch.Tensor) or d_top.dim() != 2:
            raise ValueError("d_top must be [rows, top]")
        top = d_top.shape[1]

    def given(t, name, dtype, shape):
        return None if t is None else _array(t, name, dtype, shape, dev)

    rc = (_lib._lib or _lib.load()).token_logprobs_backward(
        dlogits.data_ptr(), logits.data_ptr(), _DTYPE[logits.dtype], rows, vocab, d_stride, stride,
        _array(tokens, "tokens", torch.int32, (rows,), dev), scale,
        _array(stats, "stats", f32, (rows, 2), dev), _array(entropy, "entropy", f32, (rows,), dev),
        given(d_logprob, "d_logprob", f32, (rows,)), given(d_entropy, "d_entropy", f32, (rows,)),
        top, given(d_top, "d_top", f32, (rows, top)),
        given(top_token if d_top is not None else None, "top_token", torch.int32, (rows, top)),
        _stream_ptr(stream, dev))
    if rc:
        _lib.check(rc, "token_logprobs_backward")


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, scale: float = 1.0,
                   stream=None):
    """Allocating form of token_logprobs_forward: (logprob, entropy, stats, top_logprob,
    top_token), allocated on the call's stream."""
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, vocab]")
    rows, device = logits.shape[0], logits.device

    def make(shape, dtype=torch.float32):
        return _allocate(torch.empty, shape, dtype, device, stream)

    got = (make((rows,)), make((rows,)), make((rows, 2)), make((rows, top)),
           make((rows, top), torch.int32))
    token_logprobs_forward(got[0], got[1], got[2], logits, tokens, scale, got[3], got[4], stream)
    return got
