"""Scores of given tokens: log-probabilities with the row's log-sum-exp and entropy, the token's rank and the most likely
alternatives, and the gradient of what was scored with respect to the logits.

Functions check their tensors and allocate their outputs on the stream that the call runs on, as those of the serving
head do, and the usual calls go through _lib.calls() as theirs; the compute is in the library. Nothing here is recorded by
autograd: score_tokens_grad() is the backward pass, called with what the forward pass returned.
"""
from typing import NamedTuple

import torch

from . import _lib
from .head import _CODE, _F32, _I32, _check, _like, _rows, _status, _vec


class TokenScores(NamedTuple):
    """What score_tokens() returns for n rows: float32 [n] but for ranks int32 [n], top_ids int32 [n, top] and
    top_logprobs float32 [n, top]."""
    logprobs: torch.Tensor
    lse: torch.Tensor
    entropy: torch.Tensor
    ranks: torch.Tensor
    top_ids: torch.Tensor
    top_logprobs: torch.Tensor


def _count(name, v, most):
    if isinstance(v, bool) or not isinstance(v, int) or v < 0 or v > most:
        raise ValueError("%s: an integer from 0 to %d expected, got %r" % (name, most, v))
    return v


def score_tokens(logits, tokens, top=0, d_status=None, stream=None):
    """Scores of one given token per row of logits [n, V] (bfloat16 or float32, cuda, rows may lie apart): its
    log-probability and its rank (0: the argmax), the row's log-sum-exp and entropy, and the `top` most likely tokens with
    their log-probabilities. tokens: int32 [n], -1 for none (logprob NaN, rank -1). Returns TokenScores; a row with
    nothing in it (lse -inf), a NaN or +inf gives NaN and -1, the last two and a token >= V with a bit in d_status. Not recorded by
    autograd, whether or not logits require a gradient: score_tokens_grad() makes it. Results may share their memory by
    type: one that is kept or saved keeps or saves those beside it, unless it is cloned."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return score_tokens(logits, tokens, top, d_status)
    if d_status is None:
        r = _lib.calls().score(logits, tokens, top)
        if r is not None:
            return TokenScores._make(r) if type(r) is tuple else _check("ds_score_tokens", r)
    n, V, ld, index = _rows("logits", logits, _CODE)
    _count("top", top, min(V, _lib.DS_SCORE_MAX_TOP))
    if tokens is None:
        raise ValueError("tokens are needed")
    tok = _vec("tokens", tokens, n, _I32, index)
    st = _status(d_status, index)
    dev = logits.device
    r = TokenScores(*(torch.empty(n, dtype=t, device=dev) for t in (_F32, _F32, _F32, _I32)),
                    torch.empty((n, top), dtype=_I32, device=dev), torch.empty((n, top), dtype=_F32, device=dev))
    _check("ds_score_tokens", _lib.load().ds_score_tokens(
        logits.data_ptr(), _CODE[logits.dtype], n, V, ld, tok, top, r.logprobs.data_ptr(), r.lse.data_ptr(),
        r.entropy.data_ptr(), r.ranks.data_ptr(), r.top_ids.data_ptr(), r.top_logprobs.data_ptr(), st, _lib.raw_stream()))
    return r


def score_tokens_grad(logits, tokens, lse, entropy=None, g_logprobs=None, g_entropy=None, out=None, d_status=None,
                      stream=None):
    """The loss's gradient by the logits [n, V] that score_tokens() scored: out = g_logprobs ([j == token] - p) -
    g_entropy p (log p + entropy), p = exp(logits - lse), in the logits' type. lse and entropy: what score_tokens()
    returned; g_logprobs, g_entropy: float32 [n], the loss's gradient by its logprobs and entropy, None for none of one.
    out: such a tensor (rows may lie apart), the logits themselves to overwrite them; allocated when None. A row without
    a token has no g_logprobs, whatever is there; one with nothing in it gets zeros."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return score_tokens_grad(logits, tokens, lse, entropy, g_logprobs, g_entropy, out, d_status)
    if out is None and d_status is None:
        r = _lib.calls().score_grad(logits, tokens, lse, entropy, g_logprobs, g_entropy)
        if r is not None:
            return _check("ds_score_tokens_grad", r) if type(r) is int else r
    n, V, ld, index = _rows("logits", logits, _CODE)
    if tokens is None or lse is None or (g_logprobs is None and g_entropy is None):
        raise ValueError("tokens, lse and g_logprobs or g_entropy are needed")
    if g_entropy is not None and entropy is None:
        raise ValueError("entropy is needed with g_entropy")
    tok = _vec("tokens", tokens, n, _I32, index)
    zp = _vec("lse", lse, n, _F32, index)
    hp = _vec("entropy", entropy, n, _F32, index)
    gl = _vec("g_logprobs", g_logprobs, n, _F32, index)
    gh = _vec("g_entropy", g_entropy, n, _F32, index)
    st = _status(d_status, index)
    out, ldo = _like(out, logits, ld, index)
    _check("ds_score_tokens_grad", _lib.load().ds_score_tokens_grad(
        logits.data_ptr(), _CODE[logits.dtype], n, V, ld, tok, zp, hp, gl, gh, out.data_ptr(), ldo, st,
        _lib.raw_stream()))
    return out
