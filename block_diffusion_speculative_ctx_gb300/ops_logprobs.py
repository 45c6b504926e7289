"""Log probabilities of tokens and their gradient over torch tensors: argument checks and
marshalling, as in ops.py.

    token_logprobs       log probabilities and ranks of given tokens, entropies, likeliest tokens
    token_logprobs_grad  gradient of a loss of them by the logits"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from . import load
from . import ops as _ops
from .ops import _DTYPES, _F, _F32T, _I32, _I32T, _I64, _P, _bad, _call, _device

LOGPROBS_MAX_TOKENS = LOGPROBS_MAX_TOP = 32


class dflash_logprobs_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "rows", "vocab", "n", "k")] + [("inv_temperature", _F), ("ld_logits", _I64)]
                + [(n, _P) for n in ("logits", "tokens", "logprobs", "ranks", "entropy", "lse", "top_ids", "top_logprobs", "lse_parts")])


class dflash_logprobs_grad_args(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("dtype", "rows", "vocab", "n")] + [("inv_temperature", _F), ("reserved", _I32)]
                + [(n, _I64) for n in ("ld_logits", "ld_out")]
                + [(n, _P) for n in ("logits", "tokens", "lse", "grad_logprobs", "entropy", "grad_entropy", "out", "lse_parts")])


# (packed forms of the structs, as in ops.py)
_LOGPROBS, _GRAD = struct.Struct("5ifq9Q"), struct.Struct("4ifi2q8Q")


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor
    ranks: torch.Tensor
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


def _logits(name, t, dev):
    if t.dim() != 2:
        _bad(f"{name} must be [rows, vocab]")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        _bad(f"{name} must be float32 or bfloat16, not {t.dtype}")
    rows, vocab = t.shape
    if vocab < 1:
        _bad(f"{name} must hold a token a row")
    return dt, rows, vocab, max(_ops._mat(name, t, t.dtype, rows, vocab, dev), vocab)


def _tokens(t, rows):
    """Tokens a row of tokens [rows] or [rows, n]."""
    if t.dim() not in (1, 2) or t.shape[0] != rows:
        _bad(f"tokens must be [{rows}] or [{rows}, n]")
    n = 1 if t.dim() == 1 else t.shape[1]
    if n > LOGPROBS_MAX_TOKENS:
        _bad(f"at most {LOGPROBS_MAX_TOKENS} tokens a row")
    return n


def _inverse(temperature):
    if not 2.0 ** -20 <= temperature <= 2.0 ** 20:
        _bad("temperature must be in [2^-20, 2^20]")
    return 1.0 / temperature


def _alike(name, t, like, dtype, device):
    """An output of the shape `like`, allocated when None."""
    if t is None:
        return torch.empty(like, dtype=dtype, device=device)
    if t.shape != like:
        _bad(f"{name} must be {list(like)}, not {list(t.shape)}")
    return t


def token_logprobs(logits, tokens, *, top: int = 0, temperature: float = 1.0, logprobs=None, ranks=None, entropy=None,
                   lse=None, top_ids=None, top_logprobs=None, lse_parts=None) -> TokenLogprobs:
    """Log probabilities of given tokens (``dflash_token_logprobs``).

    logits: [rows, vocab] (fp32 or bf16); tokens: int32 [rows] or [rows, n] (n <= 32; an id outside the vocabulary
    is padding).  The law is softmax(logits / temperature).  Gives ``logprobs`` (of tokens' shape; padding 0),
    ``ranks`` (int32, tokens ahead of each; padding -1), ``entropy`` and ``lse`` [rows], and for top > 0 the
    likeliest tokens' ``top_ids`` and ``top_logprobs`` [rows, top], the lower id first among equals (top <= 32;
    -1 and -inf where fewer tokens are above -inf).  All fp32; missing outputs are allocated, but for ``lse_parts``
    ([rows, 2], written when given): the largest logit and the rest of lse, for the gradient of rows of any size."""
    dev = _device(logits, logits, logprobs, entropy, lse, top_logprobs, lse_parts)
    dt, rows, vocab, ld = _logits("logits", logits, dev)
    n = _tokens(tokens, rows)
    if not 0 <= top <= LOGPROBS_MAX_TOP:
        _bad(f"top must be in [0, {LOGPROBS_MAX_TOP}]")
    like, device = tokens.shape, logits.device
    logprobs, ranks = _alike("logprobs", logprobs, like, _F32T, device), _alike("ranks", ranks, like, _I32T, device)
    entropy, lse = _alike("entropy", entropy, (rows,), _F32T, device), _alike("lse", lse, (rows,), _F32T, device)
    p = _ops._flats(dev, "tokens", tokens, _I32T, rows * n, "logprobs", logprobs, _F32T, rows * n, "ranks", ranks, _I32T,
                    rows * n, "entropy", entropy, _F32T, rows, "lse", lse, _F32T, rows)
    p_top = (0, 0)
    if top:
        top_ids = _alike("top_ids", top_ids, (rows, top), _I32T, device)
        top_logprobs = _alike("top_logprobs", top_logprobs, (rows, top), _F32T, device)
        p_top = _ops._flats(dev, "top_ids", top_ids, _I32T, rows * top, "top_logprobs", top_logprobs, _F32T, rows * top)
    elif top_ids is not None or top_logprobs is not None:
        _bad("top_ids and top_logprobs need top")
    p_parts = 0
    if lse_parts is not None:
        p_parts = _ops._flat("lse_parts", _alike("lse_parts", lse_parts, (rows, 2), _F32T, device), _F32T, 2 * rows, dev)
    _call(load().dflash_token_logprobs, _LOGPROBS.pack,
          (dt, rows, vocab, n, top, _inverse(temperature), ld, logits.data_ptr(), *p, *p_top, p_parts), dev)
    _ops._written(logprobs, ranks, entropy, lse, top_ids, top_logprobs, lse_parts)
    return TokenLogprobs(logprobs, ranks, entropy, lse, top_ids, top_logprobs)


def token_logprobs_grad(logits, tokens, lse, grad_logprobs, *, entropy=None, grad_entropy=None, temperature: float = 1.0,
                        out=None):
    """Gradient by the logits of a loss of ``token_logprobs``' results (``dflash_token_logprobs_grad``).

    logits, tokens, temperature: as given there; lse, entropy: as it gave them; lse may be its lse_parts [rows, 2], from
    which the probabilities of rows of any size are exact (lse's own last digit is a factor of exp(2^-24 |lse|), and of a row
    all of the type's lowest value it says nothing); grad_logprobs: fp32 of tokens' shape,
    the loss's gradient by each log probability (padding's does not count); grad_entropy: fp32 [rows] or None, by the
    entropies (needs entropy).  Returns ``out`` (of logits' type, allocated when None; ``out=logits`` works in place).
    For alternatives' log probabilities, name their ids among the tokens."""
    dev = _device(logits, logits, lse, grad_logprobs, entropy, grad_entropy, out)
    dt, rows, vocab, ld = _logits("logits", logits, dev)
    n = _tokens(tokens, rows)
    if grad_logprobs is None or grad_logprobs.shape != tokens.shape:
        _bad("grad_logprobs must have the shape of tokens")
    parts = lse.dim() == 2
    if parts and lse.shape != (rows, 2):
        _bad(f"lse must be [{rows}], or lse_parts [{rows}, 2]")
    p_tok, p_lse, p_g = _ops._flats(dev, "tokens", tokens, _I32T, rows * n, "lse", lse, _F32T, rows * 2 if parts else rows,
                                    "grad_logprobs", grad_logprobs, _F32T, rows * n)
    p_ent = p_h = 0
    if grad_entropy is not None:
        if entropy is None:
            _bad("grad_entropy needs entropy")
        p_ent, p_h = _ops._flats(dev, "entropy", entropy, _F32T, rows, "grad_entropy", grad_entropy, _F32T, rows)
    if out is None:
        out = torch.empty((rows, vocab), dtype=logits.dtype, device=logits.device)
    ld_out = max(_ops._mat("out", out, logits.dtype, rows, vocab, dev), vocab)
    _call(load().dflash_token_logprobs_grad, _GRAD.pack,
          (dt, rows, vocab, n, _inverse(temperature), 0, ld, ld_out, logits.data_ptr(), p_tok,
           0 if parts else p_lse, p_g, p_ent, p_h, out.data_ptr(), p_lse if parts else 0), dev)
    _ops._written(out)
    return out
