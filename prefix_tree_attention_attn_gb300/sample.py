"""The next token of every rollout from its logits and given random numbers
(``include/tree_sample.h``).  Marshalling only.

    tokens, logprobs = sample_tokens(logits, u, temperature=0.8, top_p=0.95)   # logits [R, V] bf16, u [R] fp32

``logprobs`` are those of the untempered softmax, the ones ``loss.traj_logprobs``
gives the same tokens in training.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _binding as B
from .decode import _check_dense, _current_device, _empty, _side, _stream_of

ERR_INVALID_SAMPLING = -15      # device status: a row's parameters are invalid (token -1)


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logprobs=None, stream=None):
    """(token [R] int32, log-prob [R] fp32) drawn from logits [R, V] bf16 with the
    uniform numbers u [R] fp32 in [0, 1).  Each parameter is one number, or a tensor
    with one per row (fp32; top_k int32); 0 for top_k and min_p and 1 for top_p switch
    a filter off, temperature 0 takes the largest logit (``tree_attn_sample``)."""
    dev = _current_device()
    if logits.dtype is not torch.bfloat16 or logits.dim() != 2 or logits.get_device() != dev:   # -1 on the CPU
        raise ValueError(f"logits: expected cuda:{dev} {torch.bfloat16} [rows, vocab], got {logits.device} "
                         f"{logits.dtype} {tuple(logits.shape)}")
    R, V = logits.shape
    stride = V
    if not logits.is_contiguous():
        step, one = logits.stride()
        stride = step if R > 1 else V
        if (one != 1 and V > 1) or stride < V:
            raise ValueError(f"logits: a row's entries must be contiguous, got strides {logits.stride()}")
    rows = (R,)
    _check_dense(u, "u", rows, torch.float32, dev)
    s = B.Sampling()
    if isinstance(temperature, torch.Tensor):
        _check_dense(temperature, "temperature", rows, torch.float32, dev)
        s.temperatures = temperature.data_ptr()
    else:
        s.temperature = temperature
    if isinstance(top_k, torch.Tensor):
        _check_dense(top_k, "top_k", rows, torch.int32, dev)
        s.top_ks = top_k.data_ptr()
    else:
        if not -2 ** 31 <= top_k < 2 ** 31:            # ctypes would cut it
            raise ValueError(f"top_k: {top_k} is not an int32")
        s.top_k = top_k
    if isinstance(top_p, torch.Tensor):
        _check_dense(top_p, "top_p", rows, torch.float32, dev)
        s.top_ps = top_p.data_ptr()
    else:
        s.top_p = top_p
    if isinstance(min_p, torch.Tensor):
        _check_dense(min_p, "min_p", rows, torch.float32, dev)
        s.min_ps = min_p.data_ptr()
    else:
        s.min_p = min_p
    side = _side(stream)
    if tokens is None:
        tokens = _empty(side, rows, torch.int32, logits.device)
    else:
        _check_dense(tokens, "tokens", rows, torch.int32, dev)
    if logprobs is None:
        logprobs = _empty(side, rows, torch.float32, logits.device)
    else:
        _check_dense(logprobs, "logprobs", rows, torch.float32, dev)
    st = B.load().tree_attn_sample(logits.data_ptr(), stride, R, V, u.data_ptr(), C.byref(s), tokens.data_ptr(),
                                   logprobs.data_ptr(), _stream_of(side, dev, logits, u, tokens, logprobs, temperature,
                                                                   top_k, top_p, min_p))
    if st:
        B.check(st, "tree_attn_sample")
    return tokens, logprobs
