"""The next token of every rollout from its logits and given random numbers
(``include/tree_sample.h``).  Marshalling only.

    tokens, logprobs = sample_tokens(logits, u, temperature=0.8, top_p=0.95)   # logits [R, V] bf16, u [R] fp32

``logprobs`` are those of the untempered softmax, the ones ``loss.traj_logprobs``
gives the same tokens in training.
"""
from __future__ import annotations

import ctypes as C

from . import _binding as B
from .decode import _check_vec, _stream_of

ERR_INVALID_SAMPLING = -15      # device status: a row's parameters are invalid (token -1)


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logprobs=None, stream=None):
    """(token [R] int32, log-prob [R] fp32) drawn from logits [R, V] bf16 with the
    uniform numbers u [R] fp32 in [0, 1).  Each parameter is one number, or a tensor
    with one per row (fp32; top_k int32); 0 for top_k and min_p and 1 for top_p switch
    a filter off, temperature 0 takes the largest logit (``tree_attn_sample``)."""
    import torch
    if not logits.is_cuda or logits.dtype != torch.bfloat16 or logits.dim() != 2:
        raise ValueError(f"logits: expected cuda {torch.bfloat16} [rows, vocab], got {logits.device} {logits.dtype} "
                         f"{tuple(logits.shape)}")
    dev = torch.cuda.current_device()
    if logits.get_device() != dev:
        raise ValueError(f"logits: on {logits.device}, the current device is cuda:{dev}")
    R, V = logits.shape
    stride = logits.stride(0) if R > 1 else V
    if (logits.stride(1) != 1 and V > 1) or stride < V:
        raise ValueError(f"logits: a row's entries must be contiguous, got strides {logits.stride()}")
    _check_vec(u, "u", R, torch.float32, dev)
    s = B.Sampling()
    for name, many, x, dtype in (("temperature", "temperatures", temperature, torch.float32),
                                 ("top_k", "top_ks", top_k, torch.int32), ("top_p", "top_ps", top_p, torch.float32),
                                 ("min_p", "min_ps", min_p, torch.float32)):
        if isinstance(x, torch.Tensor):
            _check_vec(x, name, R, dtype, dev)
            setattr(s, many, x.data_ptr())
        else:
            setattr(s, name, x)
    if tokens is None:
        tokens = torch.empty(R, dtype=torch.int32, device=logits.device)
    else:
        _check_vec(tokens, "tokens", R, torch.int32, dev)
    if logprobs is None:
        logprobs = torch.empty(R, dtype=torch.float32, device=logits.device)
    else:
        _check_vec(logprobs, "logprobs", R, torch.float32, dev)
    st = B.load().tree_attn_sample(logits.data_ptr(), stride, R, V, u.data_ptr(), C.byref(s), tokens.data_ptr(),
                                   logprobs.data_ptr(), _stream_of(stream, tokens, logprobs))
    if st:
        B.check(st, "tree_attn_sample")
    return tokens, logprobs
