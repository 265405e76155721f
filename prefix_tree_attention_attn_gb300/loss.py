"""Loss-boundary calls (``include/tree_loss.h``): trajectory views of a plan,
per-token weights folded into a gradient, per-trajectory next-token log-probs
from compact logits, subtree (segment-level) advantages, and the clipped policy
loss with the gradient of the logits.  Marshalling only; the work runs in the
library's kernels.

    mult, pos = token_info(plan)                       # host, [N] each
    dO_w = scale_rows(dO, w)                           # y[t] = x[t] * w[t]
    lse, lp = traj_logprobs(plan, logits, tokens)      # logits [N, V] bf16
    adv, node_c, tok_c = subtree_advantage(plan, rewards, flags=NORM_STD)
    r = policy_loss(plan, logits, tokens, old_logprobs, adv, weights=w, kl_coef=0.04, ref_logprobs=ref)
    r.loss, r.dlogits                                  # loss fp32, dlogits [N, V] bf16
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional, Tuple

import numpy as np
import torch

from . import TreePlan, _check_tensor, _dptr, _stream_ptr
from . import _binding as B
from .decode import _check_dense, _current_device, _empty, _side, _stream_of

NORM_STD = 1
SIZE_WEIGHTED = 2
NO_ROOT = 4


def trajectory_info(plan: TreePlan) -> Tuple[int, int]:
    """(number of trajectories = leaves, total trajectory tokens)."""
    nl, ne = C.c_int32(0), C.c_int64(0)
    B.check(B.load().tree_attn_plan_trajectory_info(plan.handle, C.byref(nl), C.byref(ne)),
            "tree_attn_plan_trajectory_info")
    return int(nl.value), int(ne.value)


def trajectories(plan: TreePlan) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(leaf ids ascending, offsets [L+1], compact token of every trajectory position)."""
    nl, ne = trajectory_info(plan)
    leaves, ptr, tok = np.zeros(nl, np.int32), np.zeros(nl + 1, np.int64), np.zeros(max(ne, 1), np.int32)
    B.check(B.load().tree_attn_plan_trajectories(plan.handle, leaves.ctypes.data_as(B.c_int32_p),
                                                 ptr.ctypes.data_as(B.c_int64_p), tok.ctypes.data_as(B.c_int32_p)),
            "tree_attn_plan_trajectories")
    return leaves, ptr, tok[:ne]


def token_info(plan: TreePlan) -> Tuple[np.ndarray, np.ndarray]:
    """(multiplicity, position id) of every compact token, packed order."""
    N = plan.n_tokens
    mult, pos = np.zeros(N, np.int32), np.zeros(N, np.int32)
    B.check(B.load().tree_attn_plan_token_info(plan.handle, mult.ctypes.data_as(B.c_int32_p),
                                               pos.ctypes.data_as(B.c_int32_p)), "tree_attn_plan_token_info")
    return mult, pos


def scale_rows(x, w, out=None, stream=None):
    """out[t, ...] = x[t, ...] * w[t] (bf16 x / out, fp32 w; ``tree_attn_scale_rows``)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x: contiguous cuda bf16 expected")
    n = x.shape[0]
    _check_tensor(w, "w", (n,), torch.float32)
    out = torch.empty_like(x) if out is None else out
    _check_tensor(out, "out", tuple(x.shape), torch.bfloat16)
    row = x.numel() // max(n, 1)
    B.check(B.load().tree_attn_scale_rows(_dptr(x), _dptr(w), _dptr(out), n, row, _stream_ptr(stream)),
            "tree_attn_scale_rows")
    return out


def traj_logprobs(plan: TreePlan, logits, tokens, row_lse=None, out=None, stream=None):
    """(row logsumexp [N], next-token log-probs of every trajectory position
    [n_expanded - n_leaves]) from compact logits [N, V] bf16 and token ids [N] int32."""
    import torch
    N = plan.n_tokens
    V = logits.shape[1]
    _check_tensor(logits, "logits", (N, V), torch.bfloat16)
    _check_tensor(tokens, "tokens", (N,), torch.int32)
    nl, ne = trajectory_info(plan)
    row_lse = torch.empty(N, dtype=torch.float32, device=logits.device) if row_lse is None else row_lse
    out = torch.empty(ne - nl, dtype=torch.float32, device=logits.device) if out is None else out
    _check_tensor(row_lse, "row_lse", (N,), torch.float32)
    _check_tensor(out, "out", (ne - nl,), torch.float32)
    B.check(B.load().tree_attn_traj_logprobs(plan.handle, _dptr(logits), V, _dptr(tokens), _dptr(row_lse),
                                             _dptr(out) if out.numel() else None, _stream_ptr(stream)),
            "tree_attn_traj_logprobs")
    return row_lse, out


def subtree_advantage(plan: TreePlan, rewards, flags: int = 0, eps: float = 1e-6, stream=None):
    """(advantage of each trajectory, coefficient of each node by id, of each
    compact token) from per-trajectory rewards (leaves ascending id)."""
    import torch
    nl, _ = trajectory_info(plan)
    _check_tensor(rewards, "rewards", (nl,), torch.float32)
    dev = rewards.device
    adv = torch.empty(nl, dtype=torch.float32, device=dev)
    node_c = torch.empty(plan.info["n_nodes"], dtype=torch.float32, device=dev)
    tok_c = torch.empty(plan.n_tokens, dtype=torch.float32, device=dev)
    B.check(B.load().tree_attn_subtree_advantage(plan.handle, _dptr(rewards), flags, eps, _dptr(adv), _dptr(node_c),
                                                 _dptr(tok_c), _stream_ptr(stream)), "tree_attn_subtree_advantage")
    return adv, node_c, tok_c


class PolicyLoss(NamedTuple):
    loss: torch.Tensor                   # [] fp32
    logprobs: torch.Tensor               # [n_pred] fp32, 0 where a prediction has no weight
    entropy: torch.Tensor                # [N] fp32, 0 where a row has no weight
    dlogits: Optional[torch.Tensor]      # [N, V] bf16


def _check_matrix(x, name: str, rows: int, dev: int) -> int:
    """Row stride of a bf16 [rows, vocab] tensor whose rows are contiguous."""
    if x.dtype is not torch.bfloat16 or x.dim() != 2 or x.shape[0] != rows or x.get_device() != dev:   # -1 on the CPU
        raise ValueError(f"{name}: expected cuda:{dev} {torch.bfloat16} [{rows}, vocab], got {x.device} {x.dtype} "
                         f"{tuple(x.shape)}")
    V = x.shape[1]
    if x.is_contiguous():
        return V
    step, one = x.stride()
    if (one != 1 and V > 1) or (rows > 1 and step < V):
        raise ValueError(f"{name}: a row's entries must be contiguous, got strides {x.stride()}")
    return step if rows > 1 else V


def policy_workspace(plan: TreePlan) -> int:
    """Bytes of device workspace that ``policy_loss`` needs."""
    b = C.c_size_t()
    B.check(B.load().tree_attn_policy_loss_workspace(plan.handle, C.byref(b)), "tree_attn_policy_loss_workspace")
    return int(b.value)


def _policy_sizes(plan: TreePlan):
    """(trajectories, shape of the predictions, workspace bytes): a plan does not change, asked once."""
    sizes = getattr(plan, "_policy_sizes", None)
    if sizes is None:
        nl, ne = trajectory_info(plan)
        sizes = plan._policy_sizes = nl, (ne - nl,), policy_workspace(plan)
    return sizes


def policy_loss(plan: TreePlan, logits, tokens, old_logprobs, advantages, weights=None, ref_logprobs=None,
                per_token: bool = False, clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                entropy_coef: float = 0.0, grad: bool = True, grad_scale: float = 1.0, dlogits=None, workspace=None,
                stream=None) -> PolicyLoss:
    """Clipped policy loss of the trajectories' predictions, with its gradient for the
    compact logits [N, V] bf16 (``tree_attn_policy_loss``).

    Per prediction, in the order of ``traj_logprobs`` (n_pred = n_expanded - n_leaves):
    ``old_logprobs`` (None: a ratio of 1), ``weights`` (None: 1 / n_pred each; a prediction of
    weight 0 is left out) and ``ref_logprobs``; ``advantages`` per trajectory
    (``subtree_advantage``), or per prediction with ``per_token``.  ``dlogits`` may be the
    logits themselves (None: a new tensor, whose rows lie up to 7 elements further apart where the
    logits' are padded: both then lie alike in their 16 bytes, which is four times as fast).
    ``grad=False`` gives the loss, log-probs and entropies alone."""
    dev = _current_device()
    N = plan.n_tokens
    stride = _check_matrix(logits, "logits", N, dev)
    V = logits.shape[1]
    nl, n_pred, need = _policy_sizes(plan)
    _check_dense(tokens, "tokens", (N,), torch.int32, dev)
    _check_dense(advantages, "advantages", n_pred if per_token else (nl,), torch.float32, dev)
    s = B.Policy(None, advantages.data_ptr(), None, None, int(bool(per_token)), clip_low, clip_high, kl_coef,
                 entropy_coef, grad_scale)
    if old_logprobs is not None:
        _check_dense(old_logprobs, "old_logprobs", n_pred, torch.float32, dev)
        s.old_logprobs = old_logprobs.data_ptr()
    if weights is not None:
        _check_dense(weights, "weights", n_pred, torch.float32, dev)
        s.weights = weights.data_ptr()
    if ref_logprobs is not None:
        _check_dense(ref_logprobs, "ref_logprobs", n_pred, torch.float32, dev)
        s.ref_logprobs = ref_logprobs.data_ptr()
    elif kl_coef != 0:
        raise ValueError("ref_logprobs: needed for a kl_coef other than 0")
    side = _side(stream)
    if not grad:
        if dlogits is not None:
            raise ValueError("dlogits: given with grad=False")
        d_stride = 0
    elif dlogits is None:
        # a row starts where the logits' row starts in its 16 bytes: gradients then leave by whole vectors
        d_stride, at = V + (stride - V) % 8, logits.data_ptr() // 2 % 8
        if d_stride == V and at == 0:
            dlogits = _empty(side, (N, V), torch.bfloat16, logits.device)
        else:
            dlogits = _empty(side, (N * d_stride + at,), torch.bfloat16, logits.device).as_strided((N, V), (d_stride, 1), at)
    else:
        d_stride = _check_matrix(dlogits, "dlogits", N, dev)
        if dlogits.shape != logits.shape:
            raise ValueError(f"dlogits: expected {tuple(logits.shape)}, got {tuple(dlogits.shape)}")
    if workspace is None:
        workspace = _empty(side, (need,), torch.uint8, logits.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous cuda:{dev} uint8, got {workspace.device} {workspace.dtype}")
    f32 = (torch.float32, logits.device)
    loss, logprobs, entropy = _empty(side, (), *f32), _empty(side, n_pred, *f32), _empty(side, (N,), *f32)
    st = B.load().tree_attn_policy_loss(
        plan.handle, logits.data_ptr(), stride, V, tokens.data_ptr(), C.byref(s), loss.data_ptr(),
        logprobs.data_ptr() or None, entropy.data_ptr(), dlogits.data_ptr() if grad else None, d_stride,
        workspace.data_ptr(), workspace.numel(),
        _stream_of(side, dev, logits, tokens, old_logprobs, advantages, weights, ref_logprobs, dlogits, workspace, loss,
                   logprobs, entropy))
    if st:
        B.check(st, "tree_attn_policy_loss")
    return PolicyLoss(loss, logprobs, entropy, dlogits)
