"""Linear attention over a packed rollout tree (``include/tree_linear.h``):
chunks of at most 128 tokens inside each node, the recurrent state carried
from every node into its children.  Marshalling only.

    o = tree_linear_fwd(plan, q, k, v, decay, scale)   # decay: fp32 [hkv] in (0, 1]
    dq, dk, dv = tree_linear_bwd(plan, q, k, v, do, decay, scale)

Growing a tree, from and to states in slots of a pool fp32 [n_slots, hkv, d, d]:

    slots = StateSlots([-1, -1, -1], [-1, 0, 1], n_slots)          # a prompt and two branches: their states kept
    o = tree_linear_prefill(plan, states, slots, q, k, v, decay, scale)
    fork = StateSlots([0, 0, 1], [3, 2, 1], n_slots)               # two branches go on from slot 0, one in its own
    o1 = tree_linear_step(states, fork, q1, k1, v1, decay, scale)  # one token per branch
"""
from __future__ import annotations

import ctypes as C

import numpy as np
import torch

from . import TreePlan, _check_tensor, _dptr, _i32, _stream_ptr
from . import _binding as B
from .decode import _check_dense, _check_rows, _current_device, _empty, _side, _stream_of

ERR_INVALID_SLOT = -16          # device status: a slot number outside the pool


def linear_workspace(plan: TreePlan, hkv: int, d: int):
    """(number of chunks, workspace bytes)."""
    nc, ws = C.c_int64(0), C.c_size_t(0)
    B.check(B.load().tree_attn_linear_workspace_size(plan.handle, hkv, d, C.byref(nc), C.byref(ws)),
            "tree_attn_linear_workspace_size")
    return int(nc.value), int(ws.value)


def tree_linear_fwd(plan: TreePlan, q, k, v, decay, scale: float, o=None, workspace=None, stream=None):
    """O [N, hq, d] bf16 = scale * sum over each token's path of gamma^(distance) (q.k) v."""
    import torch
    _, hq, d = q.shape
    hkv = k.shape[1]
    N = plan.n_tokens
    for name, t, shp in (("q", q, (N, hq, d)), ("k", k, (N, hkv, d)), ("v", v, (N, hkv, d))):
        _check_tensor(t, name, shp, torch.bfloat16)
    _check_tensor(decay, "decay", (hkv,), torch.float32)
    o = torch.empty_like(q) if o is None else o
    _check_tensor(o, "o", (N, hq, d), torch.bfloat16)
    _, need = linear_workspace(plan, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    B.check(B.load().tree_attn_linear_fwd(plan.handle, _dptr(q), _dptr(k), _dptr(v), _dptr(o), _dptr(decay), hq, hkv,
                                          d, scale, _dptr(workspace), workspace.numel(), _stream_ptr(stream)),
            "tree_attn_linear_fwd")
    return o


def tree_linear_bwd(plan: TreePlan, q, k, v, do, decay, scale: float, dq=None, dk=None, dv=None, workspace=None,
                    stream=None):
    """dQ [N, hq, d], dK / dV [N, hkv, d] bf16 for the compact output gradient dO."""
    import torch
    _, hq, d = q.shape
    hkv = k.shape[1]
    N = plan.n_tokens
    for name, t, shp in (("q", q, (N, hq, d)), ("k", k, (N, hkv, d)), ("v", v, (N, hkv, d)),
                         ("do", do, (N, hq, d))):
        _check_tensor(t, name, shp, torch.bfloat16)
    _check_tensor(decay, "decay", (hkv,), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t, shp in (("dq", dq, (N, hq, d)), ("dk", dk, (N, hkv, d)), ("dv", dv, (N, hkv, d))):
        _check_tensor(t, name, shp, torch.bfloat16)
    _, need = linear_workspace(plan, hkv, d)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    B.check(B.load().tree_attn_linear_bwd(plan.handle, _dptr(q), _dptr(k), _dptr(v), _dptr(do), _dptr(dq), _dptr(dk),
                                          _dptr(dv), _dptr(decay), hq, hkv, d, scale, _dptr(workspace),
                                          workspace.numel(), _stream_ptr(stream)),
            "tree_attn_linear_bwd")
    return dq, dk, dv


class StateSlots:
    """Which slot of a pool of ``n_slots`` states each branch (row of a step, node of a
    prefill) starts from and leaves its state in: ``slot_in`` (-1: a zero state) and
    ``slot_out`` (-1: not kept; in a step, a padding row).  The slots of ``slot_out`` are all
    different.  Checked and uploaded once, without waiting for what the device still has to do; call
    ``upload()`` before a stream capture, and keep the object as long as the graph is replayed."""

    _copies = {}                                           # a stream by device

    def __init__(self, slot_in, slot_out, n_slots: int):
        a, b = _i32(slot_in), _i32(slot_out)
        if a.ndim != 1 or a.shape != b.shape:
            raise ValueError("slot_in and slot_out must be 1-D arrays of equal length")
        if not 0 <= n_slots < 2 ** 31:
            raise ValueError(f"n_slots: {n_slots} is not a number of slots")
        for name, x in (("slot_in", a), ("slot_out", b)):
            if x.size and not (-1 <= x.min() and x.max() < n_slots):
                raise ValueError(f"{name}: numbers from -1 to {n_slots - 1} expected")
        kept = b[b >= 0]
        if np.unique(kept).size != kept.size:
            raise ValueError("slot_out: two states for one slot")
        self.slot_in, self.slot_out, self.n_slots = a.copy(), b.copy(), int(n_slots)
        # a row of a step may read the slot that it writes itself, not another's
        live = np.flatnonzero((a >= 0) & (b >= 0) & (a != b))
        self._rows_apart = not np.isin(a[live], kept).any()
        self._plan = None
        self._on, self._readers = {}, {}

    def __len__(self):
        return len(self.slot_in)

    def upload(self, device=None):
        """The tables on the device (int32, int32)."""
        dev = _current_device() if device is None else torch.device(device).index
        t = self._on.get(dev)
        if t is None:
            d = torch.device("cuda", dev)
            s = self._copies.get(dev)
            if s is None:
                s = self._copies[dev] = torch.cuda.Stream(d)
            with torch.cuda.stream(s):                     # its own: the copy alone is waited for, any stream may read next
                t = self._on[dev] = tuple(torch.from_numpy(np.stack([self.slot_in, self.slot_out])).to(d))
            self._readers[dev] = set()
        return t

    def _tables(self, dev: int, side):
        """The addresses of the tables, for a call on the current stream or on ``side``: their memory is kept until
        it has read them."""
        a, b = self.upload()
        s = torch._C._cuda_getCurrentRawStream(dev) if side is None else side.cuda_stream
        if s not in self._readers[dev] and len(self):
            a.record_stream(torch.cuda.current_stream() if side is None else side)   # (one memory: b's too)
            self._readers[dev].add(s)
        return a.data_ptr(), b.data_ptr()

    def _check_plan(self, plan: TreePlan) -> None:
        """No tree starts from a slot that another tree, or another root beside it, leaves a state in."""
        if self._plan is plan:
            return
        if len(self) != len(plan.parent):
            raise ValueError(f"slots: {len(plan.parent)} nodes expected, got {len(self)}")
        root = np.arange(len(plan.parent))
        for _ in range(len(root)):                         # pointers jump until they stand on roots
            up = np.where(plan.parent[root] < 0, root, root[np.maximum(plan.parent[root], 0)])
            if np.array_equal(up, root):
                break
            root = up
        readers = {}
        for u in np.flatnonzero(plan.parent < 0):
            if self.slot_in[u] >= 0:
                readers.setdefault(int(self.slot_in[u]), []).append(int(u))
        for v in np.flatnonzero(self.slot_out >= 0):
            r = readers.get(int(self.slot_out[v]), [])
            if r and r != [int(root[v])]:
                raise ValueError(f"slot {self.slot_out[v]}: node {v} leaves its state where another tree starts from")
        self._plan = plan


def _check_states(states, slots: StateSlots, hkv: int, d: int, dev: int) -> None:
    shape = states.shape
    if len(shape) != 4 or shape[0] < slots.n_slots:
        raise ValueError(f"states: at least {slots.n_slots} slots [{hkv}, {d}, {d}] expected, got {tuple(shape)}")
    _check_dense(states, "states", (shape[0], hkv, d, d), torch.float32, dev)


def prefill_workspace(plan: TreePlan, hkv: int, d: int) -> int:
    """Bytes of device workspace that ``tree_linear_prefill`` needs."""
    ws = C.c_size_t()
    B.check(B.load().tree_attn_linear_prefill_workspace_size(plan.handle, hkv, d, C.byref(ws)),
            "tree_attn_linear_prefill_workspace_size")
    return int(ws.value)


def tree_linear_prefill(plan: TreePlan, states, slots: StateSlots, q, k, v, decay, scale: float, o=None,
                        workspace=None, stream=None):
    """``tree_linear_fwd`` of fresh tokens that continue stored states: each root of the plan's
    tree or forest starts from the state in its slot of ``states`` [n_slots, hkv, d, d] fp32, nodes
    with a slot leave their last state there (``tree_attn_linear_prefill``).  d = 128."""
    dev = _current_device()
    N, hq, d = q.shape
    hkv = k.shape[1]
    N = plan.n_tokens
    for name, t, shp in (("q", q, (N, hq, d)), ("k", k, (N, hkv, d)), ("v", v, (N, hkv, d))):
        _check_dense(t, name, shp, torch.bfloat16, dev)
    _check_dense(decay, "decay", (hkv,), torch.float32, dev)
    _check_states(states, slots, hkv, d, dev)
    slots._check_plan(plan)
    side = _side(stream)
    if o is None:
        o = _empty(side, (N, hq, d), torch.bfloat16, q.device)
    else:
        _check_dense(o, "o", (N, hq, d), torch.bfloat16, dev)
    if workspace is None:
        workspace = _empty(side, (max(prefill_workspace(plan, hkv, d), 256),), torch.uint8, q.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous cuda:{dev} uint8, got {workspace.device} {workspace.dtype}")
    a, b = slots._tables(dev, side)
    st = B.load().tree_attn_linear_prefill(
        plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), states.data_ptr() or None, states.shape[0],
        a, b, decay.data_ptr(), hq, hkv, d, scale, workspace.data_ptr(), workspace.numel(),
        _stream_of(side, dev, q, k, v, o, states, decay, workspace))
    if st:
        B.check(st, "tree_attn_linear_prefill")
    return o


def tree_linear_step(states, slots: StateSlots, q, k, v, decay, scale: float, o=None, stream=None):
    """O [R, hq, d] bf16 of one token per branch: S = gamma S + k v^T, o = scale q^T S, from
    and to the slots of ``states`` [n_slots, hkv, d, d] fp32 (``tree_attn_linear_step``); q [R, hq, d], k and
    v [R, hkv, d] bf16, d 64 or 128.  Padding rows of ``o`` are left as they were: pass ``o`` to keep them."""
    dev = _current_device()
    R, hq, d = q.shape
    hkv = k.shape[1]
    if R != len(slots.slot_in):
        raise ValueError(f"q: {len(slots)} rows expected, got {R}")
    if not slots._rows_apart:
        raise ValueError("slots: a row starts from a slot that another row writes")
    qs, ks, vs = _check_rows(q, "q", R, hq, d, dev), _check_rows(k, "k", R, hkv, d, dev), _check_rows(v, "v", R, hkv, d, dev)
    _check_dense(decay, "decay", (hkv,), torch.float32, dev)
    _check_states(states, slots, hkv, d, dev)
    side = _side(stream)
    if o is None:
        o = _empty(side, (R, hq, d), torch.bfloat16, q.device)
    else:
        _check_dense(o, "o", (R, hq, d), torch.bfloat16, dev)
    a, b = slots._tables(dev, side)
    st = B.load().tree_attn_linear_step(
        states.data_ptr() or None, states.shape[0], a, b, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs,
        o.data_ptr(), decay.data_ptr(), R, hq, hkv, d, scale, _stream_of(side, dev, states, q, k, v, o, decay))
    if st:
        B.check(st, "tree_attn_linear_step")
    return o
