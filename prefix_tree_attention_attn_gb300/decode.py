"""Growing a rollout tree (``include/tree_decode.h``): a key/value cache in 8
bits that stores every shared prefix once, and the attention of the decoding
nodes' new tokens over it.  Marshalling only.

    plan = DecodePlan(parent, seg_len, query_nodes, hq, hkv, d, capacity=room)   # host, C++ planner
    cache = TreeCache.empty(plan.n_pages, hkv, d)          # e4m3 pages of 64 tokens, a scale per page and kv-head
    lens = plan.lens()                                     # int32 [n_nodes], tokens per node
    tree_cache_write(plan, cache, k, v)                    # the fresh nodes' tokens, e.g. of a prefill
    tree_cache_append(plan, cache, lens, k1, v1)           # one new token per query, lens grows
    o, lse = tree_decode(plan, cache, lens, q, scale)      # q [R, hq, d] bf16

A plan stays valid while its nodes grow inside their capacity, so a whole
segment is decoded with one plan; branching makes a new plan over the same
pages.  Keep a plan while calls or captured graphs that use it run.

Calls on a ``stream`` other than the current one do not wait for the current
one: what they read has to be there (``stream.wait_stream``).
"""
from __future__ import annotations

import ctypes as C
from typing import Dict, Optional, Sequence

import numpy as np
import torch

from . import _i32, _ptr_i32
from . import _binding as B

PAGE = 64                       # tokens per page (TREE_DECODE_PAGE)
ERR_CACHE_FULL = -14            # device status: an append found no room


class DecodePlan:
    """Plan of the decode calls (``tree_attn_decode_plan``).

    ``seg_len[v]`` tokens are in node v, which has room for ``capacity[v]``
    (default: ``seg_len``); ``query_nodes[r]`` is the node that query r decodes
    in (-1: padding).  ``pages`` lists the nodes' pages by node id (default
    0, 1, ...), ``n_pages`` the pool's pages; ``fresh[v]`` says whether
    ``tree_cache_write`` brings node v's tokens (default: every node)."""

    def __init__(self, parent: Sequence[int], seg_len: Sequence[int], query_nodes: Sequence[int], hq: int, hkv: int,
                 d: int, capacity: Optional[Sequence[int]] = None, pages: Optional[Sequence[int]] = None,
                 n_pages: Optional[int] = None, fresh: Optional[Sequence[bool]] = None,
                 cta_pages: int = 0, warp_pages: int = 0):
        self._lib = B.load()
        self._h = None
        for name, x in (("hq", hq), ("hkv", hkv), ("d", d), ("n_pages", n_pages or 0), ("cta_pages", cta_pages),
                        ("warp_pages", warp_pages)):
            if not -2 ** 31 <= x < 2 ** 31:                # ctypes would cut it
                raise ValueError(f"{name}: {x} is not an int32")
        par, sl, qn = _i32(parent), _i32(seg_len), _i32(query_nodes)
        cap = sl if capacity is None else _i32(capacity)
        if par.ndim != 1 or sl.shape != par.shape or cap.shape != par.shape or qn.ndim != 1:
            raise ValueError("parent, seg_len and capacity must be 1-D arrays of equal length, query_nodes 1-D")
        need = int((np.maximum(cap, 0).astype(np.int64) + PAGE - 1).__floordiv__(PAGE).sum())
        pg = None if pages is None else _i32(pages)
        if pg is not None and pg.shape != (need,):
            raise ValueError(f"pages: {need} page numbers expected, got shape {pg.shape}")
        if n_pages is None:
            n_pages = need if pg is None else int(pg.max(initial=-1)) + 1
        fr = None if fresh is None else (np.asarray(fresh) != 0).astype(np.uint8)
        if fr is not None and fr.shape != par.shape:
            raise ValueError("fresh must have one entry per node")
        opts, h = B.DecodeOpts(cta_pages, warp_pages), C.c_void_p()
        B.check(self._lib.tree_attn_decode_plan(
            _ptr_i32(par), _ptr_i32(sl), _ptr_i32(cap), len(par), None if pg is None else _ptr_i32(pg), int(n_pages),
            None if fr is None else fr.ctypes.data_as(B.c_uint8_p), _ptr_i32(qn), len(qn), hq, hkv, d, C.byref(opts),
            C.byref(h)), "tree_attn_decode_plan")
        self._h = h
        self.seg_len, self.query_nodes = sl.copy(), qn.copy()   # the caller's arrays may change
        self.n_nodes, self.n_queries, self.n_pages = len(par), len(qn), int(n_pages)
        self.hq, self.hkv, self.d = hq, hkv, d
        inf = B.DecodeInfo()
        B.check(self._lib.tree_attn_decode_plan_info(h, C.byref(inf)), "tree_attn_decode_plan_info")
        self.info = {f: getattr(inf, f) for f, _ in B.DecodeInfo._fields_}
        self.workspace_bytes = int(inf.workspace_bytes)

    @property
    def handle(self):
        return self._h

    def lens(self, device=None):
        """The nodes' lengths at plan time as the device array the calls read."""
        return torch.from_numpy(self.seg_len.copy()).to(device or torch.device("cuda", torch.cuda.current_device()))

    def export(self) -> Dict[str, np.ndarray]:
        """Copies of the plan arrays (``tree_attn_decode_plan_export``)."""
        i = self.info
        sizes = {"entries": (i["n_entries"], 4), "items": (i["n_ctas"], 6, 8), "query_order": (i["n_live"],),
                 "combine_ptr": (i["n_live"] * i["n_sub"] + 1,), "combine_row": (i["n_combine"],),
                 "write_jobs": (i["n_write_jobs"], 4)}
        out, arr = {f: np.zeros(s, dtype=np.int32) for f, s in sizes.items()}, B.DecodeArrays()
        for f, a in out.items():
            setattr(arr, f, _ptr_i32(a))
        B.check(self._lib.tree_attn_decode_plan_export(self._h, C.byref(arr)), "tree_attn_decode_plan_export")
        return out

    def upload(self) -> None:
        B.check(self._lib.tree_attn_decode_plan_upload(self._h), "tree_attn_decode_plan_upload")

    def close(self) -> None:
        if self._h is not None:
            self._lib.tree_attn_decode_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TreeCache:
    """Pages of 64 tokens: ``k`` [n_pages, hkv, 64, d] and ``v`` [n_pages, hkv, d, 64]
    float8_e4m3fn, ``k_scale`` / ``v_scale`` [n_pages, hkv] fp32 powers of two."""

    def __init__(self, k, v, k_scale, v_scale):
        P, hkv, page, d = k.shape
        if page != PAGE:
            raise ValueError(f"k: pages of {PAGE} tokens expected, got shape {tuple(k.shape)}")
        for name, x, shape, dtype in (("k", k, (P, hkv, PAGE, d), torch.float8_e4m3fn),
                                      ("v", v, (P, hkv, d, PAGE), torch.float8_e4m3fn),
                                      ("k_scale", k_scale, (P, hkv), torch.float32),
                                      ("v_scale", v_scale, (P, hkv), torch.float32)):
            if not x.is_cuda or x.dtype != dtype or tuple(x.shape) != shape or not x.is_contiguous():
                raise ValueError(f"{name}: expected contiguous cuda {dtype} {shape}, got {x.device} {x.dtype} "
                                 f"{tuple(x.shape)}")
            if x.device != k.device:
                raise ValueError(f"{name}: on {x.device}, k on {k.device}")
        self._tensors = (k, v, k_scale, v_scale)
        self.n_pages, self.hkv, self.d, self.device = P, hkv, d, k.device

    # Read-only: a cache is checked once, other tensors are another TreeCache.
    k, v, k_scale, v_scale = (property(lambda self, i=i: self._tensors[i]) for i in range(4))

    @property
    def _ptrs(self):
        """The addresses of the moment: a program may free the tensors' storage and bring it back."""
        return [x.data_ptr() for x in self._tensors]

    @classmethod
    def empty(cls, n_pages: int, hkv: int, d: int, device=None) -> "TreeCache":
        dev = device or torch.device("cuda", torch.cuda.current_device())
        code = {"dtype": torch.float8_e4m3fn, "device": dev}
        real = {"dtype": torch.float32, "device": dev}
        return cls(torch.empty((n_pages, hkv, PAGE, d), **code), torch.empty((n_pages, hkv, d, PAGE), **code),
                   torch.empty((n_pages, hkv), **real), torch.empty((n_pages, hkv), **real))


# The calls below run once per token and layer: their checks read attributes only.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _check_cache(plan: DecodePlan, cache: TreeCache) -> int:
    """The call's device (the cache's, which must be the current one)."""
    if cache.n_pages < plan.n_pages or cache.hkv != plan.hkv or cache.d != plan.d:
        raise ValueError(f"cache: [{cache.n_pages}, {cache.hkv}, {PAGE}, {cache.d}] does not fit the plan's "
                         f"{plan.n_pages} pages of {plan.hkv} kv-heads of {plan.d}")
    dev = _current_device()
    if cache.device.index != dev:
        raise ValueError(f"cache: on {cache.device}, the current device is cuda:{dev}")
    return dev


def _expected(x, name: str, dtype, shape, dev: int, what: str = "contiguous ") -> ValueError:
    return ValueError(f"{name}: expected {what}cuda:{dev} {dtype} {tuple(shape)}, got {x.device} {x.dtype} "
                      f"{tuple(x.shape)} with strides {x.stride()}")


def _check_rows(x, name: str, rows: int, heads: int, d: int, dev: int) -> int:
    """Row stride of a bf16 [rows, heads, d] tensor whose rows are contiguous."""
    if x.dtype is not torch.bfloat16 or x.shape != (rows, heads, d) or x.get_device() != dev:   # -1 on the CPU
        raise _expected(x, name, torch.bfloat16, (rows, heads, d), dev, "")
    if x.is_contiguous():
        return heads * d
    s = x.stride()
    if s[2] != 1 or (s[1] != d and heads > 1):
        raise ValueError(f"{name}: heads and features must be contiguous in a row, got strides {s}")
    if rows == 1:
        return heads * d
    if s[0] < heads * d or s[0] % 8:
        raise ValueError(f"{name}: row stride {s[0]} must be a multiple of 8 and at least {heads * d}")
    return s[0]


def _check_dense(x, name: str, shape, dtype, dev: int) -> None:
    if x.dtype is not dtype or x.shape != shape or x.get_device() != dev or not x.is_contiguous():
        raise _expected(x, name, dtype, shape, dev)


def _side(stream):
    """`stream` where it is not the current one, else None."""
    return None if stream is None or stream == torch.cuda.current_stream() else stream


def _empty(side, shape, dtype, device):
    """A new tensor for a call on the stream `side`: out of that stream's pool, because work that
    the current stream still has for a block of its own pool is not waited for; kept, once freed,
    until the current stream, on which the caller has it, is done with it."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        x = torch.empty(shape, dtype=dtype, device=device)
    x.record_stream(torch.cuda.current_stream())
    return x


def _stream_of(side, dev: int, *used):
    """The stream's handle; the memory of what the call uses is kept until a side stream is done
    with it, whenever the caller lets go of it."""
    if side is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    for t in used:
        if isinstance(t, torch.Tensor):
            t.record_stream(side)
    return side.cuda_stream


def tree_cache_write(plan: DecodePlan, cache: TreeCache, k, v, stream=None) -> None:
    """Write the fresh nodes' tokens: k, v [n, hkv, d] bf16, rows in depth-first
    order (``tree_attn_cache_write``)."""
    dev = _check_cache(plan, cache)
    n = plan.info["n_fresh_tokens"]
    ks, vs = _check_rows(k, "k", n, plan.hkv, plan.d, dev), _check_rows(v, "v", n, plan.hkv, plan.d, dev)
    st = plan._lib.tree_attn_cache_write(plan._h, k.data_ptr(), v.data_ptr(), ks, vs, *cache._ptrs,
                                         _stream_of(_side(stream), dev, k, v, *cache._tensors))
    if st:
        B.check(st, "tree_attn_cache_write")


def tree_cache_append(plan: DecodePlan, cache: TreeCache, lens, k, v, lens_out=None, stream=None):
    """Append one token per query to its node: k, v [R, hkv, d] bf16.  Returns the
    lengths with the new tokens: ``lens_out``, by default ``lens`` itself
    (``tree_attn_cache_append``)."""
    dev = _check_cache(plan, cache)
    lens_out = lens if lens_out is None else lens_out
    _check_dense(lens, "lens", (plan.n_nodes,), torch.int32, dev)
    if lens_out is not lens:
        _check_dense(lens_out, "lens_out", (plan.n_nodes,), torch.int32, dev)
    ks = _check_rows(k, "k", plan.n_queries, plan.hkv, plan.d, dev)
    vs = _check_rows(v, "v", plan.n_queries, plan.hkv, plan.d, dev)
    st = plan._lib.tree_attn_cache_append(plan._h, lens.data_ptr(), lens_out.data_ptr(), k.data_ptr(), v.data_ptr(), ks,
                                          vs, *cache._ptrs,
                                          _stream_of(_side(stream), dev, lens, lens_out, k, v, *cache._tensors))
    if st:
        B.check(st, "tree_attn_cache_append")
    return lens_out


def tree_decode(plan: DecodePlan, cache: TreeCache, lens, q, softmax_scale: float, o=None, lse=None, workspace=None,
                stream=None):
    """O [R, hq, d] bf16 and LSE [hq, R] fp32 of one new token per query over the
    tokens of its node and the node's ancestors (``tree_attn_decode``).  Rows of
    padding queries are left as they were: pass ``o`` and ``lse`` to keep them."""
    dev = _check_cache(plan, cache)
    R, hq, d = plan.n_queries, plan.hq, plan.d
    _check_dense(lens, "lens", (plan.n_nodes,), torch.int32, dev)
    qs = _check_rows(q, "q", R, hq, d, dev)
    side = _side(stream)
    if o is None:
        o = _empty(side, (R, hq, d), torch.bfloat16, q.device)
    else:
        _check_dense(o, "o", (R, hq, d), torch.bfloat16, dev)
    if lse is None:
        lse = _empty(side, (hq, R), torch.float32, q.device)
    else:
        _check_dense(lse, "lse", (hq, R), torch.float32, dev)
    if workspace is None:
        workspace = _empty(side, (max(plan.workspace_bytes, 1),), torch.uint8, q.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected contiguous cuda:{dev} uint8, got {workspace.device} {workspace.dtype}")
    st = plan._lib.tree_attn_decode(plan._h, lens.data_ptr(), q.data_ptr(), qs, *cache._ptrs, o.data_ptr(),
                                    lse.data_ptr(), softmax_scale, workspace.data_ptr(), workspace.numel(),
                                    _stream_of(side, dev, lens, q, o, lse, workspace, *cache._tensors))
    if st:
        B.check(st, "tree_attn_decode")
    return o, lse
