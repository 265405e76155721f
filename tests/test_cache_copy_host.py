"""Page pools, and refusals of the page copy, on the host (CPU only; nothing is launched)."""
import ctypes as C

import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import decode as TD


def test_pool():
    p = TD.PagePool(10)
    a, b = p.alloc(4), p.alloc(3)
    assert a.tolist() == [0, 1, 2, 3] and b.tolist() == [4, 5, 6] and p.n_free == 3 and a.dtype == np.int32
    with pytest.raises(MemoryError):
        p.alloc(4)
    with pytest.raises(MemoryError):
        p.alloc(-1)
    assert p.n_free == 3 and p.alloc(0).size == 0
    p.free(a[1:3])
    for bad in ([1], [9], [-1], [10], [4, 4], [4, 1]):
        with pytest.raises(ValueError):
            p.free(bad)
    assert p.n_free == 5
    src, dst, page = p.compact()
    assert src.tolist() == [5, 6] and dst.tolist() == [1, 2] and page.tolist() == [0, 1, 2, 3, 4, 1, 2, 7, 8, 9]
    assert not set(src) & set(dst) and p.alloc(1).tolist() == [5]
    src, dst, page = p.compact()
    assert src.size == dst.size == 0 and page.tolist() == list(range(10))
    assert TD.PagePool(0).alloc(0).size == 0
    for bad in (-1, 2 ** 31):
        with pytest.raises(ValueError):
            TD.PagePool(bad)


def test_random_compactions():
    rng = np.random.default_rng(0)
    for _ in range(50):
        P = int(rng.integers(1, 60))
        p = TD.PagePool(P)
        p.alloc(P)
        gone = rng.permutation(P)[:rng.integers(0, P + 1)].astype(np.int32)
        p.free(gone)
        used = np.setdiff1d(np.arange(P), gone)
        src, dst, page = p.compact()
        assert sorted(page[used].tolist()) == list(range(len(used))) and not set(src) & set(dst)
        moved = dict(zip(src.tolist(), dst.tolist()))
        assert all(page[u] == moved.get(u, u) for u in used.tolist())


def test_bad_arguments(lib):
    fake = [0x1000, 0x2000]

    def status(n=2, k=fake, v=fake, ks=fake, vs=fake, pages=10, hkv=2, d=64, src=(0, 1), dst=(2, 3), m=None):
        arr = lambda x: None if x is None else (C.c_void_p * len(x))(*x)  # noqa: E731
        keep = [np.asarray(x, np.int32) if x is not None else None for x in (src, dst)]
        ptr = [None if x is None else x.ctypes.data for x in keep]
        return lib.tree_attn_cache_copy(n, arr(k), arr(v), arr(ks), arr(vs), pages, hkv, d, *ptr, len(src or ()) if m is None else m, None)

    for name in ("k", "v", "ks", "vs"):
        assert status(**{name: None}) == -1 and status(**{name: [0x1000, None]}) == -1
    assert status(src=None, m=2) == -1 and status(dst=None) == -1
    assert status(n=-1) == -1 and status(m=-1) == -1 and status(pages=-1) == -1 and status(hkv=0) == -1
    assert status(d=32) == -4 and status(hkv=2 ** 30) == -3
    assert status(k=[0x1000, 0x1008]) == -5 and status(v=[0x1004, 0x1000]) == -5 and status(ks=[0x1000, 0x1002]) == -5
    for src, dst in (((0, 1), (2, 2)), ((0, 1), (1, 2)), ((0, 1), (2, 0)), ((0,), (0,)), ((-1,), (2,)), ((0,), (-1,)), ((10,), (2,)),
                     ((0,), (10,))):
        assert status(src=src, dst=dst) == -1, (src, dst)
    assert status(src=tuple(range(11)), dst=tuple(range(11, 22)), pages=10) == -1
    assert status(m=0) == 0 and status(n=0) == 0 and status(m=0, k=None, src=None) == 0


def test_binding(lib, monkeypatch):
    monkeypatch.setattr(TD, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="none given"):
        TD.tree_cache_copy([], [0], [1])

    class Fake(TD.TreeCache):
        def __init__(self, P, hkv=1, d=64, index=0):
            self.n_pages, self.hkv, self.d, self.device, self._tensors = P, hkv, d, torch.device("cuda", index), ()
            self._shape = (P, hkv, d, index)

    with pytest.raises(ValueError, match="beside"):
        TD.tree_cache_copy([Fake(4), Fake(5)], [0], [1])
    with pytest.raises(ValueError, match="beside"):
        TD.tree_cache_copy([Fake(4), Fake(4, index=1)], [0], [1])
    with pytest.raises(ValueError, match="current device"):
        TD.tree_cache_copy([Fake(4, index=1), Fake(4, index=1)], [0], [1])
    for src, dst in (([0], [1, 2]), ([[0]], [[1]]), ([0.5], [1]), ([2 ** 31], [1])):
        with pytest.raises(ValueError):
            TD.tree_cache_copy(Fake(4), src, dst)


@pytest.mark.parametrize("pages", [2000, 10 ** 6])
def test_moves_that_meet(lib, pages):
    """Refusals in small and in large pools, which check the moves in different ways."""
    def status(src, dst):
        one = (C.c_void_p * 1)(0x1000)
        a, b = np.asarray(src, np.int32), np.asarray(dst, np.int32)
        return lib.tree_attn_cache_copy(1, one, one, one, one, pages, 1, 64, a.ctypes.data, b.ctypes.data, len(a), None)

    many, top = list(range(100)), pages - 1
    assert status(many, [1000 + i for i in many[:99]] + [1098]) == -1
    assert status(many, [1000 + i for i in many[:99]] + [50]) == -1
    assert status([5, 5, 6], [7, 8, 7]) == -1 and status([5, 5, 6], [7, 8, 5]) == -1 and status([top], [top]) == -1
    assert status([top + 1], [0]) == -1 and status([top], [-1]) == -1
