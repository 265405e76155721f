"""Copies of cache pages: exact, in one cache and in several, and what they are for -- a branch inside a
page whose attention is that of the tokens it shares, and a compaction that changes no answer."""
import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import build as _build, device_status
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import decode as TD

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib, cuda_device):
    yield
    torch.cuda.synchronize()
    assert device_status() == 0


def pool(n, P, hkv, d, device, seed=0):
    """n caches with arbitrary bytes, one behind the other."""
    g = torch.Generator(device).manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device=device, dtype=torch.uint8).view(torch.float8_e4m3fn)  # noqa: E731
    real = lambda: torch.randn((n, P, hkv), generator=g, device=device)  # noqa: E731
    k, v, ks, vs = byte(n, P, hkv, 64, d), byte(n, P, hkv, d, 64), real(), real()
    return [TD.TreeCache(k[i], v[i], ks[i], vs[i]) for i in range(n)], [k.view(torch.uint8), v.view(torch.uint8), ks, vs]


@pytest.mark.parametrize("n,P,hkv,d", [(1, 5, 1, 64), (1, 40, 3, 64), (2, 9, 8, 128), (33, 6, 2, 128), (70, 4, 1, 64), (1, 3, 16, 128),
                                       (3, 4, 5, 64)])
def test_exact(cuda_device, n, P, hkv, d):
    rng = np.random.default_rng(P)
    caches, whole = pool(n, P, hkv, d, cuda_device)
    for m in {1, P // 2}:
        perm = rng.permutation(P)
        src, dst = perm[:m], perm[P - m:]
        if m == 1:
            dst = perm[1:3]
            src = np.repeat(src, 2)                         # one page to several
        want = [t.clone() for t in whole]
        for t in want:
            t[:, dst] = t[:, src]
        TD.tree_cache_copy(caches if n > 1 else caches[0], src, dst)
        assert all(torch.equal(a, b) for a, b in zip(whole, want))


def test_many_pages_and_nothing(cuda_device):
    caches, whole = pool(1, 5000, 1, 64, cuda_device)
    perm = np.random.default_rng(1).permutation(5000)
    want = [t.clone() for t in whole]
    TD.tree_cache_copy(caches, [], [])
    assert all(torch.equal(a, b) for a, b in zip(whole, want))
    for t in want:
        t[:, perm[2500:]] = t[:, perm[:2500]]
    TD.tree_cache_copy(caches, perm[:2500], perm[2500:])
    assert all(torch.equal(a, b) for a, b in zip(whole, want))
    with B.library(_build.build_library(debug=True)):
        TD.tree_cache_copy(caches, perm[:2500], perm[2500:])
        torch.cuda.synchronize()
        assert device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(whole, want))


def test_pages_behind_32_bit_offsets(cuda_device):
    """Pages whose codes lie beyond 2^32 bytes."""
    P, hkv, d = 70000, 8, 128                               # 4.6 GB of keys
    code = lambda *s: torch.empty(s, dtype=torch.float8_e4m3fn, device=cuda_device)  # noqa: E731
    cache = TD.TreeCache(code(P, hkv, 64, d), code(P, hkv, d, 64), torch.empty((P, hkv), device=cuda_device),
                         torch.empty((P, hkv), device=cuda_device))
    k, v = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    for page, x in ((3, 11), (69998, 22), (69999, 33), (2000, 44), (4464, 55), (4463, 66)):   # 69999 = 4463 + 65536
        k[page], v[page], cache.k_scale[page], cache.v_scale[page] = x, x + 1, x + 2.0, x + 3.0
    TD.tree_cache_copy(cache, [69998, 3], [2000, 69999])
    for page, x in ((3, 11), (69998, 22), (69999, 11), (2000, 22), (4464, 55), (4463, 66)):
        assert (k[page] == x).all() and (v[page] == x + 1).all() and (cache.k_scale[page] == x + 2).all() and (cache.v_scale[page] == x + 3).all()


def test_capture_and_side_stream(cuda_device):
    caches, whole = pool(3, 8, 2, 64, cuda_device)
    other, _ = pool(3, 8, 2, 64, cuda_device, 9)
    src, dst = np.array([1, 2, 3], np.int32), np.array([4, 5, 0], np.int32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in whole]
    for t in want:
        t[:, [4, 5, 0]] = t[:, [1, 2, 3]]
    torch.cuda.synchronize()
    TD.tree_cache_copy(caches, src, dst, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(whole, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        TD.tree_cache_copy(caches, src, dst)
    src[:], dst[:] = 0, 7                                   # the call has read them
    for c, o in zip(caches, other):
        for a, b in zip(c._tensors, o._tensors):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
    want = [t.clone() for t in whole]
    for t in want:
        t[:, [4, 5, 0]] = t[:, [1, 2, 3]]
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(whole, want))


@pytest.mark.parametrize("at", [1, 63, 64, 65, 100, 128])
def test_branch_inside_a_page(cuda_device, at):
    """A branch at token `at` of a node of 150: the new node's attention is that of the node cut there and
    written afresh to as many tokens; the old node answers as before."""
    hq, hkv, d, L = 8, 2, 64, 150
    g = torch.Generator(cuda_device).manual_seed(at)
    make = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    k, v, q = make(L, hkv, d), make(L, hkv, d), make(2, hq, d)
    P = TD.PagePool(8)
    cache = TD.TreeCache.empty(8, hkv, d, cuda_device)
    pages = P.alloc(3)
    plan = TD.DecodePlan([-1], [L], [0], hq, hkv, d, pages=pages, n_pages=8)
    TD.tree_cache_write(plan, cache, k, v)
    o0, lse0 = TD.tree_decode(plan, cache, plan.lens(), q[:1], 0.125)
    full, rest = at // 64, at % 64
    new = P.alloc(1)
    if rest:
        TD.tree_cache_copy(cache, pages[full:full + 1], new)
    # node 0: the full pages; 1: what the old node has behind them; 2: the branch
    tree = TD.DecodePlan([-1, 0, 0], [64 * full, L - 64 * full, rest], [1, 2], hq, hkv, d, capacity=[64 * full, L - 64 * full, 64],
                         pages=np.concatenate([pages, new]), n_pages=8)
    o, lse = TD.tree_decode(tree, cache, tree.lens(), q, 0.125)
    assert (o[0].float() - o0[0].float()).abs().max() <= 2.0 ** -7 * o0.float().abs().max()     # joined from other runs
    assert (lse[:, 0] - lse0[:, 0]).abs().max() <= 2.0 ** -14
    # the values that the cache holds, in 64 bits
    deq = lambda t, s: t.double() * s.double()[:, :, None, None]  # noqa: E731
    idx = torch.from_numpy(pages.astype(np.int64)).to(cuda_device)
    kk = deq(cache.k, cache.k_scale)[idx].permute(0, 2, 1, 3).reshape(-1, hkv, d)[:at]
    vv = deq(cache.v, cache.v_scale)[idx].permute(0, 3, 1, 2).reshape(-1, hkv, d)[:at]
    for h in range(hq):
        x = kk[:, h // 4] @ q[1, h].double() * 0.125
        want = torch.softmax(x, 0) @ vv[:, h // 4]
        # (o rounded once, weights to f16: 2^-8 of itself, 2^-11 of the values)
        assert ((o[1, h].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * vv.abs().max()).all()
        assert abs(float(lse[h, 1]) - float(torch.logsumexp(x, 0))) <= 2.0 ** -13
    # it grows on its own: the other node's answer stays
    lens = TD.tree_cache_append(TD.DecodePlan([-1, 0, 0], [64 * full, L - 64 * full, rest], [2], hq, hkv, d,
                                              capacity=[64 * full, L - 64 * full, 64], pages=np.concatenate([pages, new]), n_pages=8),
                                cache, tree.lens(), 50 * make(1, hkv, d), make(1, hkv, d))
    again, _ = TD.tree_decode(tree, cache, lens, q, 0.125)
    assert torch.equal(again[0], o[0]) and not torch.equal(again[1], o[1])


def test_compaction(cuda_device):
    """Half of the nodes go, the others' pages move down in two layers' caches: the same answers, bit by bit."""
    hq, hkv, d, n = 4, 1, 128, 20
    rng = np.random.default_rng(3)
    g = torch.Generator(cuda_device).manual_seed(3)
    make = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    seg = [200] + [int(x) for x in rng.integers(1, 200, n)]
    count = [-(-x // 64) for x in seg]
    P = TD.PagePool(100)
    mine = [P.alloc(c) for c in count]
    caches = [TD.TreeCache.empty(100, hkv, d, cuda_device) for _ in range(2)]
    parent = [-1] + [0] * n
    plan = TD.DecodePlan(parent, seg, range(1, n + 1), hq, hkv, d, pages=np.concatenate(mine), n_pages=100)
    for c in caches:
        TD.tree_cache_write(plan, c, make(sum(seg), hkv, d), make(sum(seg), hkv, d))
    q = make(n, hq, d)
    stay = list(range(2, n + 1, 2))
    for v in range(1, n + 1, 2):
        P.free(mine[v])
    keep = [0] + stay
    ask = lambda pages: TD.DecodePlan([-1] + [0] * len(stay), [seg[v] for v in keep], range(1, len(keep)), hq, hkv, d,  # noqa: E731
                                      pages=pages, n_pages=100)
    rows = torch.tensor([v - 1 for v in stay], device=cuda_device)
    before = ask(np.concatenate([mine[v] for v in keep]))
    want = [TD.tree_decode(before, c, before.lens(), q[rows], 0.1) for c in caches]
    src, dst, page = P.compact()
    assert len(src) > 0
    TD.tree_cache_copy(caches, src, dst)
    now = np.concatenate([page[mine[v]] for v in keep])
    assert sorted(now.tolist()) == list(range(len(now))) and P.n_free == 100 - len(now)
    after = ask(now)
    for c, w in zip(caches, want):
        c.k.view(torch.uint8)[len(now):] = 0x7f                        # NaN where pages came from
        got = TD.tree_decode(after, c, after.lens(), q[rows], 0.1)
        assert all(torch.equal(a, b) for a, b in zip(got, w))
