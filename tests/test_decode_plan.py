"""The decode planner on the host: every page of a query's path is covered once, the
tables stay in range, and bad arguments are refused (CPU only)."""
import ctypes as C

import numpy as np
import pytest

from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300.decode import PAGE, DecodePlan
from workloads import trees as WT


def random_case(rng):
    n = int(rng.integers(1, 14))
    t = WT.random_tree(rng, n, [1, 2, 63, 64, 65, 130, 300], n_roots=int(rng.integers(1, min(n, 3) + 1)))
    seg = [0 if rng.random() < 0.15 else x for x in t.seg_len]
    cap = [x + int(rng.choice([0, 0, 1, 64, 100])) for x in seg]
    need = sum(-(-c // PAGE) for c in cap)
    pool = need + int(rng.integers(0, 5))
    pages = rng.permutation(pool)[:need]
    queries = [int(x) for x in rng.integers(-1, n, size=int(rng.integers(1, 12)))]
    group = int(rng.choice([1, 2, 5, 8, 64, 65, 130, 200]))
    return t.parent, seg, cap, pages, pool, queries, group


@pytest.mark.parametrize("seed", range(60))
def test_items_cover_every_path_once(lib, seed):
    rng = np.random.default_rng(seed)
    parent, seg, cap, pages, pool, queries, group = random_case(rng)
    cta, warp = int(rng.choice([0, 1, 3, 128])), int(rng.choice([0, 1, 2, 32]))
    fresh = rng.random(len(parent)) < 0.7
    p = DecodePlan(parent, seg, queries, 2 * group, 2, 64, capacity=cap, pages=pages, n_pages=pool, fresh=fresh,
                   cta_pages=cta, warp_pages=warp)
    x, info = p.export(), p.info
    first = np.concatenate([[0], np.cumsum([-(-c // PAGE) for c in cap])])
    live = [r for r, u in enumerate(queries) if u >= 0]
    assert sorted(x["query_order"]) == live
    sub, rows = info["n_sub"], info["rows_per_sub"]
    assert rows <= 128 and (sub - 1) * rows < group <= sub * rows
    # a page entry names its node, its first token and the room behind it
    for page, node, at, room in x["entries"]:
        assert (room >> 16 == 1) == (at < seg[node])
        room &= 0xFFFF
        assert at % PAGE == 0 and 0 < room <= PAGE and room == min(PAGE, cap[node] - at)
        assert pages[first[node] + at // PAGE] == page
    seen = {}
    part_rows = []
    items = []
    for slots in x["items"]:
        assert slots[0][1] > 0 and all(not y[1] or y[5] == slots[0][5] for y in slots)
        assert not slots[0][5] or not slots[1:, 1].any()               # a CTA's item is alone
        items += [y for y in slots if y[1]]
    for e0, n, g0, g1, part, wide, _, _ in items:
        assert 0 <= e0 and 0 < n and e0 + n <= info["n_entries"] and 0 <= g0 < g1 <= len(live) * sub
        assert (g1 - g0) * rows <= (128 if wide else 8)
        assert n <= ((cta or 128) if wide else (warp or 32))
        for g in range(g0, g1):
            for e in range(e0, e0 + n):
                key = (g, int(x["entries"][e][0]))
                assert key not in seen
                seen[key] = True
        part_rows.append((part, part + (g1 - g0) * rows))
    # partial rows: disjoint and all inside the workspace
    part_rows.sort()
    assert all(a[1] <= b[0] for a, b in zip(part_rows, part_rows[1:]))
    assert not part_rows or part_rows[-1][1] <= info["n_part_rows"]
    assert info["workspace_bytes"] >= info["n_part_rows"] * 2 * (64 + 2) * 4
    want = set()
    for s, r in enumerate(x["query_order"]):
        u = queries[r]
        while u >= 0:
            for pg in pages[first[u]:first[u + 1]]:
                want |= {(s * sub + j, int(pg)) for j in range(sub)}
            u = parent[u]
    assert set(seen) == want
    # every row group finds its items' partial rows
    items_of = {g: [] for g in range(len(live) * sub)}
    for _, _, g0, g1, part, _, _, _ in items:
        for g in range(g0, g1):
            items_of[g].append(part + (g - g0) * rows)
    for g, parts in items_of.items():
        assert sorted(x["combine_row"][x["combine_ptr"][g]:x["combine_ptr"][g + 1]]) == sorted(parts)
    # write jobs: the fresh nodes' tokens in depth-first order
    kids = {v: [c for c in range(len(parent)) if parent[c] == v] for v in range(-1, len(parent))}
    order, stack = [], list(reversed(kids[-1]))
    while stack:
        v = stack.pop()
        order.append(v)
        stack.extend(reversed(kids[v]))
    want_jobs, row = [], 0
    for v in order:
        if fresh[v]:
            for t in range(0, seg[v], PAGE):
                n = min(PAGE, seg[v] - t)
                want_jobs.append([pages[first[v] + t // PAGE], row, n, 0])
                row += n
    assert x["write_jobs"].tolist() == want_jobs and info["n_fresh_tokens"] == row


def test_shared_prefix_is_one_run(lib):
    """A prompt under 8 siblings is in one item, not one per sibling; a chain that one
    query reads is one run."""
    p = DecodePlan([-1] + [0] * 8, [256] + [64] * 8, range(1, 9), 16, 1, 128, cta_pages=128, warp_pages=32)
    x = p.export()["items"].reshape(-1, 8)
    assert sorted(x[x[:, 1] > 0][:, 1].tolist()) == [1] * 8 + [4] and p.info["n_entries"] == 4 + 8
    c = DecodePlan([-1, 0, 1, 2], [64, 64, 64, 10], [3], 8, 1, 128, warp_pages=32)
    x = c.export()["items"].reshape(-1, 8)
    assert x[x[:, 1] > 0][:, 1].tolist() == [4] and c.info["n_part_rows"] == 8


def status(lib, parent, seg, queries, hq=2, hkv=1, d=64, cap=None, pages=None, n_pages=None, cta=0, warp=0):
    a = lambda x: None if x is None else np.asarray(x, np.int32).ctypes.data_as(B.c_int32_p)  # noqa: E731
    keep = [np.asarray(x, np.int32) if x is not None else None for x in (parent, seg, cap, pages, queries)]
    ptr = [None if x is None else x.ctypes.data_as(B.c_int32_p) for x in keep]
    h = C.c_void_p()
    pool = 1000 if n_pages is None else n_pages
    st = lib.tree_attn_decode_plan(ptr[0], ptr[1], ptr[2], len(parent), ptr[3], pool, None, ptr[4], len(queries), hq, hkv,
                                   d, C.byref(B.DecodeOpts(cta, warp)), C.byref(h))
    assert (st == 0) == bool(h.value)
    lib.tree_attn_decode_plan_destroy(h)
    return st


def test_plan_refusals(lib):
    ok = dict(parent=[-1, 0], seg=[100, 3], queries=[1])
    assert status(lib, **ok) == 0
    assert status(lib, **{**ok, "seg": [0, 0]}) == 0                        # nodes may be empty
    for bad in ([0, 0], [-1, 2], [-1, -2], [1, 0]):
        assert status(lib, **{**ok, "parent": bad}) == -2
    assert status(lib, [-1, 2, 1], [1, 1, 1], [0]) == -2                    # a cycle beside a root
    assert status(lib, **{**ok, "seg": [100, -1]}) == -2
    assert status(lib, **ok, cap=[100, 2]) == -2                            # room below the tokens
    for q in ([2], [-2]):
        assert status(lib, **{**ok, "queries": q}) == -1
    assert status(lib, [], [], [0]) == -1 and status(lib, [-1], [1], []) == -1
    assert status(lib, **ok, pages=[0, 1, 1]) == -1                         # a page twice
    assert status(lib, **ok, pages=[0, 1, 7], n_pages=7) == -1              # behind the pool
    assert status(lib, **ok, pages=[0, 1, -1]) == -1
    assert status(lib, **ok, n_pages=2) == -1                               # three are needed
    assert status(lib, **ok, n_pages=3) == 0
    for kw in ({"cta": -1}, {"cta": 129}, {"warp": -1}, {"warp": 33}):
        assert status(lib, **ok, **kw) == -1
    for hq, hkv, d in ((3, 2, 64), (0, 1, 64), (2, 0, 64), (2, 1, 96), (2, 1, 256)):
        assert status(lib, **ok, hq=hq, hkv=hkv, d=d) == -4
    assert status(lib, **ok, hkv=2, n_pages=2 ** 31 - 1) == -3              # page rows pass 31 bits
    assert status(lib, [-1, 0], [2 ** 31 - 1, 2 ** 31 - 1], [1]) != 0
    assert lib.tree_attn_decode_plan(None, None, None, 1, None, 1, None, None, 1, 1, 1, 64, None, None) == -1
    assert lib.tree_attn_decode_plan_info(None, None) == -1 and lib.tree_attn_decode_plan_export(None, None) == -1
    assert lib.tree_attn_decode_plan_upload(None) == -1
    lib.tree_attn_decode_plan_destroy(None)
    assert lib.tree_attn_strerror(-14).decode() == "a token was appended to a node without room"
    with pytest.raises(ValueError):
        DecodePlan([-1, 0], [100, 3], [1], 2, 1, 64, pages=[0, 1])          # three pages are needed
    with pytest.raises(ValueError):
        DecodePlan([-1, 0], [100], [1], 2, 1, 64)
    with pytest.raises(ValueError):
        DecodePlan([-1, 0], [100, 3], [1], 2, 1, 64, fresh=[True])


def test_calls_validate_before_touching_the_device(lib):
    p = DecodePlan([-1, 0, 0], [100, 60, 60], [1, 2], 4, 2, 128)
    f, odd = C.c_void_p(0x1000), C.c_void_p(0x1008)
    w = lib.tree_attn_cache_write
    assert w(None, f, f, 256, 256, f, f, f, f, None) == -1
    assert w(p.handle, None, f, 256, 256, f, f, f, f, None) == -1
    assert w(p.handle, f, f, 248, 256, f, f, f, f, None) == -1              # rows overlap
    assert w(p.handle, f, f, 256, 260, f, f, f, f, None) == -1              # not a multiple of 8
    assert w(p.handle, odd, f, 256, 256, f, f, f, f, None) == -5
    assert w(p.handle, f, f, 256, 256, f, f, f, C.c_void_p(0x1001), None) == -5
    a = lib.tree_attn_cache_append
    assert a(p.handle, None, f, f, f, 256, 256, f, f, f, f, None) == -1
    assert a(p.handle, f, f, f, f, 128, 256, f, f, f, f, None) == -1
    assert a(p.handle, f, f, f, odd, 256, 256, f, f, f, f, None) == -5
    twice = DecodePlan([-1, 0], [100, 60], [1, 1], 4, 2, 128)
    assert a(twice.handle, f, f, f, f, 256, 256, f, f, f, f, None) == -1    # one node, two tokens
    dec = lib.tree_attn_decode
    big = 1 << 30
    assert p.workspace_bytes > 0
    assert dec(p.handle, f, None, 512, f, f, f, f, f, f, 1.0, f, big, None) == -1
    assert dec(p.handle, f, f, 504, f, f, f, f, f, f, 1.0, f, big, None) == -1
    assert dec(p.handle, f, f, 516, f, f, f, f, f, f, 1.0, f, big, None) == -1
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert dec(p.handle, f, f, 512, f, f, f, f, f, f, scale, f, big, None) == -1
    assert dec(p.handle, f, odd, 512, f, f, f, f, f, f, 1.0, f, big, None) == -5
    assert dec(p.handle, f, f, 512, f, f, f, f, f, f, 1.0, None, big, None) == -6
    assert dec(p.handle, f, f, 512, f, f, f, f, f, f, 1.0, f, 16, None) == -6
    assert dec(p.handle, f, f, 512, f, f, f, f, f, f, 1.0, C.c_void_p(0x1080), big, None) == -5


def test_encode_is_the_format(lib):
    """The oracle's codes against the framework's e4m3 type, and its page scales."""
    import torch
    from oracle import decode as OD
    rng = np.random.default_rng(5)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-14, 10, 4000), OD.VALUES[:127],
                        (OD.VALUES[:126] + OD.VALUES[1:127]) / 2, [0.0, -0.0, 2.0 ** -10, 2.0 ** -11]])
    x = np.clip(x.astype(np.float32), -448, 448)
    assert np.array_equal(OD.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert OD.encode([1e9, -np.inf]).tolist() == [126, 254] and OD.encode([np.nan])[0] & 127 == 127
    assert OD.page_exp([448.0]) == 0 and OD.page_exp([448.1]) == 1 and OD.page_exp([0.0]) == -100
    assert OD.page_exp([np.inf, 3.5, np.nan]) == -7


def test_a_pool_of_no_pages_is_taken(lib):
    """A tree whose nodes have no room at all: its plan has no pages, no items and no workspace,
    and its calls are not refused for a pool without an address (here: for want of a device)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would be made")
    p = DecodePlan([-1, 0], [0, 0], [1, -1, 0], 4, 2, 128)
    assert p.n_pages == 0 and p.info["n_ctas"] == 0 and p.workspace_bytes == 0
    f = C.c_void_p(0x1000)
    assert lib.tree_attn_decode(p.handle, f, f, 512, None, None, None, None, f, f, 1.0, None, 0, None) == -8
    one = DecodePlan([-1, 0], [0, 0], [1, 0], 4, 2, 128)
    assert lib.tree_attn_cache_append(one.handle, f, f, f, f, 256, 256, None, None, None, None, None) == -8
    assert lib.tree_attn_cache_append(one.handle, f, f, f, None, 256, 256, None, None, None, None, None) == -1
    some = DecodePlan([-1, 0], [0, 0], [1, 0], 4, 2, 128, n_pages=1)
    assert lib.tree_attn_cache_append(some.handle, f, f, f, f, 256, 256, None, None, None, None, None) == -1


def test_values_that_are_no_int32_are_refused(lib):
    """Nothing is cut to 32 bits or to an integer on the way to the planner."""
    ok = dict(parent=[-1, 0], seg_len=[100, 3], query_nodes=[1], hq=2, hkv=1, d=64)
    big = np.array([2 ** 32 + 1], np.int64)
    for kw in ({"seg_len": np.concatenate([100 + 0 * big, big])}, {"parent": np.concatenate([big - 2 ** 33, 0 * big])},
               {"query_nodes": big}, {"query_nodes": [1.5]}, {"query_nodes": [float("nan")]},
               {"capacity": np.concatenate([big + 100, big])}, {"pages": np.array([2 ** 32, 1, 2])}, {"hq": 2 ** 32 + 2},
               {"hkv": 2 ** 32 + 1}, {"d": 2 ** 32 + 64}, {"n_pages": 2 ** 32 + 9}, {"cta_pages": 2 ** 32 + 3},
               {"warp_pages": 2 ** 32 + 3}):
        with pytest.raises((ValueError, OverflowError)):
            DecodePlan(**{**ok, **kw})
    p = DecodePlan(**{**ok, "parent": np.array([-1, 0], np.int64), "query_nodes": (np.int64(1),), "fresh": np.array([256, 0])})
    assert p.info["n_fresh_tokens"] == 100


def test_a_plan_keeps_its_own_lengths(lib):
    """plan.lens() gives the lengths at plan time, whatever becomes of the arrays given."""
    seg, queries = np.array([100, 3], np.int32), np.array([1], np.int32)
    p = DecodePlan(np.array([-1, 0], np.int32), seg, queries, 2, 1, 64, capacity=[100, 60])
    seg += 7
    queries[0] = 0
    assert p.lens("cpu").tolist() == [100, 3] and p.query_nodes.tolist() == [1]
