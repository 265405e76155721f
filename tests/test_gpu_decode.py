"""The 8-bit tree cache and its single-token attention on the GPU, against the fp64
reference.  Codes, scales and lengths are compared bit for bit.

Error bounds of the attention, per element (derived, not fitted).  With
A = sum_j p_j |v_j| and X = max_j scale * sum_f |q_f k_jf|:
  * bf16 output: half a step, 2^-8 relative to the value (2^-9 plus the next terms);
  * P rounded to f16: 2^-11 of A (half a step of 11 bits);
  * P below f16's normal numbers: the weights are lifted so that the largest
    p_j s_j (s_j the page's scale, the weight of j's codes) is at least 2^12, f16's
    subnormals are multiples of 2^-24, so rounding them moves a weight by at most 2^-25,
    that is 2^-37 of the largest; times the codes: 2^-37 * max_j(p_j s_j) * sum_j |v_j / s_j|;
  * the query row in f16 after a power of two: exact but for features below 2^-14 of
    the row's largest, which lose 2^-25 of it: 2^-25 * d * X' inside the fp32 bound;
  * logits in fp32: products are exact, d / 16 accumulations that may truncate, and the
    scaling: 2^-18 * X is above (d / 8 + 8) * 2^-23 * 2 * X; a logit's error e changes
    p by a factor within 1 +- 2e, numerator and denominator: 4 e A;
  * 2^x and the sums over keys and partial rows: 2^-20 relative, 2^-13 of A covers
    them for up to 2^7 pages a chunk.
The log-sum-exp: 2^-18 * X + 2^-20 * (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from oracle import decode as OD
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import build as _build
from prefix_tree_attention_attn_gb300 import device_status
from prefix_tree_attention_attn_gb300 import decode as TD
from workloads import trees as WT

pytestmark = pytest.mark.gpu

POISON = 0x7F        # an e4m3 NaN


def cache_pair(P, hkv, d, dev, fill=POISON):
    """A device cache whose every byte is `fill` and every scale NaN, and its copy."""
    c = TD.TreeCache.empty(P, hkv, d, dev)
    for x in (c.k, c.v):
        x.view(torch.uint8).fill_(fill)
    c.k_scale.fill_(float("nan"))
    c.v_scale.fill_(float("nan"))
    return c, host_cache(c)


def host_cache(c):
    return OD.Cache(c.k.view(torch.uint8).cpu().numpy(), c.v.view(torch.uint8).cpu().numpy(), c.k_scale.cpu().numpy(),
                    c.v_scale.cpu().numpy())


def assert_same_cache(c, ref):
    """Bit for bit, untouched bytes included.  The sign of a NaN code is free."""
    got = host_cache(c)
    for n in ("k8", "v8"):
        a, b = getattr(got, n), getattr(ref, n)
        nan = ((a & 127) == 127) & ((b & 127) == 127)
        assert np.array_equal(np.where(nan, 127, a), np.where(nan, 127, b)), n
    for n in ("ks", "vs"):
        assert np.array_equal(getattr(got, n), getattr(ref, n), equal_nan=True), n


def rows(rng, n, heads, d, dev, spread=0.0):
    x = rng.standard_normal((n, heads, d)) * 2.0 ** (rng.standard_normal((n, 1, 1)) * spread)
    return torch.from_numpy(x.astype(np.float32)).bfloat16().to(dev)


def write_all(plan, cache, ref, parent, seg, cap, pages, k, v, fresh=None):
    """The library's write and the reference's."""
    TD.tree_cache_write(plan, cache, k, v)
    kn, vn = (x.float().cpu().numpy().astype(np.float64) for x in (k, v))
    for page, row, n, _ in plan.export()["write_jobs"]:
        ref.write_page(int(page), kn[row:row + n], vn[row:row + n])


def check(plan, cache, ref, parent, lens, cap, pages, queries, q, scale, o, lse):
    wo, wl, mass, coarse, reach = OD.decode(ref, parent, lens, cap, pages, queries, q.float().cpu().numpy(), scale)
    go, gl = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    live = np.asarray(queries) >= 0
    fine = np.isfinite(wl)
    assert np.array_equal(gl[:, live][~fine[:, live]], wl[:, live][~fine[:, live]])      # -inf where nothing is attended
    x = 2.0 ** -18 * reach
    err = np.abs(np.where(fine, gl - np.where(fine, wl, 0), 0))[:, live]
    tol = (x + 2.0 ** -20 * (1 + np.abs(np.where(fine, wl, 0))))[:, live]
    assert (err <= tol).all(), f"LSE: {(err / tol).max():.2f} of the bound"
    err = np.abs(go - wo)[live]
    tol = (2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2.0 ** -13 + 4 * x.T[:, :, None]) * mass + 2.0 ** -37 * coarse)[live]
    assert (err <= tol + 1e-30).all(), f"O: {(err / (tol + 1e-30)).max():.2f} of the bound"


def build(rng, parent, seg, queries, hq, hkv, d, dev, cap=None, items=(0, 0), spread=0.0, spare=3):
    cap = seg if cap is None else cap
    need = sum(-(-int(c) // 64) for c in cap)
    pages = rng.permutation(need + spare)[:need]
    plan = TD.DecodePlan(parent, seg, queries, hq, hkv, d, capacity=cap, pages=pages, n_pages=need + spare,
                         cta_pages=items[0], warp_pages=items[1])
    cache, ref = cache_pair(need + spare, hkv, d, dev)
    n = plan.info["n_fresh_tokens"]
    k, v = rows(rng, n, hkv, d, dev, spread), rows(rng, n, hkv, d, dev, spread)
    write_all(plan, cache, ref, parent, seg, cap, pages, k, v)
    return plan, cache, ref, pages


TREES = {
    "one token": ([-1], [1], [0]),
    "one page": ([-1], [64], [0, 0, 0]),
    "page and one": ([-1], [65], [0]),
    "empty branches": ([-1, 0, 0, 1], [70, 0, 3, 0], [1, 2, 3, -1]),
    "nothing at all": ([-1, 0], [0, 0], [1, -1, 0]),
    "chain": ([-1, 0, 1, 2, 3], [1, 127, 64, 2, 200], [4, 2, 0]),
    "forest": ([-1, 0, -1, 2, -1], [130, 1, 63, 66, 5], [1, 3, 4, -1, 1]),
    "star": ([-1] + [0] * 21, [300] + [5 + 7 * i for i in range(21)], list(range(1, 22))),
}


@pytest.mark.parametrize("heads", [(2, 2, 64), (8, 1, 128), (14, 2, 128), (3, 3, 128), (67, 1, 64), (130, 1, 128), (20, 2, 64)])
@pytest.mark.parametrize("name", list(TREES))
def test_write_and_decode(lib, cuda_device, name, heads):
    parent, seg, queries = TREES[name]
    hq, hkv, d = heads
    rng = np.random.default_rng([hq, d, len(name)])
    plan, cache, ref, pages = build(rng, parent, seg, queries, hq, hkv, d, cuda_device)
    assert_same_cache(cache, ref)
    q = rows(rng, len(queries), hq, d, cuda_device)
    o = torch.full((len(queries), hq, d), 7.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((hq, len(queries)), 7.0, device=cuda_device)
    got = TD.tree_decode(plan, cache, plan.lens(), q, d ** -0.5, o=o, lse=lse)
    assert got[0] is o and got[1] is lse and device_status() == 0
    pad = [r for r, u in enumerate(queries) if u < 0]
    assert (o[pad] == 7).all() and (lse[:, pad] == 7).all()          # padding rows stay
    check(plan, cache, ref, parent, seg, seg, pages, queries, q, d ** -0.5, o, lse)


@pytest.mark.parametrize("items", [(0, 0), (1, 1), (5, 3), (128, 32)])
@pytest.mark.parametrize("seed", range(6))
def test_random_trees(lib, cuda_device, seed, items):
    """Random forests, inner and repeated queries, spare room, lengths of the moment
    below, at and beyond the room, and pages whose magnitudes differ widely."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(3, 25))
    t = WT.random_tree(rng, n, [1, 7, 64, 100, 129, 500], n_roots=int(rng.integers(1, 4)))
    cap = [x + int(rng.choice([0, 1, 70])) for x in t.seg_len]
    queries = [int(x) for x in rng.integers(-1, n, size=int(rng.integers(1, 40)))]
    hq, hkv, d = [(8, 2, 64), (16, 2, 128), (5, 1, 128)][seed % 3]
    plan, cache, ref, pages = build(rng, t.parent, t.seg_len, queries, hq, hkv, d, cuda_device, cap=cap, items=items,
                                    spread=3.0)
    lens = [int(rng.choice([x, x, max(0, x - 1), x // 2, 0])) for x in t.seg_len]
    q = rows(rng, len(queries), hq, d, cuda_device)
    o = torch.zeros((len(queries), hq, d), dtype=torch.bfloat16, device=cuda_device)
    lse = torch.zeros((hq, len(queries)), device=cuda_device)
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    TD.tree_decode(plan, cache, ln, q, d ** -0.5, o=o, lse=lse)
    check(plan, cache, ref, t.parent, lens, cap, pages, queries, q, d ** -0.5, o, lse)
    again = TD.tree_decode(plan, cache, ln, q, d ** -0.5, o=torch.zeros_like(o), lse=torch.zeros_like(lse))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)          # bitwise reproducible
    assert device_status() == 0


def test_lengths_out_of_range_are_clamped(lib, cuda_device):
    """Negative lengths read nothing, lengths beyond the room read the room."""
    rng = np.random.default_rng(3)
    parent, seg, queries = [-1, 0, 0], [130, 65, 10], [1, 2]
    plan, cache, ref, pages = build(rng, parent, seg, queries, 4, 2, 128, cuda_device)
    q = rows(rng, 2, 4, 128, cuda_device)
    for lens in ([-5, 65, 10], [10 ** 9, 66, 2 ** 31 - 1], [-2 ** 31, 0, -1]):
        o, lse = TD.tree_decode(plan, cache, torch.tensor(lens, dtype=torch.int32, device=cuda_device), q, 0.1)
        check(plan, cache, ref, parent, [max(0, min(a, b)) for a, b in zip(lens, seg)], seg, pages, queries, q, 0.1, o, lse)


@pytest.mark.parametrize("kv", [(0, 0), (12, -12), (-30, 30), (-90, -90), (60, 60)])
def test_page_scales_far_apart(lib, cuda_device, kv):
    """Alternate pages scaled by powers of two: each term keeps its weight whatever the
    scales are, including pages that vanish beside the others."""
    rng = np.random.default_rng(9)
    d, hkv, seg = 128, 1, [64 * 6 + 9]
    plan = TD.DecodePlan([-1], seg, [0], 4, hkv, d)
    cache, ref = cache_pair(plan.n_pages, hkv, d, cuda_device)
    k, v = rows(rng, seg[0], hkv, d, cuda_device), rows(rng, seg[0], hkv, d, cuda_device)
    odd = (torch.arange(seg[0], device=cuda_device) // 64 % 2 == 1)[:, None, None]
    k = torch.where(odd, k * 2.0 ** min(kv[0], 0), k)      # keys only smaller: logits stay in range
    v = torch.where(odd, v * 2.0 ** kv[1], v)
    write_all(plan, cache, ref, [-1], seg, seg, range(plan.n_pages), k, v)
    assert_same_cache(cache, ref)
    q = rows(rng, 1, 4, d, cuda_device)
    o, lse = TD.tree_decode(plan, cache, plan.lens(), q, d ** -0.5)
    check(plan, cache, ref, [-1], seg, seg, list(range(plan.n_pages)), [0], q, d ** -0.5, o, lse)


@pytest.mark.parametrize("rows_", [1, 3])
@pytest.mark.parametrize("apart", [(0, None), (100, None), (None, 100), (100, -90), (None, None)])
def test_weights_survive_any_scale(lib, cuda_device, rows_, apart):
    """Pages whose values lie up to 2^200 apart, all zero (scale 2^-100) included: every key
    counts in the normaliser.  Both bodies; parts joined across items."""
    rng = np.random.default_rng(15)
    d, hq, seg = 64, 4 * rows_, [64 * 9 + 5]
    plan = TD.DecodePlan([-1], seg, [0], hq, 1, d, cta_pages=3, warp_pages=3)
    cache, ref = cache_pair(plan.n_pages, 1, d, cuda_device)
    k, v = rows(rng, seg[0], 1, d, cuda_device), rows(rng, seg[0], 1, d, cuda_device)
    for start, a in zip((0, 64), apart):                # even and odd pages
        pick = (torch.arange(seg[0], device=cuda_device) // 64 * 64 % 128 == start)[:, None, None]
        v = torch.where(pick, v * (0.0 if a is None else 2.0 ** a), v)
    write_all(plan, cache, ref, [-1], seg, seg, range(plan.n_pages), k, v)
    q = rows(rng, 1, hq, d, cuda_device)
    o, lse = TD.tree_decode(plan, cache, plan.lens(), q, d ** -0.5)
    check(plan, cache, ref, [-1], seg, seg, list(range(plan.n_pages)), [0], q, d ** -0.5, o, lse)


@pytest.mark.parametrize("hq", [4, 12])
def test_long_prefix_of_zero_values(lib, cuda_device, hq):
    """131,072 keys with values of zero: O = 0 exactly, the log-sum-exp that of the scores."""
    n, d = 131072, 64
    plan = TD.DecodePlan([-1], [n], [0], hq, 1, d)
    cache = TD.TreeCache.empty(plan.n_pages, 1, d, cuda_device)
    k = torch.randn((n, 1, d), device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(1)).bfloat16()
    TD.tree_cache_write(plan, cache, k, torch.zeros_like(k))
    o, lse = TD.tree_decode(plan, cache, plan.lens(), torch.zeros((1, hq, d), dtype=torch.bfloat16, device=cuda_device), 0.1)
    # zero scores: every weight is the same power of two, the sums are exact; the logarithm is
    # within two units and its product with ln 2 within one
    assert (o == 0).all() and np.abs(lse.cpu().numpy() - np.log(n)).max() <= 4 * 2.0 ** -23 * np.log(n)
    assert device_status() == 0


@pytest.mark.parametrize("size", [-120, -40, 0, 40, 100])
def test_query_magnitudes(lib, cuda_device, size):
    """Query rows of any magnitude, one row of zeros, one with a single large feature."""
    rng = np.random.default_rng(11)
    parent, seg = [-1, 0, 0], [200, 30, 64]
    plan, cache, ref, pages = build(rng, parent, seg, [1, 2, 2, 1], 8, 2, 64, cuda_device)
    q = rows(rng, 4, 8, 64, cuda_device) * 2.0 ** size
    q[1] = 0
    q[2, :, 5] = 2.0 ** size * 300
    scale = 2.0 ** -min(max(size, -100), 100) * 0.05
    o, lse = TD.tree_decode(plan, cache, plan.lens(), q, scale)
    check(plan, cache, ref, parent, seg, seg, pages, [1, 2, 2, 1], q, scale, o, lse)


def test_write_keeps_what_is_not_its_own(lib, cuda_device):
    """Only fresh nodes' tokens and their pages' scales change; specials are kept."""
    rng = np.random.default_rng(4)
    parent, seg, cap, fresh = [-1, 0, 0, 1], [70, 64, 129, 5], [70, 100, 130, 64], [True, False, True, True]
    pages = rng.permutation(9)[:8]
    for d, hkv in ((64, 3), (128, 2)):
        plan = TD.DecodePlan(parent, seg, [2], hkv, hkv, d, capacity=cap, pages=pages, n_pages=9, fresh=fresh)
        cache, ref = cache_pair(9, hkv, d, cuda_device, fill=0x2B)
        n = plan.info["n_fresh_tokens"]
        assert n == 70 + 129 + 5
        k, v = rows(rng, n, hkv, d, cuda_device, spread=4), rows(rng, n, hkv, d, cuda_device, spread=4)
        k[3, 0, 1], k[4, 1, 2], v[5, 0, 3], v[150, 1, 9] = float("inf"), float("-inf"), float("nan"), float("inf")
        k[70:134, 0] = 0                                    # a page of zeros: the smallest scale
        v[70:134, 0] = 0
        k[140, 0, 0], v[141, 0, 0] = 3.3e38, -3.3e38        # bf16's last octave
        v[199:, 1] = 1e-39                                  # subnormal
        write_all(plan, cache, ref, parent, seg, cap, pages, k, v)
        assert_same_cache(cache, ref)
        # the same rows out of a wider projection, strided
        cache2, _ = cache_pair(9, hkv, d, cuda_device, fill=0x2B)
        qkv = torch.full((n, 5 * hkv + 3, d), 9.0, dtype=torch.bfloat16, device=cuda_device)
        qkv[:, 3:3 + hkv], qkv[:, 3 + hkv:3 + 2 * hkv] = k, v
        TD.tree_cache_write(plan, cache2, qkv[:, 3:3 + hkv], qkv[:, 3 + hkv:3 + 2 * hkv])
        assert_same_cache(cache2, ref)


@pytest.mark.parametrize("heads", [(2, 64), (1, 128), (11, 128)])
def test_append_token_by_token(lib, cuda_device, heads):
    """130 appends to three nodes -- one empty, one inside a page, one at a page's end --
    with tokens whose size jumps, codes and scales bit for bit after every one."""
    hkv, d = heads
    rng = np.random.default_rng(hkv)
    parent, seg, cap = [-1, 0, 0, 0, 1], [64, 0, 37, 64, 12], [64, 130, 200, 200, 12]
    queries = [3, 1, -1, 2]
    need = sum(-(-c // 64) for c in cap)
    pages = rng.permutation(need)
    plan = TD.DecodePlan(parent, seg, queries, hkv, hkv, d, capacity=cap, pages=pages)
    cache, ref = cache_pair(need, hkv, d, cuda_device)
    n = plan.info["n_fresh_tokens"]
    write_all(plan, cache, ref, parent, seg, cap, pages, rows(rng, n, hkv, d, cuda_device), rows(rng, n, hkv, d, cuda_device))
    at, lens, host = OD.node_pages(cap, pages), plan.lens(), list(seg)
    for step in range(130):
        k, v = rows(rng, 4, hkv, d, cuda_device, spread=2.5), rows(rng, 4, hkv, d, cuda_device, spread=2.5)
        if step == 5:
            k[0, 0, 0], v[1, 0, 1], v[3, 0, 2] = float("inf"), float("nan"), 1e30
        if step == 70:
            k[:] = 0
        kn, vn = (x.float().cpu().numpy().astype(np.float64) for x in (k, v))
        assert TD.tree_cache_append(plan, cache, lens, k, v) is lens
        for r, u in enumerate(queries):
            if u >= 0:
                ref.append(at[u][host[u] // 64], host[u] % 64, kn[r], vn[r])
                host[u] += 1
        if step % 8 in (0, 5) or step > 120:
            assert_same_cache(cache, ref)
        assert lens.tolist() == host
    assert device_status() == 0
    # node 1 is full: its token is dropped and said so, the others go on
    out = torch.full_like(lens, -9)
    k = rows(rng, 4, hkv, d, cuda_device)
    assert TD.tree_cache_append(plan, cache, lens, k, k, lens_out=out) is out
    kn = k.float().cpu().numpy().astype(np.float64)
    for r in (0, 3):
        ref.append(at[queries[r]][host[queries[r]] // 64], host[queries[r]] % 64, kn[r], kn[r])
    assert_same_cache(cache, ref)
    assert out.tolist() == [-9, host[1], host[2] + 1, host[3] + 1, -9] and lens.tolist() == host
    assert device_status() == TD.ERR_CACHE_FULL and device_status() == 0


def test_strided_query_rows(lib, cuda_device):
    rng = np.random.default_rng(8)
    parent, seg, queries = [-1, 0, 0], [100, 65, 10], [1, 2, 1]
    plan, cache, ref, pages = build(rng, parent, seg, queries, 6, 2, 128, cuda_device)
    qkv = rows(rng, 3, 10, 128, cuda_device)
    o, lse = TD.tree_decode(plan, cache, plan.lens(), qkv[:, :6], 0.09)
    want = TD.tree_decode(plan, cache, plan.lens(), qkv[:, :6].contiguous(), 0.09)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    check(plan, cache, ref, parent, seg, seg, pages, queries, qkv[:, :6], 0.09, o, lse)


def test_nan_is_not_hidden(lib, cuda_device):
    """A NaN key or value on a path reaches the queries that attend to it, and no others."""
    rng = np.random.default_rng(6)
    parent, seg, queries = [-1, 0, 0], [100, 65, 70], [1, 2]
    plan = TD.DecodePlan(parent, seg, queries, 4, 2, 64)
    cache, _ = cache_pair(plan.n_pages, 2, 64, cuda_device)
    k, v = rows(rng, 235, 2, 64, cuda_device), rows(rng, 235, 2, 64, cuda_device)
    v[100 + 3, 1, 7] = float("nan")          # node 1, kv-head 1, feature 7
    k[165 + 69, 0, 3] = float("nan")         # node 2's last token, kv-head 0
    TD.tree_cache_write(plan, cache, k, v)
    o, lse = TD.tree_decode(plan, cache, plan.lens(), rows(rng, 2, 4, 64, cuda_device), 0.1)
    bad = torch.isnan(o.float())
    assert bad[0, 2:, 7].all() and int(bad[0].sum()) == 2 and torch.isfinite(lse[:, 0]).all()
    assert bad[1, :2].all() and int(bad[1].sum()) == 2 * 64 and torch.isnan(lse[:2, 1]).all()
    # one token fewer, and the NaN key is behind the node's end
    o, lse = TD.tree_decode(plan, cache, torch.tensor([100, 65, 69], dtype=torch.int32, device=cuda_device),
                            rows(rng, 2, 4, 64, cuda_device), 0.1)
    assert torch.isfinite(o[1].float()).all() and torch.isfinite(lse[:, 1]).all()


def test_graph_and_streams(lib, cuda_device):
    """A captured append + attention step replayed over a growing node gives the eager
    results; two streams with a workspace each do not disturb one another."""
    rng = np.random.default_rng(12)
    parent, seg, cap, queries = [-1, 0, 0], [700, 60, 3], [700, 300, 300], [1, 2]
    pages = list(range(11 + 5 + 5))
    made = []
    for _ in range(2):
        plan = TD.DecodePlan(parent, seg, queries, 16, 2, 128, capacity=cap, pages=pages)
        cache, _ = cache_pair(len(pages), 2, 128, cuda_device)
        made.append((plan, cache, plan.lens()))
    k, v = rows(rng, 763, 2, 128, cuda_device), rows(rng, 763, 2, 128, cuda_device)
    k1, v1, q = (torch.zeros((2, h, 128), dtype=torch.bfloat16, device=cuda_device) for h in (2, 2, 16))
    steps = [(rows(rng, 2, 2, 128, cuda_device, 1.0), rows(rng, 2, 2, 128, cuda_device, 1.0), rows(rng, 2, 16, 128, cuda_device))
             for _ in range(10)]
    for plan, cache, _ in made:
        TD.tree_cache_write(plan, cache, k, v)
    (pa, ca, la), (pb, cb, lb) = made
    pa.upload()
    ws = torch.empty(pa.workspace_bytes, dtype=torch.uint8, device=cuda_device)
    o, lse = torch.empty((2, 16, 128), dtype=torch.bfloat16, device=cuda_device), torch.empty((16, 2), device=cuda_device)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        TD.tree_cache_append(pa, ca, la, k1, v1)
        TD.tree_decode(pa, ca, la, q, 0.08, o=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    for a, b, c in steps:
        k1.copy_(a), v1.copy_(b), q.copy_(c)
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        TD.tree_cache_append(pb, cb, lb, a, b, stream=side)
        o2, lse2 = TD.tree_decode(pb, cb, lb, c, 0.08, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert la.tolist() == [700, 70, 13] and torch.equal(ca.k.view(torch.uint8), cb.k.view(torch.uint8))
    assert device_status() == 0


def test_many_pages_in_flight(lib, cuda_device):
    """Pages land in any order and the warps of an item take them in turn: long items of
    one row tile and of several, called back to back, give the same bits every time."""
    rng = np.random.default_rng(13)
    parent, seg = [-1] + [0] * 24, [64 * 150 + 5] + [64 * int(x) + 9 for x in rng.integers(5, 90, 24)]
    for hq, queries in ((4, [3]), (8, [1, 2, 3, 4, 5]), (8, list(range(1, 25)))):
        plan, cache, ref, pages = build(rng, parent, seg, queries, hq, 2, 128, cuda_device, items=(128, 32))
        q, ln = rows(rng, len(queries), hq, 128, cuda_device), plan.lens()
        outs = [TD.tree_decode(plan, cache, ln, q, 0.09) for _ in range(150)]
        assert device_status() == 0
        assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
        sub = [queries[-1]]
        wo = OD.decode(ref, parent, seg, seg, pages, sub, q[-1:].float().cpu().numpy(), 0.09)[0]
        assert np.abs(outs[0][0][-1].float().cpu().numpy() - wo[0]).max() <= 2e-2


def test_refused_tensors(lib, cuda_device):
    plan = TD.DecodePlan([-1, 0], [70, 5], [1, 0], 4, 2, 64)
    cache = TD.TreeCache.empty(plan.n_pages, 2, 64, cuda_device)
    bf = dict(dtype=torch.bfloat16, device=cuda_device)
    q, k, lens = torch.zeros((2, 4, 64), **bf), torch.zeros((75, 2, 64), **bf), plan.lens()
    one = torch.zeros((2, 2, 64), **bf)
    bad = [lambda: TD.tree_decode(plan, cache, lens, q.half(), 1.0), lambda: TD.tree_decode(plan, cache, lens, q.float(), 1.0),
           lambda: TD.tree_decode(plan, cache, lens, q[:1], 1.0), lambda: TD.tree_decode(plan, cache, lens, q.cpu(), 1.0),
           lambda: TD.tree_decode(plan, cache, lens.long(), q, 1.0), lambda: TD.tree_decode(plan, cache, lens[:1], q, 1.0),
           lambda: TD.tree_decode(plan, cache, lens, q.transpose(1, 2).contiguous().transpose(1, 2), 1.0),
           lambda: TD.tree_decode(plan, cache, lens, torch.zeros((2, 257), **bf)[:, :256].view(2, 4, 64), 1.0),
           lambda: TD.tree_decode(plan, cache, lens, q[:1].expand(2, 4, 64), 1.0),
           lambda: TD.tree_decode(plan, cache, lens, q, 1.0, o=q.float()),
           lambda: TD.tree_decode(plan, cache, lens, q, 1.0, lse=torch.zeros((2, 4), device=cuda_device)),
           lambda: TD.tree_decode(plan, cache, lens, q, 1.0, workspace=torch.zeros(9, device=cuda_device)),
           lambda: TD.tree_cache_write(plan, cache, k[:74], k), lambda: TD.tree_cache_write(plan, cache, k, k.float()),
           lambda: TD.tree_cache_append(plan, cache, lens, one[:1], one),
           lambda: TD.tree_cache_append(plan, cache, lens, one, one, lens_out=lens.long()),
           lambda: TD.tree_decode(plan, TD.TreeCache.empty(plan.n_pages, 1, 64, cuda_device), lens, q, 1.0),
           lambda: TD.tree_decode(plan, TD.TreeCache.empty(plan.n_pages - 1, 2, 64, cuda_device), lens, q, 1.0),
           lambda: TD.TreeCache(cache.k, cache.v, cache.k_scale, cache.v_scale[:1]),
           lambda: TD.TreeCache(cache.k, cache.k, cache.k_scale, cache.v_scale.cpu()),
           lambda: TD.TreeCache(cache.k.view(torch.uint8), cache.v, cache.k_scale, cache.v_scale)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            f()
            pytest.fail(f"call {i} was taken", pytrace=False)


@pytest.mark.parametrize("heads", [(8, 2, 64), (16, 2, 128)])
def test_debug_build_is_clean_and_gives_the_same_bits(lib, cuda_device, heads):
    """Write, append and attention of items of both kinds through the
    bounds-checked build."""
    hq, hkv, d = heads
    parent, seg, queries = [-1, 0, 0, 2, 2], [400, 63, 90, 10, 0], [1, 3, -1, 4]
    cap, out = [400, 66, 90, 130, 1], []
    for path in (_build.LIB, _build.build_library(debug=True)):
        with B.library(path):
            rng = np.random.default_rng(31)
            plan, cache, _, _ = build(rng, parent, seg, queries, hq, hkv, d, cuda_device, cap=cap)
            lens = plan.lens()
            o, lse = torch.zeros((4, hq, d), dtype=torch.bfloat16, device=cuda_device), torch.zeros((hq, 4), device=cuda_device)
            TD.tree_cache_append(plan, cache, lens, rows(rng, 4, hkv, d, cuda_device), rows(rng, 4, hkv, d, cuda_device))
            TD.tree_decode(plan, cache, lens, rows(rng, 4, hq, d, cuda_device), d ** -0.5, o=o, lse=lse)
            torch.cuda.synchronize()
            assert device_status() == 0, path
            out.append((o, lse, cache.k.view(torch.uint8), cache.v.view(torch.uint8), lens))
            plan.close()
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("hq", [8, 32])
def test_pages_behind_32_bit_offsets(lib, cuda_device, hq):
    """Pages whose codes lie behind 2^32 bytes of their pool: write, append and attention of
    both kinds of item give what the first pages of a small pool give."""
    rng = np.random.default_rng(41)
    hkv, d, far = 8, 128, 65600                            # 65,536 bytes per page of K, and of V
    parent, seg, cap, queries = [-1, 0, 0], [150, 64, 3], [150, 65, 70], [1, 2]
    k, v = rows(rng, 217, hkv, d, cuda_device), rows(rng, 217, hkv, d, cuda_device)
    k1, v1, q = (rows(rng, 2, h, d, cuda_device) for h in (hkv, hkv, hq))
    outs = []
    for first in (0, far):
        plan = TD.DecodePlan(parent, seg, queries, hq, hkv, d, capacity=cap, pages=range(first, first + 7))
        cache, lens = TD.TreeCache.empty(plan.n_pages, hkv, d, cuda_device), plan.lens()
        assert first == 0 or cache.k.numel() > 2 ** 32
        for x in (cache.k, cache.v):
            x[first:].view(torch.uint8).fill_(POISON)
        TD.tree_cache_write(plan, cache, k, v)
        TD.tree_cache_append(plan, cache, lens, k1, v1)
        o, lse = TD.tree_decode(plan, cache, lens, q, 0.09)
        torch.cuda.synchronize()
        outs.append((o, lse, lens, cache.k[first:].view(torch.uint8).clone(), cache.v[first:].view(torch.uint8).clone(),
                     cache.k_scale[first:].clone()))
    assert torch.isfinite(outs[0][0].float()).all() and device_status() == 0
    for n, a, b in zip(("o", "lse", "lens", "k", "v"), *outs):
        assert torch.equal(a, b), n


@pytest.mark.parametrize("pages", [2, 3, 4, 5])
@pytest.mark.parametrize("hq,n_queries", [(9, 1), (16, 1), (12, 2), (32, 1), (33, 1), (16, 8)])
def test_short_items_of_shared_rows_hold_their_last_page(lib, cuda_device, hq, n_queries, pages):
    """Items of a few pages read by 9 to 128 rows, many of them at once and from memory that is
    not in L2: every output holds the last page's values, every time.  The last page's keys
    weigh most, so an output without it would be far outside the bound."""
    rng = np.random.default_rng([hq, n_queries, pages])
    d, hkv, runs = 128, 1, 300
    parent, seg = [-1] * runs, [64 * pages - 9] * runs
    queries = [u for u in range(runs) for _ in range(n_queries)]
    plan = TD.DecodePlan(parent, seg, queries, hq, hkv, d, cta_pages=pages, warp_pages=1)
    assert all(x[0][5] == 1 and x[0][1] == pages for x in plan.export()["items"])
    cache, ref = cache_pair(plan.n_pages, hkv, d, cuda_device)
    k, v = (rows(rng, sum(seg), hkv, d, cuda_device) for _ in range(2))
    last = torch.arange(sum(seg), device=cuda_device) % seg[0] >= 64 * (pages - 1)
    q = rows(rng, len(queries), hq, d, cuda_device)
    k[:, 0, 0], q[:, :, 0] = torch.where(last, 4.0, -4.0).bfloat16(), 4.0
    v[last] += 2
    write_all(plan, cache, ref, parent, seg, seg, range(plan.n_pages), k, v)
    ln, flush = plan.lens(), torch.empty(2 ** 27, dtype=torch.int32, device=cuda_device)
    outs = []
    for _ in range(12):
        flush.zero_()
        outs.append(TD.tree_decode(plan, cache, ln, q, d ** -0.5))
    assert device_status() == 0
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
    check(plan, cache, ref, parent, seg, seg, list(range(plan.n_pages)), queries, q, d ** -0.5, *outs[0])


def test_a_cache_is_where_its_tensors_are(lib, cuda_device):
    """Its tensors cannot be exchanged behind its back; storage given up is refused, and storage
    brought back elsewhere is found there."""
    rng = np.random.default_rng(51)
    parent, seg, queries = [-1, 0, 0], [130, 65, 10], [1, 2]
    plan, cache, ref, pages = build(rng, parent, seg, queries, 4, 2, 128, cuda_device)
    q, lens = rows(rng, 2, 4, 128, cuda_device), plan.lens()
    want = TD.tree_decode(plan, cache, lens, q, 0.1)
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name).clone())
    kept = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)]
    torch.cuda.synchronize()
    mine = (cache.k, cache.v, cache.k_scale, cache.v_scale)
    size = [x.untyped_storage().nbytes() for x in mine]
    for x in mine:
        x.untyped_storage().resize_(0)
    one = torch.zeros((2, 2, 128), dtype=torch.bfloat16, device=cuda_device)
    for call in (lambda: TD.tree_decode(plan, cache, lens, q, 0.1), lambda: TD.tree_cache_append(plan, cache, lens, one, one)):
        with pytest.raises(B.TreeAttnError):
            call()
    others = [torch.empty(n, dtype=torch.uint8, device=cuda_device) for n in size]   # in their old places
    for x, n, b in zip(mine, size, kept):
        x.untyped_storage().resize_(n)
        (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x).copy_(b)
    assert len(others) == 4
    got = TD.tree_decode(plan, cache, lens, q, 0.1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_a_pool_of_no_pages(lib, cuda_device, d):
    """Nodes without room: the attention gives O = 0 and LSE = -inf, an append is dropped."""
    plan = TD.DecodePlan([-1, 0], [0, 0], [1, -1, 0], 4, 2, d)
    cache, lens = TD.TreeCache.empty(plan.n_pages, 2, d, cuda_device), plan.lens()
    assert plan.n_pages == 0
    q = torch.ones((3, 4, d), dtype=torch.bfloat16, device=cuda_device)
    o, lse = torch.full_like(q, 7), torch.full((4, 3), 7.0, device=cuda_device)
    TD.tree_cache_write(plan, cache, q[:0, :2], q[:0, :2])
    TD.tree_decode(plan, cache, lens, q, 0.1, o=o, lse=lse)
    assert (o[[0, 2]] == 0).all() and (lse[:, [0, 2]] == -float("inf")).all()
    assert (o[1] == 7).all() and (lse[:, 1] == 7).all() and device_status() == 0
    TD.tree_cache_append(plan, cache, lens, q[:, :2], q[:, :2])
    assert lens.tolist() == [0, 0] and device_status() == TD.ERR_CACHE_FULL and device_status() == 0


@pytest.mark.parametrize("seed", range(4))
def test_random_lengths_beyond_the_room(lib, cuda_device, seed):
    """Random trees whose lengths of the moment lie below, at and beyond the room (where the room
    counts), at both kinds of items."""
    rng = np.random.default_rng([seed, 77])
    n = int(rng.integers(4, 20))
    t = WT.random_tree(rng, n, [1, 7, 64, 100, 129, 500], n_roots=int(rng.integers(1, 4)))
    cap = [x + int(rng.choice([0, 1, 70])) for x in t.seg_len]
    queries = [int(x) for x in rng.integers(-1, n, size=int(rng.integers(8, 40)))]
    hq, hkv, d = [(8, 2, 64), (16, 2, 128), (5, 1, 128), (24, 2, 64)][seed]
    plan, cache, ref, pages = build(rng, t.parent, t.seg_len, queries, hq, hkv, d, cuda_device, cap=cap)
    # every slot of the room holds a token
    full = TD.DecodePlan(t.parent, cap, queries, hq, hkv, d, pages=pages, n_pages=plan.n_pages)
    k, v = (rows(rng, sum(cap), hkv, d, cuda_device) for _ in range(2))
    write_all(full, cache, ref, t.parent, cap, cap, pages, k, v)
    lens = [int(rng.choice([x, c, c + 1, c + 1000, 2 ** 31 - 1, 0, -3])) for x, c in zip(t.seg_len, cap)]
    q = rows(rng, len(queries), hq, d, cuda_device)
    o = torch.zeros((len(queries), hq, d), dtype=torch.bfloat16, device=cuda_device)
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    o, lse = TD.tree_decode(plan, cache, ln, q, d ** -0.5, o=o, lse=torch.zeros((hq, len(queries)), device=cuda_device))
    now = [max(0, min(a, c)) for a, c in zip(lens, cap)]
    check(plan, cache, ref, t.parent, now, cap, pages, queries, q, d ** -0.5, o, lse)
    assert device_status() == 0
