"""Linear attention from and to states in slots (include/tree_linear.h): whole turns and single
tokens, against the fp64 oracle.

Tolerances, from the arithmetic.  Step: k v^T is within 2^-24 of itself, its sum with gamma S within
2^-24 of the result: together below 2^-23 of |gamma S| + |k v|.  o sums d products in fp32: within
(d + 8) 2^-24 of the sum of their magnitudes, then 2^-8 of itself.  Prefill: an increment sums 3 * 128
products on the tensor cores, each addition within 2^-23 of the sum of magnitudes; a power
2^(n log2 gamma) is within 2^-22 (1 + n |log2 gamma|) of itself, and where n |log2 gamma| > 24 it does
not count; chunks and nodes add as much again once for each of fewer than 16 chunks: states within
2^-13 of their sums of magnitudes.  o: one rounding to bf16 of each of its two parts, within 2^-8 of the
magnitudes that are multiplied, 2^-12 for everything in fp32, and 2^-8 of itself.  (The
rows of a decay below 2^(-100/128) round the scaled query too: 2^-8 of the entering part once more.)"""
import numpy as np
import pytest
import torch

from oracle import layout as OL
from oracle import linear as OLN
from prefix_tree_attention_attn_gb300 import TreePlan, build as _build, device_status
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import linear as TL

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib, cuda_device):
    yield
    torch.cuda.synchronize()
    assert device_status() == 0


def num(t):
    return t.double().cpu().numpy()


def draw(seed, N, hq, hkv, d, device, size=1.0):
    g = torch.Generator(device).manual_seed(seed)
    make = lambda *s: (torch.randn(s, device=device, generator=g) * size).bfloat16()  # noqa: E731
    return make(N, hq, d), make(N, hkv, d), make(N, hkv, d)


def randn(shape, device, seed=91):
    return torch.randn(shape, device=device, generator=torch.Generator(device).manual_seed(seed))


def decays(hkv, device, values=(1.0, 0.9, 0.99, 0.999)):
    return torch.tensor([values[i % len(values)] for i in range(hkv)], device=device)


def check_prefill(parent, seg, hq, hkv, device, seed=1, slot_in=None, slot_out=None, values=(1.0, 0.9, 0.99, 0.999), n_slots=9):
    N, n = sum(seg), len(parent)
    q, k, v = draw(seed, N, hq, hkv, 128, device)
    dec = decays(hkv, device, values)
    g = torch.Generator(device).manual_seed(seed + 100)
    states = torch.randn((n_slots, hkv, 128, 128), device=device, generator=g) * 3
    before = states.clone()
    slot_in = [-1] * n if slot_in is None else slot_in
    slot_out = list(range(n)) if slot_out is None else slot_out
    plan = TreePlan(parent, seg)
    o = TL.tree_linear_prefill(plan, states, TL.StateSlots(slot_in, slot_out, n_slots), q, k, v, dec, 0.125)
    start = [num(before[s]) if p < 0 and s >= 0 else None for p, s in zip(parent, slot_in)]
    want, end, size, mass = OLN.from_states(parent, seg, num(q), num(k), num(v), num(dec), 0.125, start)
    wide = 2 if min(values) < 0.58 else 1
    lim = 2.0 ** -8 * np.abs(want) + (wide * 2.0 ** -8 + 2.0 ** -12) * size + 1e-30
    e = np.abs(num(o) - want)
    assert (e <= lim).all(), (np.unravel_index(np.argmax(e / lim), e.shape), (e / lim).max())
    for u in range(n):
        if slot_out[u] >= 0:
            e = np.abs(num(states[slot_out[u]]) - end[u])
            assert (e <= 2.0 ** -13 * mass[u] + 1e-30).all(), (u, (e / mass[u]).max())
    kept = [s for s in range(n_slots) if s not in slot_out]
    assert torch.equal(states[kept], before[kept])
    return o, states


@pytest.mark.parametrize("parent,seg,hq,hkv", [
    ([-1], [1], 2, 1),
    ([-1], [300], 2, 2),
    ([-1, 0, 0], [127, 129, 1], 8, 2),
    ([-1, 0, 0, 1, 1, 2], [128, 200, 5, 64, 300, 33], 4, 1),
    ([-1, 0, 1, -1, 3], [70, 60, 5, 257, 2], 3, 3),
    ([-1] + [0] * 8, [50] + [(17 * i) % 140 + 1 for i in range(8)], 4, 4),
])
def test_prefill_from_zero(cuda_device, parent, seg, hq, hkv):
    check_prefill(parent, seg, hq, hkv, cuda_device)


def test_prefill_continues_states(cuda_device):
    # two trees from stored states, one from nothing; some states not kept, one left in the slot it came from
    parent, seg = [-1, 0, 0, -1, -1, 3], [130, 17, 260, 33, 128, 5]
    check_prefill(parent, seg, 4, 2, cuda_device, 5, slot_in=[7, 7, -1, 2, -1, 0], slot_out=[-1, 7, 3, -1, 0, 2])
    # two trees fork one state
    check_prefill([-1, -1], [40, 150], 2, 2, cuda_device, 6, slot_in=[8, 8], slot_out=[1, 0])
    check_prefill([-1], [5], 2, 2, cuda_device, 7, slot_in=[4], slot_out=[4])
    check_prefill([-1, 0], [5, 6], 2, 2, cuda_device, 7, slot_in=[4, -1], slot_out=[-1, -1])


@pytest.mark.parametrize("values", [(0.58, 0.585), (0.5, 0.1), (0.001, 1.0), (2.0 ** -100, 0.57)])
def test_prefill_strong_decays(cuda_device, values):
    check_prefill([-1, 0, 0], [150, 129, 40], 4, 2, cuda_device, 8, slot_in=[3, -1, -1], values=values)


def test_prefill_deep_tree(cuda_device):
    # 40 nested nodes: deeper than the scans by depth take; states on the way, and a second root
    n = 40
    parent, seg = [-1] + list(range(n - 1)) + [-1], [(37 * i) % 30 + 1 for i in range(n)] + [12]
    check_prefill(parent, seg, 2, 1, cuda_device, 9, slot_in=[1] + [-1] * (n - 1) + [0],
                  slot_out=[-1] * 20 + [2] + [-1] * (n - 22) + [1, 5])


@pytest.mark.parametrize("seg,kept", [([12 * 128 + 1], [0]), ([3500], [2]), ([2100, 40, 1540, 1537], [0, -1, 3, 4]), ([1536, 4608], [5, 6])])
def test_prefill_in_segments(cuda_device, seg, kept):
    # four: a long root, a short and two long children
    check_segments([-1, 0, 0, 0] if len(seg) == 4 else [-1] + list(range(len(seg) - 1)), seg, kept, 2, cuda_device)


@pytest.mark.parametrize("hkv", [1, 4, 8, 16])
@pytest.mark.parametrize("parent,seg,kept", [
    ([-1], [14 * 128], [0]), ([-1], [15 * 128 - 3], [7]), ([-1], [2048], [7]), ([-1], [5000], [1]), ([-1], [131 * 128 - 7], [2]),
    ([-1] + [0] * 8, [300] + [2000] * 3 + [1, 2, 127, 128, 129], [-1, 0, 1, 2, 3, 4, 5, 6, -1]),
    ([-1] + [0] * 9, [2500] + [1000] * 9, [0, 1, 2, 3, 4, 5, 6, -1, -1, -1]),
    ([-1, -1, 0, 1], [3000, 2200, 1, 4000], [-1, 1, 2, 0])])
def test_prefill_in_pieces(cuda_device, parent, seg, kept, hkv):
    """The numbers of heads and of chunks around which nodes are cut and walks get narrow, some states over the one that
    their root came from."""
    check_segments(parent, seg, kept, hkv, cuda_device)


def check_segments(parent, seg, kept, hkv, cuda_device):
    """Nodes long enough to be walked in segments: against the same tokens as a chain of short nodes, whose
    states are handed on node by node."""
    n_slots, hq, N = 8, 2 * hkv, sum(seg)
    q, k, v = draw(51, N, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (0.999, 1.0))
    first = randn((n_slots, hkv, 128, 128), cuda_device)
    a, b = first.clone(), first.clone()
    o = TL.tree_linear_prefill(TreePlan(parent, seg), a, TL.StateSlots([7] + [-1] * (len(seg) - 1), kept, n_slots), q, k, v, dec, 0.1)
    short, up, out, tip = [], [], [], {}
    for u, L in enumerate(seg):                             # pieces of at most 5 chunks
        for x in range(0, L, 640):
            up.append((tip[parent[u]] if parent[u] >= 0 else -1) if x == 0 else len(short) - 1)
            short.append(min(640, L - x))
            out.append(kept[u] if x + 640 >= L else -1)
        tip[u] = len(short) - 1
    o2 = TL.tree_linear_prefill(TreePlan(up, short), b, TL.StateSlots([7] + [-1] * (len(short) - 1), out, n_slots), q, k, v, dec, 0.1)
    # sums of at most 131 chunks in another order, 2^-13 of the magnitudes as above: here 2^-18 of the largest
    # state of N(0, 1) products, and outputs one rounding of the entering state, of P and of o apart
    assert (a - b).abs().max() <= 2.0 ** -18 * N
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert torch.linalg.vector_norm(o.float() - o2.float()) <= 2.0 ** -9 * torch.linalg.vector_norm(o.float())


@pytest.mark.parametrize("seg,hkv", [([20000], 32), ([9000, 4000], 16)])
def test_prefill_in_segments_over_its_own_slot(cuda_device, seg, hkv):
    """More segments than run at a time, of a root that leaves its state in the slot that it started from."""
    q, k, v = draw(61, sum(seg), hkv, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (0.9999, 1.0))
    first = randn((3, hkv, 128, 128), cuda_device) * 100
    plan = TreePlan([-1] + [0] * (len(seg) - 1), seg)
    rest = [-1] * (len(seg) - 1)
    a, b = first.clone(), first.clone()
    o = TL.tree_linear_prefill(plan, a, TL.StateSlots([1] + rest, [2] + rest, 3), q, k, v, dec, 0.1)
    for _ in range(3):
        b.copy_(first)
        o2 = TL.tree_linear_prefill(plan, b, TL.StateSlots([1] + rest, [1] + rest, 3), q, k, v, dec, 0.1)
        assert torch.equal(o, o2) and torch.equal(a[2], b[1]) and torch.equal(b[[0, 2]], first[[0, 2]])


def test_prefill_in_two_turns_is_the_whole(cuda_device):
    """A prompt, then its branches from the prompt's state: the outputs of the tree brought in at once, and the
    same states, within the bounds of one more rounding of what enters."""
    parent, seg = [-1, 0, 0], [200, 90, 140]
    q, k, v = draw(11, 430, 4, 2, 128, cuda_device)
    dec = decays(2, cuda_device, (0.97, 1.0))
    whole, parts = (torch.zeros((3, 2, 128, 128), device=cuda_device) for _ in range(2))
    o = TL.tree_linear_prefill(TreePlan(parent, seg), whole, TL.StateSlots([-1] * 3, [0, 1, 2], 3), q, k, v, dec, 0.1)
    a = TL.tree_linear_prefill(TreePlan([-1], [200]), parts, TL.StateSlots([-1], [0], 3), q[:200].contiguous(),
                               k[:200].contiguous(), v[:200].contiguous(), dec, 0.1)
    b = TL.tree_linear_prefill(TreePlan([-1, -1], [90, 140]), parts, TL.StateSlots([0, 0], [1, 2], 3), q[200:].contiguous(),
                               k[200:].contiguous(), v[200:].contiguous(), dec, 0.1)
    assert torch.equal(o, torch.cat([a, b])) and torch.equal(whole, parts)


def test_prefill_keeps_other_branches_clean(cuda_device):
    """Infinities and NaN in one branch reach it and its descendants alone, whatever lies beside it in a tile."""
    parent, seg = [-1, 0, 0, 2, 0], [30, 21, 35, 9, 77]
    q, k, v = draw(12, 172, 2, 1, 128, cuda_device)
    for value in (float("inf"), float("nan")):
        for values in ((0.99,), (0.3,)):
            run = lambda k, v: (st := torch.zeros((5, 1, 128, 128), device=cuda_device),  # noqa: E731
                                TL.tree_linear_prefill(TreePlan(parent, seg), st, TL.StateSlots([-1] * 5, range(5), 5), q, k, v,
                                                       decays(1, cuda_device, values), 0.1))
            st0, o0 = run(k, v)
            k2, v2 = k.clone(), v.clone()
            k2[51:86, 0, 3], v2[51:86, 0, 100] = value, value          # node 2; node 3 is below it
            st, o = run(k2, v2)
            rows = [*range(51), *range(95, 172)]
            assert torch.equal(o[rows], o0[rows]) and torch.equal(st[[0, 1, 4]], st0[[0, 1, 4]])
            assert not torch.isfinite(st[2]).all() and not torch.isfinite(st[3]).all()


def check_step(R, hq, hkv, d, device, seed, slot_in, slot_out, n_slots, strided=False):
    g = torch.Generator(device).manual_seed(seed)
    states = torch.randn((n_slots, hkv, d, d), device=device, generator=g) * 4
    before = states.clone()
    if strided:                                                        # rows of one fused projection
        x = torch.randn((R, (hq + 2 * hkv) * d + 8), device=device, generator=g).bfloat16()
        q, k, v = (x[:, a:b].view(R, -1, d) for a, b in ((0, hq * d), (hq * d, (hq + hkv) * d), ((hq + hkv) * d, (hq + 2 * hkv) * d)))
    else:
        q, k, v = draw(seed, R, hq, hkv, d, device)
    dec = decays(hkv, device)
    slots = TL.StateSlots(slot_in, slot_out, n_slots)
    o = torch.full((R, hq, d), 7.0, dtype=torch.bfloat16, device=device)
    assert TL.tree_linear_step(states, slots, q, k, v, dec, 0.2, o=o) is o
    gam = num(dec)[:, None, None]
    for r in range(R):
        if slot_out[r] < 0:
            assert (o[r] == 7).all()
            continue
        S0 = num(before[slot_in[r]]) if slot_in[r] >= 0 else np.zeros((hkv, d, d))
        kv = num(k[r])[:, :, None] * num(v[r])[:, None, :]
        S = gam * S0 + kv
        assert (np.abs(num(states[slot_out[r]]) - S) <= 2.0 ** -23 * (np.abs(gam * S0) + np.abs(kv)) + 1e-37).all()
        S, A = np.repeat(S, hq // hkv, 0), np.repeat(np.abs(gam * S0) + np.abs(kv), hq // hkv, 0)
        want, size = (0.2 * np.einsum("hk,hkv->hv", f(num(q[r])), x) for f, x in ((lambda y: y, S), (np.abs, A)))
        e = np.abs(num(o[r]) - want)
        assert (e <= 2.0 ** -8 * np.abs(want) + (d + 8) * 2.0 ** -24 * size).all()
    kept = [s for s in range(n_slots) if s not in list(slot_out)]
    assert torch.equal(states[kept], before[kept])


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (32, 8, 128), (8, 1, 128), (14, 2, 128), (12, 4, 64), (5, 5, 128), (20, 1, 64)])
def test_step(cuda_device, hq, hkv, d):
    check_step(1, hq, hkv, d, cuda_device, 1, [0], [0], 1)
    check_step(1, hq, hkv, d, cuda_device, 2, [-1], [2], 4)
    check_step(5, hq, hkv, d, cuda_device, 3, [3, 3, 3, 1, -1], [0, 4, -1, 1, 6], 8)       # forks, padding, in place, new
    check_step(3, hq, hkv, d, cuda_device, 4, [2, 0, 1], [2, 0, 1], 3, strided=True)
    R = 1 + 400 // hkv
    perm = np.random.default_rng(5).permutation(R + 3)
    check_step(R, hq, hkv, d, cuda_device, 5, perm[:R], perm[:R], R + 3)


def test_steps_continue_a_prefill(cuda_device):
    """A turn brought in at once and the same turn token by token leave the same states and give the same outputs:
    each within its own bounds of the oracle."""
    seg, hq, hkv = 70, 4, 2
    q, k, v = draw(21, seg, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (0.95, 1.0))
    states = randn((2, hkv, 128, 128), cuda_device)
    start = num(states[0])
    o = TL.tree_linear_prefill(TreePlan([-1], [seg]), states, TL.StateSlots([0], [1], 2), q, k, v, dec, 0.1)
    slots = TL.StateSlots([0], [0], 2)
    steps = torch.cat([TL.tree_linear_step(states, slots, q[i:i + 1], k[i:i + 1], v[i:i + 1], dec, 0.1) for i in range(seg)])
    want, end, size, mass = OLN.from_states([-1], [seg], num(q), num(k), num(v), num(dec), 0.1, [start])
    assert (np.abs(num(states[0]) - end[0]) <= seg * 2.0 ** -23 * mass[0]).all()
    assert (np.abs(num(states[1]) - end[0]) <= 2.0 ** -13 * mass[0]).all()
    whole = 0.1 * np.einsum("thk,hkv->thv", np.abs(num(q)), np.repeat(mass[0], hq // hkv, 0)) + size
    assert (np.abs(num(steps) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * whole).all()
    assert (np.abs(num(o) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -12) * size).all()


def test_step_capture_and_side_stream(cuda_device):
    R, hq, hkv = 9, 8, 2
    q, k, v = draw(31, R, hq, hkv, 128, cuda_device)
    dec, slots = decays(hkv, cuda_device), TL.StateSlots(range(R), range(R), R)
    first = randn((R, hkv, 128, 128), cuda_device)
    a, b, c = first.clone(), first.clone(), first.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = TL.tree_linear_step(c, slots, q, k, v, dec, 0.1, stream=side)      # the tables' first use
    side.synchronize()
    want = TL.tree_linear_step(a, slots, q, k, v, dec, 0.1)
    assert torch.equal(got, want) and torch.equal(a, c)
    plan, ws = TreePlan([-1] * R, [7] * R), None
    pq, pk, pv = draw(32, 7 * R, hq, hkv, 128, cuda_device)
    op = TL.tree_linear_prefill(plan, a, slots, pq, pk, pv, dec, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = TL.tree_linear_step(b, slots, q, k, v, dec, 0.1)
        o2 = TL.tree_linear_prefill(plan, b, slots, pq, pk, pv, dec, 0.1, workspace=ws)
    graph.replay()
    assert torch.equal(o, want) and torch.equal(o2, op) and torch.equal(a, b)
    for _ in range(3):
        want = TL.tree_linear_step(a, slots, q, k, v, dec, 0.1)
        op = TL.tree_linear_prefill(plan, a, slots, pq, pk, pv, dec, 0.1)
        graph.replay()
        assert torch.equal(o, want) and torch.equal(o2, op) and torch.equal(a, b)


def test_reproducible_and_debug_build(cuda_device):
    parent, seg, hq, hkv = [-1, 0, 0, 1, 1, -1], [2000, 300, 129, 64, 1, 500], 8, 2
    n, N = len(seg), sum(seg)
    q, k, v = draw(71, N, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device)
    first = randn((n + 1, hkv, 128, 128), cuda_device)
    fork = TL.StateSlots([0, 0, -1, 3], [1, 2, 4, -1], n + 1)

    def both():
        s = first.clone()
        plan = TreePlan(parent, seg)
        o = TL.tree_linear_prefill(plan, s, TL.StateSlots([n] + [-1] * (n - 1), list(range(n)), n + 1), q, k, v, dec, 0.1)
        o1 = TL.tree_linear_step(s, fork, q[:4], k[:4], v[:4], dec, 0.1, o=torch.zeros_like(q[:4]))
        torch.cuda.synchronize()
        assert device_status() == 0
        return s, o, o1

    want = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(both(), want))
    with B.library(_build.build_library(debug=True)):
        got = both()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_behind_one_another(cuda_device):
    """Inputs that the kernel before a call writes, and calls that hand states on without a pause between them: launches of
    one call overlap, calls do not."""
    parent, seg, hq, hkv = [-1, 0, 0, 1], [300, 140, 700, 33], 8, 4
    N, plan = sum(seg), TreePlan(parent, seg)
    q, k, v = draw(81, N, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (0.9, 0.99))
    slots, turns = TL.StateSlots([0, -1, -1, -1], [-1, 1, -1, 0], 2), 6
    slots.upload()
    factor = torch.tensor([1.0, -0.5, 2.0, 0.25, -1.0, 4.0]).bfloat16().to(cuda_device)

    def chain(wait):
        s = torch.zeros((2, hkv, 128, 128), device=cuda_device)
        kk, vv, ws, out = torch.empty_like(k), torch.empty_like(v), None, []
        ws = torch.empty(TL.prefill_workspace(plan, hkv, 128), dtype=torch.uint8, device=cuda_device)
        for i in range(turns):
            torch.mul(k, factor[i], out=kk)
            torch.mul(v, factor[-i], out=vv)
            out.append(TL.tree_linear_prefill(plan, s, slots, q, kk, vv, dec, 0.1, workspace=ws))
            if wait:
                torch.cuda.synchronize()
        return [s, *out]

    want = chain(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def test_notices(cuda_device, lib):
    """Slot numbers outside the pool and decays outside (0, 1], past the binding's own checks."""
    q, k, v = draw(41, 3, 2, 1, 128, cuda_device)
    states = torch.zeros((2, 1, 128, 128), device=cuda_device)
    o = torch.full((3, 2, 128), 5.0, dtype=torch.bfloat16, device=cuda_device)
    dec = torch.tensor([0.9], device=cuda_device)

    def step(slot_in, slot_out, decay):
        a, b = (torch.tensor(x, dtype=torch.int32, device=cuda_device) for x in (slot_in, slot_out))
        assert lib.tree_attn_linear_step(states.data_ptr(), 2, a.data_ptr(), b.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                         256, 128, 128, o.data_ptr(), decay.data_ptr(), 3, 2, 1, 128, 1.0, None) == 0
        torch.cuda.synchronize()
        return device_status()

    torch.cuda.synchronize()
    assert step([0, -1, -1], [0, 2, -5], dec) == TL.ERR_INVALID_SLOT
    assert (o[1:] == 5).all() and not (o[0] == 5).any() and not states[1].any()
    states.fill_(1)
    assert step([2 ** 30, -1, -1], [1, -1, -1], dec) == TL.ERR_INVALID_SLOT
    kv = k[0, 0].float()[:, None] * v[0, 0].float()[None]
    assert torch.equal(states[1, 0], kv)                               # as from a zero state
    assert step([0, -1, -1], [0, -1, -1], torch.tensor([1.5], device=cuda_device)) == -12
    assert step([0, -1, -1], [0, -1, -1], torch.tensor([float("nan")], device=cuda_device)) == -12
    plan = TreePlan([-1, 0], [2, 1])
    bad = torch.tensor([-1, 2], dtype=torch.int32, device=cuda_device)
    none = torch.tensor([-1, -1], dtype=torch.int32, device=cuda_device)
    ws = torch.empty(TL.prefill_workspace(plan, 1, 128), dtype=torch.uint8, device=cuda_device)
    states.fill_(3)
    assert lib.tree_attn_linear_prefill(plan.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), states.data_ptr(), 2,
                                        none.data_ptr(), bad.data_ptr(), dec.data_ptr(), 2, 1, 128, 1.0, ws.data_ptr(),
                                        ws.numel(), None) == 0
    torch.cuda.synchronize()
    assert device_status() == TL.ERR_INVALID_SLOT and (states == 3).all()


@pytest.mark.parametrize("size", [300.0, 30000.0, 1e-9])
@pytest.mark.parametrize("values", [(0.585, 0.6), (0.65, 0.7), (0.58, 0.9), (0.5, 1.0)])
def test_prefill_of_large_and_small_inputs(cuda_device, values, size):
    """Scores and values far from 1: no power of the decay may take what lies between them out of the numbers' range.
    Bounds relative to the magnitudes, as above."""
    parent, seg, hq, hkv = [-1, 0, 0], [150, 129, 40], 4, 2
    N = sum(seg)
    q, k, v = draw(9, N, hq, hkv, 128, cuda_device, size)
    dec = decays(hkv, cuda_device, values)
    states = randn((4, hkv, 128, 128), cuda_device) * size * size
    start = [num(states[3]), None, None]
    o = TL.tree_linear_prefill(TreePlan(parent, seg), states, TL.StateSlots([3, -1, -1], [0, 1, 2], 4), q, k, v, dec, 0.088)
    want, end, mag, mass = OLN.from_states(parent, seg, num(q), num(k), num(v), num(dec), 0.088, start)
    wide = 2 if min(values) < 0.58 else 1
    assert torch.isfinite(o).all()
    assert (np.abs(num(o) - want) <= 2.0 ** -8 * np.abs(want) + (wide * 2.0 ** -8 + 2.0 ** -12) * mag).all()
    for u in range(3):
        assert (np.abs(num(states[u]) - end[u]) <= 2.0 ** -13 * mass[u]).all()


def from_states_64(parent, seg, q, k, v, dec, scale, start):
    """What ``oracle.linear.from_states`` gives, on the device: (o, states by node, the magnitudes of both), the tokens of a
    chunk of 128 at once, in 64 bits."""
    off, end, mass, hkv = OL.packed_layout(parent, seg)[1], {}, {}, k.shape[1]
    order, G, gam = OL.packed_layout(parent, seg)[0], q.shape[1] // hkv, dec.double()
    o, size = torch.empty(q.shape, dtype=torch.float64, device=q.device), torch.empty(q.shape, dtype=torch.float64, device=q.device)
    i = torch.arange(128, device=q.device)
    for u in order:
        if parent[u] >= 0:
            S, A = end[parent[u]], mass[parent[u]]
        else:
            S = start[u].double() if start[u] is not None else torch.zeros((hkv, 128, 128), dtype=torch.float64, device=q.device)
            A = S.abs()
        for t in range(off[u], off[u] + seg[u], 128):
            m = min(128, off[u] + seg[u] - t)
            Q = q[t:t + m].double().view(m, hkv, G, 128).permute(1, 2, 0, 3) * scale
            K, V = (x[t:t + m].double().transpose(0, 1) for x in (k, v))
            lag = i[:m, None] - i[None, :m]
            w = torch.where(lag >= 0, gam[:, None, None] ** lag.clamp_min(0), 0.0)
            P = (Q @ K[:, None].transpose(-1, -2)) * w[:, None]
            f = (gam[:, None] ** (i[:m] + 1))[:, None, :, None]
            o[t:t + m] = (P @ V[:, None] + f * (Q @ S[:, None])).permute(2, 0, 1, 3).reshape(m, -1, 128)
            size[t:t + m] = (P.abs() @ V.abs()[:, None] + f * (Q.abs() @ S.abs()[:, None])).permute(2, 0, 1, 3).reshape(m, -1, 128)
            left = (gam[:, None] ** (m - 1 - i[:m]))[..., None]
            S = (gam ** m)[:, None, None] * S + (K * left).transpose(1, 2) @ V
            A = (gam ** m)[:, None, None] * A + (K.abs() * left).transpose(1, 2) @ V.abs()
        end[u], mass[u] = S, A
    return o, end, size, mass


@pytest.mark.parametrize("hq,hkv,nodes,longest", [
    (8, 8, 90, 400), (40, 8, 31, 700), (64, 8, 40, 260), (64, 8, 140, 129), (40, 2, 300, 200), (16, 16, 70, 300), (152, 152, 4, 600),
    (20, 1, 420, 150), (5, 5, 100, 900), (48, 6, 53, 300)])
def test_outputs_of_many_chunks(cuda_device, hq, hkv, nodes, longest):
    """More chunks than CTAs of a kv-head, by far: whole chunks one after another, then a share of the q-heads of those that are
    left, where a CTA may begin and end within a chunk; short chunks among them.  Groups of 1, 5, 8 and 20 heads.
    States from as many as (longest / 128) chunks in three depths: the bounds above."""
    g = np.random.default_rng(hq * nodes)
    parent = [-1] + [int(g.integers(0, max(1, u // 2))) if u % 7 else -1 for u in range(1, nodes)]
    depth = []
    for u, p in enumerate(parent):
        if p >= 0 and depth[p] >= 2:
            parent[u] = p = 0
        depth.append(0 if p < 0 else depth[p] + 1)
    seg = [int(x) for x in np.exp(g.uniform(0, np.log(longest), nodes)).round()]
    seg[0] = longest
    N = sum(seg)
    q, k, v = draw(nodes, N, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (1.0, 0.9, 0.99, 0.62))
    states = randn((nodes + 2, hkv, 128, 128), cuda_device, 3) * 3
    slot_in = [nodes + u % 2 if p < 0 and u % 3 else -1 for u, p in enumerate(parent)]
    start = [states[s].clone() if s >= 0 else None for s in slot_in]
    o = TL.tree_linear_prefill(TreePlan(parent, seg), states, TL.StateSlots(slot_in, list(range(nodes)), nodes + 2), q, k, v, dec, 0.125)
    want, end, size, mass = from_states_64(parent, seg, q, k, v, dec, 0.125, start)
    for a in range(0, N, 4096):
        W = want[a:a + 4096]
        lim = 2.0 ** -8 * W.abs() + (2.0 ** -8 + 2.0 ** -12) * size[a:a + 4096] + 1e-30
        assert ((o[a:a + 4096].double() - W).abs() <= lim).all(), a
    for u in range(nodes):
        assert ((states[u].double() - end[u]).abs() <= 2.0 ** -13 * mass[u] + 1e-30).all(), u


def test_64_bit_form(cuda_device):
    """The form above against the oracle, token by token."""
    parent, seg = [-1, 0, 0, -1], [130, 17, 140, 9]
    q, k, v = draw(5, sum(seg), 4, 2, 128, cuda_device)
    dec = decays(2, cuda_device, (0.9, 0.62))
    S0 = randn((2, 128, 128), cuda_device)
    got = from_states_64(parent, seg, q, k, v, dec, 0.2, [S0, None, None, None])
    want = OLN.from_states(parent, seg, num(q), num(k), num(v), num(dec), 0.2, [num(S0), None, None, None])
    for a, b in ((got[0], want[0]), (got[2], want[2]), *((got[i][u], want[i][u]) for i in (1, 3) for u in range(4))):
        assert (np.abs(num(a) - b) <= 1e-11 * np.abs(b).max()).all()


def test_new_slots_do_not_wait_for_queued_work(cuda_device):
    """A fork is a new table: it comes to the device while what was launched before still runs, and stays there until its
    readers are done, on whatever stream they are."""
    R, hq, hkv = 5, 4, 2
    q, k, v = draw(33, R, hq, hkv, 128, cuda_device)
    dec, first = decays(hkv, cuda_device), randn((2 * R, hkv, 128, 128), cuda_device)
    fork = lambda x: TL.StateSlots(range(R), [R + (i + x) % R for i in range(R)], 2 * R)  # noqa: E731
    want = []
    for x in range(R):
        s = first.clone()
        want.append((TL.tree_linear_step(s, fork(x), q, k, v, dec, 0.1), s))
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    torch.cuda._sleep(400_000_000)                              # some 0.2 s
    done.record()
    fork(1).upload()
    assert not done.query()
    streams = [torch.cuda.Stream() for _ in range(R)]
    got = [first.clone() for _ in range(R)]
    torch.cuda.synchronize()
    for x, side in enumerate(streams):                          # each table dropped while its reader waits
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        if x % 2:
            TL.tree_linear_step(got[x], fork(x), q, k, v, dec, 0.1, stream=side)
        else:
            with torch.cuda.stream(side):
                TL.tree_linear_step(got[x], fork(x), q, k, v, dec, 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(got[x], want[x][1]) for x in range(R))


@pytest.mark.parametrize("hq,hkv", [(16, 16), (8, 8), (2, 2), (40, 2), (152, 152)])
def test_whole_and_short_chunks_in_turn(cuda_device, hq, hkv):
    """Single units of a chunk, whole chunks (128 tokens) before short ones: a short chunk's rows behind its last are set to
    zero in a buffer that the chunk before it has used.  Inputs that are in no cache, again and again the same bits, and
    those of the 64-bit form."""
    g = np.random.default_rng(hq)
    nodes = 240 if hkv < 100 else 12
    parent = [-1] + [int(g.integers(0, 3)) if u > 3 else 0 for u in range(1, nodes)]
    seg = [int(x) for x in g.choice([128, 256, 384, 1, 3, 17, 65, 130, 259, 385, 401], nodes)]
    N = sum(seg)
    q, k, v = draw(nodes + hq, N, hq, hkv, 128, cuda_device)
    dec = decays(hkv, cuda_device, (1.0, 0.62, 0.99, 0.3))
    first = randn((nodes + 1, hkv, 128, 128), cuda_device, 4)
    plan, slots = TreePlan(parent, seg), TL.StateSlots([nodes] + [-1] * (nodes - 1), list(range(nodes)), nodes + 1)
    cold = torch.empty(1 << 28, dtype=torch.uint8, device=cuda_device)
    states = first.clone()
    o = TL.tree_linear_prefill(plan, states, slots, q, k, v, dec, 0.1)
    for _ in range(12):
        again = first.clone()
        cold.zero_()
        assert torch.equal(TL.tree_linear_prefill(plan, again, slots, q, k, v, dec, 0.1), o) and torch.equal(again, states)
    want, end, size, mass = from_states_64(parent, seg, q, k, v, dec, 0.1, [first[nodes]] + [None] * (nodes - 1))
    # (a score is within 2^-16 of the sum of its products' magnitudes, which its own size may be far below)
    scores = from_states_64(parent, seg, q.abs(), k.abs(), v.abs(), dec, 0.1, [first[nodes].abs()] + [None] * (nodes - 1))[0]
    lim = 2.0 ** -8 * want.abs() + (2 * 2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -16 * scores
    assert ((o.double() - want).abs() <= lim).all()
    for u in range(nodes):
        assert ((states[u].double() - end[u]).abs() <= 2.0 ** -13 * mass[u] + 1e-30).all(), u
