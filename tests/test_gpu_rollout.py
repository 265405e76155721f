"""The rollout calls together, as they are used: a tree's prompt is written to the
cache, its branches grow token by token (append, attention, logits, sampling) as one
captured graph, then branch again with a new plan over the same pages; the training
side's calls on the finished tree give the same attention and log-probs.

Tolerances.  Attention of the training side over the decoded cache's values (bf16 holds a
code times a power of two exactly): its own bound, 2e-2, plus the decode's for |v| <= 4.5:
2^-8 |o| + (2^-11 + 2^-13) |v| + 2^-15 for the rest < 2.1e-2.  A page that grew after the
step rounds codes below 2^-6 of its scale again, by 2^-18 of its largest value: inside
that 2^-15.  Log-probs: both are x - lse in fp32; a sum of V = 1,000 positive terms in any
order is within V * 2^-24 < 2^-14, terms and logarithm within 2^-20 (1 + |lse|): 2^-13.
"""
import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan, device_status, tree_attn_fwd
from prefix_tree_attention_attn_gb300 import decode as TD
from prefix_tree_attention_attn_gb300 import loss as TL
from prefix_tree_attention_attn_gb300.sample import sample_tokens

pytestmark = pytest.mark.gpu

HQ, HKV, D, V, SCALE = 8, 2, 64, 1000, 0.125


class Model:
    """One attention layer between an embedding and logits."""

    def __init__(self, dev):
        g = torch.Generator(dev).manual_seed(5)
        make = lambda *s: torch.randn(s, device=dev, generator=g).clamp(-4, 4).bfloat16()  # noqa: E731
        self.q, self.k, self.v = make(V, HQ, D), make(V, HKV, D), make(V, HKV, D)
        self.out = make(HQ * D, V) * 0.25

    def logits(self, o):
        return o.reshape(-1, HQ * D) @ self.out


def dequantised(cache, pages, n):
    """K, V [n, hkv, d] bf16 of a node's tokens."""
    k = (cache.k.float() * cache.k_scale[:, :, None, None])[pages].permute(0, 2, 1, 3).reshape(-1, HKV, D)
    v = (cache.v.float() * cache.v_scale[:, :, None, None])[pages].permute(0, 3, 1, 2).reshape(-1, HKV, D)
    return k[:n].bfloat16(), v[:n].bfloat16()


def test_rollout(lib, cuda_device):
    m, rng = Model(cuda_device), np.random.default_rng(21)
    parent, seg, grow = [-1, 0, 0, 0], [100, 1, 1, 1], 80
    cap = [100] + [1 + grow] * 3
    at = np.cumsum([0] + [-(-c // 64) for c in cap])
    pool = 24
    pages = rng.permutation(pool)[:at[-1]].astype(np.int32)
    prompt = torch.from_numpy(rng.integers(0, V, 103)).to(cuda_device)        # the last three start a branch each
    u = torch.from_numpy(rng.random((grow, 3)).astype(np.float32)).to(cuda_device)

    def start():
        plan = TD.DecodePlan(parent, seg, [1, 2, 3], HQ, HKV, D, capacity=cap, pages=pages, n_pages=pool)
        cache, lens = TD.TreeCache.empty(pool, HKV, D, cuda_device), plan.lens()
        TD.tree_cache_write(plan, cache, m.k[prompt], m.v[prompt])
        tok = prompt[100:].int()
        o, lse = TD.tree_decode(plan, cache, lens, m.q[tok], SCALE)
        logits = m.logits(o)
        return plan, cache, lens, tok, o, logits

    def step(s, draw):
        plan, cache, lens, tok, o, logits = s
        t, lp = sample_tokens(logits, draw, temperature=0.9, top_k=200, top_p=0.95, min_p=0.001)
        TD.tree_cache_append(plan, cache, lens, m.k[t], m.v[t])
        o2, _ = TD.tree_decode(plan, cache, lens, m.q[t], SCALE)
        tok.copy_(t), o.copy_(o2), logits.copy_(m.logits(o2))
        return lp

    a, b = start(), start()
    seen = {"tok": [a[3].clone()], "o": [a[4].clone()], "logits": [a[5].clone()], "lp": []}
    draw = u[0].clone()
    b[0].upload()
    spare = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(spare, draw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lp_b = step(b, draw)
    for i in range(grow):
        seen["lp"].append(step(a, u[i]).clone())
        for n, x in zip(("tok", "o", "logits"), a[3:]):
            seen[n].append(x.clone())
        draw.copy_(u[i])
        g.replay()
        assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4]) and torch.equal(seen["lp"][-1], lp_b), i
    assert a[2].tolist() == [100, 81, 81, 81] and device_status() == 0
    assert (a[3] >= 0).all()

    # the training side on the finished tree, packed depth-first
    full = [100, 81, 81, 81]
    plan = TreePlan(parent, full)
    tok = torch.cat([prompt[:100].int()] + [torch.stack([t[r] for t in seen["tok"]]) for r in range(3)])
    kv = [dequantised(a[1], torch.from_numpy(pages[at[v]:at[v + 1]].astype(np.int64)).to(cuda_device), full[v]) for v in range(4)]
    k, v = (torch.cat([x[i] for x in kv]).contiguous() for i in (0, 1))
    o, _ = tree_attn_fwd(plan, m.q[tok].contiguous(), k, v, SCALE)
    ours = torch.cat([torch.stack([x[r] for x in seen["o"]]) for r in range(3)])
    assert (o[100:].float() - ours.float()).abs().max() <= 2e-2 + 2.1e-2
    logits = torch.zeros((len(tok), V), dtype=torch.bfloat16, device=cuda_device)
    logits[100:] = torch.cat([torch.stack([x[r] for x in seen["logits"]]) for r in range(3)])
    _, lp = TL.traj_logprobs(plan, logits, tok.contiguous())
    per = lp.reshape(3, 180)[:, 100:]                    # after the first token of the branch
    got = torch.stack(seen["lp"]).T
    assert (per - got).abs().max() <= 2.0 ** -13 * (1 + got.abs().max())

    # branch: two children under node 1, one under node 3, five tokens each brought in
    parent2, now = parent + [1, 1, 3], full + [5, 5, 5]
    cap2 = cap + [64] * 3
    free = np.setdiff1d(np.arange(pool), pages)[:3].astype(np.int32)
    plan2 = TD.DecodePlan(parent2, now, [4, 5, 6, 2], HQ, HKV, D, capacity=cap2, pages=np.concatenate([pages, free]),
                          n_pages=pool, fresh=[False] * 4 + [True] * 3)
    new = torch.from_numpy(rng.integers(0, V, 15)).to(cuda_device)
    TD.tree_cache_write(plan2, a[1], m.k[new], m.v[new])
    last = torch.stack([new[4], new[9], new[14], a[3][1].long()])
    o2, _ = TD.tree_decode(plan2, a[1], plan2.lens(), m.q[last], SCALE)
    train = TreePlan(parent2, now)                       # depth-first: 0, 1, 4, 5, 2, 3, 6
    kv += [dequantised(a[1], torch.tensor([int(p)], device=cuda_device), 5) for p in free]
    order = [0, 1, 4, 5, 2, 3, 6]
    k, v = (torch.cat([kv[n][i] for n in order]).contiguous() for i in (0, 1))
    q = torch.zeros((sum(now), HQ, D), dtype=torch.bfloat16, device=cuda_device)
    ends = np.cumsum([now[n] for n in order]) - 1
    rows = [int(ends[order.index(n)]) for n in (4, 5, 6, 2)]
    q[rows] = m.q[last]
    o, _ = tree_attn_fwd(train, q, k, v, SCALE)
    assert (o[rows].float() - o2.float()).abs().max() <= 2e-2 + 2.1e-2
    assert (o2[3].float() - a[4][1].float()).abs().max() <= 2 * 2.1e-2      # an untouched branch answers as before
    assert device_status() == 0


def test_first_call_of_a_plan_on_a_side_stream(lib, cuda_device):
    """A plan's tables are in place when its first call, on a stream that does not wait for
    the default one, reads them: fresh plans of every kind, each against one used before."""
    from prefix_tree_attention_attn_gb300.linear import tree_linear_fwd
    g = torch.Generator(cuda_device).manual_seed(8)
    make = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    parent, seg, leaves = [-1] + [0] * 30, [500] + [90 + 7 * i for i in range(30)], range(1, 31)
    n = sum(seg)
    q, k, v, q1, logits = make(n, 4, 128), make(n, 2, 128), make(n, 2, 128), make(30, 4, 128), make(n, 504)
    tokens = torch.randint(0, 504, (n,), device=cuda_device, generator=g, dtype=torch.int32)
    decay = torch.tensor([0.9, 0.99], device=cuda_device)
    first = TD.DecodePlan(parent, seg, leaves, 4, 2, 128)
    cache, lens = TD.TreeCache.empty(first.n_pages, 2, 128, cuda_device), first.lens()
    TD.tree_cache_write(first, cache, k, v)
    side = torch.cuda.Stream()
    grow, train = lambda: TD.DecodePlan(parent, seg, leaves, 4, 2, 128), lambda: TreePlan(parent, seg)  # noqa: E731
    calls = ((grow, lambda p: TD.tree_decode(p, cache, lens, q1, 0.1, stream=side)),
             (train, lambda p: tree_attn_fwd(p, q, k, v, 0.1, stream=side)),
             (train, lambda p: (tree_linear_fwd(p, q, k, v, decay, 0.1, stream=side),)),
             (train, lambda p: TL.traj_logprobs(p, logits, tokens, stream=side)))
    for make_plan, call in calls:
        want = None
        for _ in range(20):
            torch.cuda.synchronize()
            plan = make_plan()
            got = call(plan)
            side.synchronize()
            want = got if want is None else want
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    want, plan = TD.tree_decode(first, cache, lens, q1, 0.1), grow()
    torch.cuda.synchronize()
    got = calls[0][1](plan)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and device_status() == 0


def test_side_stream_memory(lib, cuda_device):
    """On a side stream, what a call allocates is no block that the current stream may still
    write, and what the caller frees after the call is not handed out while the stream has yet
    to read it.  (Addresses only: nothing is overwritten.)"""
    g = torch.Generator(cuda_device).manual_seed(9)
    make = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    seg, R, hq, hkv, d, vocab = [640] + [70] * 64, 64, 32, 2, 128, 20000
    plan = TD.DecodePlan([-1] + [0] * R, seg, range(1, R + 1), hq, hkv, d, capacity=[640] + [200] * R)
    cache, lens = TD.TreeCache.empty(plan.n_pages, hkv, d, cuda_device), plan.lens()
    TD.tree_cache_write(plan, cache, make(sum(seg), hkv, d), make(sum(seg), hkv, d))
    plan.upload()
    q0, logits0, u0 = make(R, hq, d), make(R, vocab), torch.rand(R, device=cuda_device, generator=g)
    want = (*TD.tree_decode(plan, cache, lens, q0, 0.1), *sample_tokens(logits0, u0, top_p=0.9))
    side = torch.cuda.Stream()
    shapes = [(x.shape, x.dtype) for x in want] + [((plan.workspace_bytes,), torch.uint8)]
    for _ in range(3):
        q, logits, u, k, v, n = q0.clone(), logits0.clone(), u0.clone(), make(R, hkv, d), make(R, hkv, d), lens.clone()
        torch.cuda.synchronize()
        freed = [torch.empty(s, dtype=t, device=cuda_device) for s, t in shapes]
        mine = [(x.data_ptr(), x.data_ptr() + x.numel() * x.element_size()) for x in freed]
        del freed
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)                  # some 50 ms: the calls are still to come
        got = (*TD.tree_decode(plan, cache, n, q, 0.1, stream=side), *sample_tokens(logits, u, top_p=0.9, stream=side))
        TD.tree_cache_append(plan, cache, n, k, v, stream=side)
        for x in got:
            assert not any(a <= x.data_ptr() < b for a, b in mine)
        held = {x.data_ptr(): (x.shape, x.dtype) for x in (q, logits, u, k, v, n)}
        del q, logits, u, k, v, n
        again = [torch.empty(s, dtype=t, device=cuda_device) for s, t in list(held.values()) * 2]
        assert not side.query()                             # still to come
        assert not {x.data_ptr() for x in again} & set(held)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and device_status() == 0


def test_side_stream_inside_a_capture(lib, cuda_device):
    """A captured step whose attention and draw run on two streams at once, with outputs and
    workspace made inside the calls: replays give the eager results."""
    g = torch.Generator(cuda_device).manual_seed(10)
    make = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    seg = [640] + [70] * 20
    plan = TD.DecodePlan([-1] + [0] * 20, seg, range(1, 21), 16, 2, 128)
    cache, lens = TD.TreeCache.empty(plan.n_pages, 2, 128, cuda_device), plan.lens()
    TD.tree_cache_write(plan, cache, make(sum(seg), 2, 128), make(sum(seg), 2, 128))
    plan.upload()
    q, logits, u = make(20, 16, 128), make(20, 30000), torch.rand(20, device=cuda_device, generator=g)
    side, out = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        for _ in range(3):
            out += [*TD.tree_decode(plan, cache, lens, q, 0.1, stream=side), *sample_tokens(logits, u, 0.9, 50)]
            out += [*TD.tree_decode(plan, cache, lens, q, 0.1), *sample_tokens(logits, u, 0.9, 50, stream=side)]
        now.wait_stream(side)
    for _ in range(3):
        q.copy_(make(20, 16, 128)), logits.copy_(make(20, 30000)), u.copy_(torch.rand(20, device=cuda_device, generator=g))
        for x in out:
            x.fill_(7)
        graph.replay()
        want = [*TD.tree_decode(plan, cache, lens, q, 0.1), *sample_tokens(logits, u, 0.9, 50)]
        assert len(out) == 24 and all(torch.equal(a, want[i % 4]) for i, a in enumerate(out))
    assert device_status() == 0
