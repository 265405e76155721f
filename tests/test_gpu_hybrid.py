"""A rollout of a hybrid model from its prompt to its update, as the calls are used together: a softmax layer
on the paged cache and a linear layer on states in slots; branches that grow token by token, one that
forks inside a page (its page copied, its state taken before the fork), pages compacted, then the policy loss of
the finished tree on the log-probs that were sampled.

The linear layer's states after every turn are held against the recursion on the same keys and values (fp32, so many
steps of 2^-23 each), the attention after the fork and the compaction against the training side's on the
cache's values (as in the other rollout test: 2e-2 + 2.1e-2), log-probs within 2^-13 (1 + |lp|)."""
import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan, device_status, tree_attn_fwd
from prefix_tree_attention_attn_gb300 import decode as TD
from prefix_tree_attention_attn_gb300 import linear as TLN
from prefix_tree_attention_attn_gb300 import loss as TL
from prefix_tree_attention_attn_gb300.sample import sample_tokens

pytestmark = pytest.mark.gpu

HQ, HKV, D, V, SCALE = 4, 2, 128, 1000, 0.08


class Model:
    """Queries, keys and values of a softmax layer and of a linear one by token, and logits of both outputs."""

    def __init__(self, dev):
        g = torch.Generator(dev).manual_seed(5)
        make = lambda *s: torch.randn(s, device=dev, generator=g).clamp(-4, 4).bfloat16()  # noqa: E731
        self.q, self.k, self.v = make(V, HQ, D), make(V, HKV, D), make(V, HKV, D)
        self.lq, self.lk, self.lv = make(V, HQ, D), make(V, HKV, D), make(V, HKV, D)
        self.out = make(2 * HQ * D, V) * 0.125
        self.decay = torch.tensor([0.95, 0.995], device=dev)

    def logits(self, o, ol):
        x = torch.cat([o.reshape(-1, HQ * D), torch.tanh(ol.reshape(-1, HQ * D).float() * 0.05).bfloat16()], 1)
        return x @ self.out


def recursion(m, tokens):
    S = torch.zeros((HKV, D, D), dtype=torch.float64, device=tokens.device)
    size = S.clone()
    g = m.decay.double()[:, None, None]
    for t in tokens.tolist():
        kv = m.lk[t].double()[:, :, None] * m.lv[t].double()[:, None, :]
        S, size = g * S + kv, g * size + kv.abs()
    return S, size


def test_rollout_and_update(lib, cuda_device):
    dev = cuda_device
    m, rng = Model(dev), np.random.default_rng(4)
    u = lambda n: torch.from_numpy(rng.random(n).astype(np.float32)).to(dev)  # noqa: E731
    layers = 2                                              # the softmax layer's cache twice, as two layers would have it
    pool, P = 30, TD.PagePool(30)
    caches = [TD.TreeCache.empty(pool, HKV, D, dev) for _ in range(layers)]
    states = torch.empty((6, HKV, D, D), device=dev)
    paths, tree = {}, {}                                    # tokens of each branch

    # the prompt: 100 tokens and the first of each of two branches
    prompt = torch.from_numpy(rng.integers(0, V, 102)).to(dev)
    seg, cap = [100, 1, 1], [100, 90, 90]
    pages = [P.alloc(-(-c // 64)) for c in cap]
    plan = TD.DecodePlan([-1, 0, 0], seg, [1, 2], HQ, HKV, D, capacity=cap, pages=np.concatenate(pages), n_pages=pool)
    for c in caches:
        TD.tree_cache_write(plan, c, m.k[prompt], m.v[prompt])
    lens = plan.lens()
    train = TreePlan([-1, 0, 0], seg)
    ol = TLN.tree_linear_prefill(train, states, TLN.StateSlots([-1, -1, -1], [0, 1, 2], 6), m.lq[prompt], m.lk[prompt],
                                 m.lv[prompt], m.decay, SCALE)
    o = torch.stack([TD.tree_decode(plan, caches[i], lens, m.q[prompt[100:]], SCALE)[0] for i in range(layers)])
    assert torch.equal(o[0], o[1])
    logits = m.logits(o[0], ol[100:])
    toks, lps = [prompt[100:].int()], []
    rows_logits = {(1, 0): logits[0], (2, 0): logits[1]}    # by (branch, position in it)
    slots = TLN.StateSlots([1, 2], [1, 2], 6)
    mid = None
    for step in range(70):
        t, lp = sample_tokens(logits, u(2), temperature=1.0, top_k=100)
        toks.append(t.clone())
        lps.append(lp.clone())
        lens = lens.clone()
        for i, c in enumerate(caches):
            TD.tree_cache_append(plan, c, lens if i == layers - 1 else lens.clone(), m.k[t], m.v[t])
        o, _ = TD.tree_decode(plan, caches[0], lens, m.q[t], SCALE)
        ol = TLN.tree_linear_step(states, slots, m.lq[t], m.lk[t], m.lv[t], m.decay, SCALE)
        logits = m.logits(o, ol)
        for b in (1, 2):
            rows_logits[(b, step + 1)] = logits[b - 1]
        if step == 39:                                      # 41 tokens in each branch: a state to come back to
            TLN.tree_linear_step(states, TLN.StateSlots([-1], [5], 6), m.lq[t[:1]], m.lk[t[:1]], m.lv[t[:1]], m.decay, SCALE)
            states[3].copy_(states[1])
            mid = logits[0].clone()
    seg = [100, 71, 71]
    assert lens.tolist() == seg
    one = torch.stack([t[0] for t in toks])                 # branch 1's 71 tokens
    S, size = recursion(m, torch.cat([prompt[:100], one]))
    assert ((states[1].double() - S).abs() <= (2.0 ** -13 + 72 * 2.0 ** -23) * size).all()

    # branch 1 forks at token 41, inside its first page: node 1 keeps no full page, node 3 what it had, node 4 the fork
    new = P.alloc(2)
    for c in caches:
        TD.tree_cache_copy(c, pages[1][:1], new[:1])
    parent2 = [-1, 0, 0, 0]                                 # 0 prompt, 1 old branch 1, 2 branch 2, 3 the fork from 41 tokens of it
    seg2, cap2 = [100, 71, 71, 41], [100, 90, 90, 128]
    pages2 = pages + [new]
    plan2 = TD.DecodePlan(parent2, seg2, [3], HQ, HKV, D, capacity=cap2, pages=np.concatenate(pages2), n_pages=pool)
    lens2, fork = plan2.lens(), [mid]
    t, lp = sample_tokens(mid[None], u(1), temperature=1.0, top_k=100)
    ftoks, flps = [t.clone()], [lp.clone()]
    go = TLN.StateSlots([3], [4], 6)                        # the state before the fork stays in slot 3
    for step in range(30):
        for i, c in enumerate(caches):
            TD.tree_cache_append(plan2, c, lens2 if i == layers - 1 else lens2.clone(), m.k[t], m.v[t])
        o, _ = TD.tree_decode(plan2, caches[0], lens2, m.q[t], SCALE)
        ol = TLN.tree_linear_step(states, go, m.lq[t], m.lk[t], m.lv[t], m.decay, SCALE)
        go = TLN.StateSlots([4], [4], 6) if step == 0 else go
        logits = m.logits(o, ol)
        fork.append(logits[0])
        if step < 29:
            t, lp = sample_tokens(logits, u(1), temperature=1.0, top_k=100)
            ftoks.append(t.clone())
            flps.append(lp.clone())
    seg2[3] = 71
    assert lens2.tolist() == seg2
    forked = torch.cat([one[:41], torch.cat(ftoks)])
    S, size = recursion(m, torch.cat([prompt[:100], forked]))
    assert ((states[4].double() - S).abs() <= (2.0 ** -13 + 72 * 2.0 ** -23) * size).all()
    S, size = recursion(m, torch.cat([prompt[:100], one[:41]]))
    assert ((states[3].double() - S).abs() <= (2.0 ** -13 + 72 * 2.0 ** -23) * size).all()

    # branch 2 is given up, the pool compacted; the fork's attention afterwards
    P.free(pages[2])
    ask = lambda pg: TD.DecodePlan([-1, 0, 0], [100, 71, 71], [1, 2], HQ, HKV, D, capacity=[100, 90, 128],  # noqa: E731
                                   pages=np.concatenate(pg), n_pages=pool)
    kept = [pages[0], pages[1], new]
    q = m.q[torch.stack([one[-1], forked[-1]]).long()]
    p3 = ask(kept)
    want = TD.tree_decode(p3, caches[1], p3.lens(), q, SCALE)
    src, dst, page = P.compact()
    assert len(src) == 2
    TD.tree_cache_copy(caches, src, dst)
    kept = [page[x] for x in kept]
    p3 = ask(kept)
    for c in caches:
        got = TD.tree_decode(p3, c, p3.lens(), q, SCALE)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    full = [100, 71, 71]
    deq = lambda x, s: (x.float() * s[:, :, None, None])  # noqa: E731
    kv = [(deq(caches[0].k, caches[0].k_scale)[torch.from_numpy(pg.astype(np.int64)).to(dev)].permute(0, 2, 1, 3).reshape(-1, HKV, D)[:n],
           deq(caches[0].v, caches[0].v_scale)[torch.from_numpy(pg.astype(np.int64)).to(dev)].permute(0, 3, 1, 2).reshape(-1, HKV, D)[:n])
          for pg, n in zip(kept, full)]
    tok = torch.cat([prompt[:100].int(), one.int(), forked.int()])
    train = TreePlan([-1, 0, 0], full)
    o, _ = tree_attn_fwd(train, m.q[tok.long()], torch.cat([k for k, _ in kv]).bfloat16(), torch.cat([v for _, v in kv]).bfloat16(), SCALE)
    assert (o[[170, 241]].float() - got[0].float()).abs().max() <= 2e-2 + 2.1e-2

    # the update: the two branches that are left, weights on what was sampled (not on the tokens given)
    x = torch.zeros((242, V), dtype=torch.bfloat16, device=dev)
    x[100:171] = torch.stack([rows_logits[(1, i)] for i in range(71)])
    x[171:212] = x[100:141]                                 # the fork's copy of the shared tokens
    x[211:242] = torch.stack(fork)
    old = torch.zeros(2 * 170, device=dev)
    w = torch.zeros(2 * 170, device=dev)
    old[100:170], old[270:340] = torch.stack([p[0] for p in lps]), torch.cat([torch.stack([p[0] for p in lps[:40]]), torch.cat(flps)])
    w[100:170], w[270:340] = 1 / 140, 1 / 140
    adv, _, _ = TL.subtree_advantage(train, torch.tensor([1.0, 0.0], device=dev))
    r = TL.policy_loss(train, x, tok, old, adv, weights=w, ref_logprobs=old, kl_coef=0.1)
    live = w != 0
    _, again = TL.traj_logprobs(train, x, tok)
    assert (r.logprobs - again)[live].abs().max() <= 2.0 ** -12 * (1 + again.abs().max())
    assert (r.logprobs - old)[live].abs().max() <= 2.0 ** -13 * (1 + old.abs().max())
    # ratios of 1: the mean advantage, 0 here; the gradient is that of the advantages' weighted log-probs
    assert abs(float(r.loss)) <= 2.0 ** -11
    p = torch.softmax(x.double(), 1)
    want = torch.zeros((242, V), dtype=torch.float64, device=dev)
    for first, a in ((100, float(adv[0])), (171, float(adv[1]))):
        for i in range(70):
            want[first + i] += a / 140 * p[first + i]
            want[first + i, int(tok[first + i + 1])] -= a / 140
    err = (r.dlogits.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -12 / 140 * (p + 1)).all() and not r.dlogits[:100].any()
    assert device_status() == 0
