"""Workloads of a rollout-to-update cycle of a hybrid model on rollout trees: linear
attention from and to states in slots (whole turns, single tokens), pages of the
key/value cache copied for forks and compaction, and the clipped policy loss of the
finished tree with the gradient of its logits.

Each operator is written twice: in elementary torch operations, and as the calls
a program makes of the library (``own``).

Linear attention.  Per kv-head g with a decay gamma_g in (0, 1], along each root-to-leaf
path: S_j = gamma S_{j-1} + k_j v_j^T and O_i = scale q_i^T S_i.  States are fp32
[slot, kv-head, key feature, value feature].

Policy loss.  Prediction k of the trajectories (leaves by id, positions in order) is made by
a compact row r of logits x for the token y of the next position; lp = x_ry - LSE_r,
rho = exp(lp - old), H_r the row's entropy:

    loss = sum_k w_k (-min(rho A, clip(rho, 1 - lo, 1 + hi) A) + kl_coef (e^(ref - lp) - (ref - lp) - 1)
                      - entropy_coef H_r)

over the predictions with w_k != 0.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
CHUNK = 128
F8 = torch.float8_e4m3fn
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tree_case(kind, prompt, width, lo, hi, depth, shape):
    return {"kind": kind, "prompt": prompt, "width": width, "lo": lo, "hi": hi, "depth": depth, "shape": shape}


TINY = _tree_case("binary", 64, 4, 32, 32, 2, 1)             # the tiny binary tree, 256 tokens
SEGMENTS = _tree_case("binary", 512, 16, 256, 256, 4, 3)      # binary segments of 256 tokens, 16 leaves
STAR = _tree_case("star", 1024, 16, 256, 1024, 1, 2)          # one prompt, 16 responses
TURN = _tree_case("star", 777, 0, 1, 1, 1, 1)                 # one tool answer of 777 tokens
LONG = _tree_case("chains", 32768, 64, 1024, 8192, 3, 5)      # a long shared context with 64 chains


def listed():
    return [
        # a tiny tree with a small vocabulary: latency
        {"name": "policy tiny binary", "op": "policy", **TINY, "vocab": 1000, "per_token": False, "kl": 0.0,
         "entropy": 0.0, "masked": False, "grad": True},
        # a segment tree, advantage per token, no reference model, entropy bonus
        {"name": "policy segment tree", "op": "policy", **SEGMENTS, "vocab": 32000, "per_token": True, "kl": 0.0,
         "entropy": 0.01, "masked": True, "grad": True},
        # one prompt with 16 responses and the full vocabulary: an update of a group; the prompt is no target
        {"name": "policy group star", "op": "policy", **STAR, "vocab": 152064, "per_token": False, "kl": 0.04,
         "entropy": 0.0, "masked": True, "grad": True},
        # the same rollouts' loss, log-probs and entropies without a gradient, as between updates
        {"name": "policy group star value", "op": "policy", **STAR, "vocab": 152064, "per_token": False, "kl": 0.04,
         "entropy": 0.0, "masked": True, "grad": False},
        # one tool answer joins a branch that has a state
        {"name": "prefill one turn", "op": "prefill", **TURN, "hq": 32, "hkv": 8, "entered": True},
        # a prompt and the responses brought in, every leaf's state kept
        {"name": "prefill group star", "op": "prefill", **STAR, "hq": 32, "hkv": 8, "entered": False},
        # the prefill of the long shared context, 64/8 heads
        {"name": "prefill long context", "op": "prefill", **LONG, "hq": 64, "hkv": 8, "entered": False},
        # one token of one branch: latency
        {"name": "step 1", "op": "step", "rows": 1, "forked": 0, "hq": 32, "hkv": 8, "d": 128},
        # 64 branches, 16 of them just forked
        {"name": "step 64", "op": "step", "rows": 64, "forked": 16, "hq": 64, "hkv": 8, "d": 128},
        # 1,024 rollouts in flight
        {"name": "step 1024", "op": "step", "rows": 1024, "forked": 0, "hq": 32, "hkv": 8, "d": 128},
        # 16 branches fork inside a page, in the caches of 32 layers
        {"name": "fork 16 in 32 layers", "op": "copy", "pages": 16, "pool": 64, "layers": 32, "hkv": 8, "d": 128},
        # a pool is compacted: 2,000 pages move down
        {"name": "compact 2000", "op": "copy", "pages": 2000, "pool": 6000, "layers": 1, "hkv": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["policy", "policy", "prefill", "prefill", "step", "copy"])
    if op == "step":
        hq, hkv, d = rng.choice([(2, 2, 64), (32, 8, 128), (64, 8, 128), (8, 1, 128), (12, 4, 64), (14, 2, 128),
                                 (16, 16, 128), (40, 2, 128)])
        rows = _log_int(rng, 1, 8192 // max(hkv, hq // 4))
        return {"op": op, "rows": rows, "forked": rng.randint(0, rows), "hq": hq, "hkv": hkv, "d": d}
    if op == "copy":
        hkv, d = rng.choice([(2, 64), (8, 128), (1, 128), (4, 64), (16, 128)])
        pages = _log_int(rng, 1, 16000 // hkv)
        layers = rng.choice([1, 1, 2, 7, 32])
        pages = max(1, pages // layers)
        return {"op": op, "pages": pages, "pool": 2 * pages + rng.randint(0, pages), "layers": layers, "hkv": hkv,
                "d": d}
    hi = _log_int(rng, 1, 2048)
    kind = rng.choice(["star", "binary", "chains", "irregular"])
    width = {"star": _log_int(rng, 1, 64), "binary": 2 ** rng.randint(0, 5), "chains": _log_int(rng, 1, 32),
             "irregular": _log_int(rng, 2, 60)}[kind]
    case = {"op": op, **_tree_case(kind, _log_int(rng, 1, 8000), width, _log_int(rng, 1, hi), hi,
                                   int(math.log2(width)) if kind == "binary" else rng.randint(1, 4),
                                   rng.randint(0, 10 ** 6))}
    if op == "prefill":
        hq, hkv = rng.choice([(2, 2), (32, 8), (64, 8), (8, 1), (14, 2), (16, 16), (40, 2)])
        return {**case, "hq": hq, "hkv": hkv, "entered": rng.random() < 0.5}
    most = max(500, min(152064, 1600000000 // sum(_tree(case)[1])))
    return {**case, "vocab": _log_int(rng, 500, most), "per_token": rng.random() < 0.5,
            "kl": rng.choice([0.0, 0.001, 0.04]), "entropy": rng.choice([0.0, 0.0, 0.01]),
            "masked": rng.random() < 0.7 and width > 1, "grad": rng.random() < 0.8}


# ---------------------------------------------------------------------------
# trees and inputs
# ---------------------------------------------------------------------------

def _tree(case):
    """(parent, tokens per node)."""
    rng = np.random.default_rng(case["shape"])
    lo, hi, width = case["lo"], case["hi"], case["width"]
    length = lambda: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    parent, seg = [-1], [case["prompt"]]
    if case["kind"] == "star":
        for _ in range(width):
            parent.append(0)
            seg.append(length())
    elif case["kind"] == "binary":
        level = [0]
        for _ in range(case["depth"]):
            grown = []
            for u in level:
                for _ in range(2):
                    grown.append(len(parent))
                    parent.append(u)
                    seg.append(length())
            level = grown
    elif case["kind"] == "chains":
        for _ in range(width):
            u = 0
            for _ in range(int(rng.integers(1, case["depth"] + 1))):
                parent.append(u)
                seg.append(length())
                u = len(parent) - 1
    else:
        depth = [0]
        for _ in range(width - 1):
            u = int(rng.choice([v for v in range(max(0, len(parent) - 24), len(parent)) if depth[v] < case["depth"]]
                               or [0]))
            depth.append(depth[u] + 1)
            parent.append(u)
            seg.append(length())
    return parent, seg


def _packed(parent, seg):
    """(nodes in depth-first pre-order, children by ascending id; first row of each node)."""
    kids = [[] for _ in parent]
    for v, p in enumerate(parent):
        if p >= 0:
            kids[p].append(v)
    order, stack = [], [v for v in range(len(parent) - 1, -1, -1) if parent[v] < 0]
    while stack:
        v = stack.pop()
        order.append(v)
        stack.extend(reversed(kids[v]))
    off = np.zeros(len(parent), np.int64)
    off[order] = np.cumsum([0] + [seg[v] for v in order])[:-1]
    return order, off


def _path(parent, u):
    nodes = []
    while u >= 0:
        nodes.append(u)
        u = parent[u]
    return nodes[::-1]


def _predictions(parent, seg):
    """(row, target row, trajectory) of every prediction; the leaves by id."""
    off = _packed(parent, seg)[1]
    inner = set(parent)
    row, target, traj = [], [], []
    leaves = [v for v in range(len(parent)) if v not in inner]
    for l, leaf in enumerate(leaves):
        at = np.concatenate([np.arange(off[v], off[v] + seg[v]) for v in _path(parent, leaf)])
        row.append(at[:-1])
        target.append(at[1:])
        traj.append(np.full(len(at) - 1, l))
    return np.concatenate(row), np.concatenate(target), np.concatenate(traj), len(leaves)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _normal(g, *shape):
    """bf16 normals, a slab of rows at a time."""
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    slab = max(1, (1 << 28) // max(1, x[0].numel()))
    for i in range(0, len(x), slab):
        x[i:i + slab] = torch.randn(x[i:i + slab].shape, generator=g, device=DEV)
    return x


def _cuda(a, dtype):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=DEV)


def _decay(hkv):
    """Memories of 16 tokens up to 8,192, and one head without decay."""
    g = 1 - 2.0 ** -np.linspace(4, 13, hkv)
    g[-1] = 1.0
    return _cuda(g, torch.float32)


def prepare(case, seed):
    return {"policy": _prepare_policy, "prefill": _prepare_prefill, "step": _prepare_step,
            "copy": _prepare_copy}[case["op"]](case, seed)


def _prepare_policy(case, seed):
    parent, seg = _tree(case)
    g, N, V = _gen(seed), sum(seg), case["vocab"]
    row, target, traj, L = _predictions(parent, seg)
    s = {"case": case, "row": _cuda(row, torch.int64), "target": _cuda(target, torch.int64),
         "traj": _cuda(traj, torch.int64)}
    s["tokens"] = torch.randint(0, V, (N,), generator=g, device=DEV, dtype=torch.int32)
    s["logits"] = _normal(g, N, V).mul_(2)
    y = s["tokens"][s["target"]].long()
    s["logits"][s["row"], y] = (_rand(g, N) * 2 + 9).bfloat16()[s["row"]]    # what was sampled is likely
    lse = torch.cat([torch.logsumexp(x.float(), 1) for x in s["logits"].split(2048)])
    lp = s["logits"][s["row"], y].float() - lse[s["row"]]
    s["old"] = lp + 0.15 * _rand(g, len(row))                               # of the policy that sampled
    s["ref"] = lp + 0.3 * _rand(g, len(row)) if case["kl"] else None
    s["adv"] = _rand(g, len(row) if case["per_token"] else L)
    w = torch.full((len(row),), 1.0 / max(1, len(row)), device=DEV)
    if case["masked"]:                                                       # the root's tokens are no targets
        first = _packed(parent, seg)[1][0]
        w[(s["target"] >= first) & (s["target"] < first + seg[0])] = 0
    s["weights"] = w
    if own:
        from prefix_tree_attention_attn_gb300 import TreePlan

        s["plan"] = TreePlan(parent, seg)
    return s


def _prepare_prefill(case, seed):
    parent, seg = _tree(case)
    g, N, n = _gen(seed), sum(seg), len(parent)
    hq, hkv, d = case["hq"], case["hkv"], 128
    s = {"case": case, "scale": 1 / math.sqrt(d), "decay": _decay(hkv), "q": _normal(g, N, hq, d),
         "k": _normal(g, N, hkv, d), "v": _normal(g, N, hkv, d)}
    inner = set(parent)
    slot_in = [0 if p < 0 and case["entered"] else -1 for p in parent]      # the root goes on from a stored state
    slot_out, slots = [-1] * n, 1
    for v in range(n):
        if v not in inner:                                                  # the leaves decode next
            slot_out[v] = slots
            slots += 1
    s["slot_in"], s["slot_out"] = slot_in, slot_out
    s["states"] = _rand(g, slots, hkv, d, d) * 4
    # chunks of 128 tokens inside each node, for the plain form: their rows, and how many tokens lie
    # between a chunk's end and another chunk's start (a node's end) further down the same path
    order, off = _packed(parent, seg)
    rows, count, start, node, first = [], [], [], [], {}
    pos = {-1: 0}
    for v in order:
        base = pos[parent[v]]
        first[v] = len(rows)
        for a in range(0, seg[v], CHUNK):
            m = min(CHUNK, seg[v] - a)
            rows.append(np.where(np.arange(CHUNK) < m, off[v] + a + np.arange(CHUNK), N))
            count.append(m)
            start.append(base + a)
            node.append(v)
        pos[v] = base + seg[v]
    start, count, node = np.array(start), np.array(count), np.array(node)
    above = np.zeros((n, n), bool)                                          # above[v, u]: u is v or its ancestor
    for v in range(n):
        above[v, _path(parent, v)] = True
    place = np.arange(len(start)) - np.array([first[v] for v in node])
    before = above[node][:, node] & ((node[:, None] != node[None]) | (place[None] < place[:, None]))
    gap = start[:, None] - (start + count)[None]
    kept = [v for v in range(n) if slot_out[v] >= 0]
    end = np.array([pos[v] for v in kept])
    s["rows"], s["count"] = _cuda(np.stack(rows), torch.int64), _cuda(count, torch.int64)
    s["gap"] = _cuda(np.where(before, gap, -1), torch.int64)                # [chunk, chunk before it]
    s["end_gap"] = _cuda(np.where(above[kept][:, node], end[:, None] - (start + count)[None], -1), torch.int64)
    s["start"], s["end"], s["kept"] = _cuda(start, torch.int64), _cuda(end, torch.int64), _cuda([slot_out[v] for v in kept], torch.int64)
    if own:
        from prefix_tree_attention_attn_gb300 import TreePlan, linear

        s["plan"] = TreePlan(parent, seg)
        s["slots"] = linear.StateSlots(slot_in, slot_out, slots)
        s["workspace"] = torch.empty(linear.prefill_workspace(s["plan"], hkv, d), dtype=torch.uint8, device=DEV)
    return s


def _prepare_step(case, seed):
    g, R, hq, hkv, d = _gen(seed), case["rows"], case["hq"], case["hkv"], case["d"]
    pool, rng = R + R // 4 + 1, np.random.default_rng(seed)
    out = rng.permutation(pool)[:R]
    into, rest = out.copy(), np.setdiff1d(np.arange(pool), out)
    into[:case["forked"]] = rng.choice(rest, case["forked"])                # forks start from a state that stays
    s = {"case": case, "scale": 1 / math.sqrt(d), "decay": _decay(hkv), "into": _cuda(into, torch.int64),
         "out": _cuda(out, torch.int64), "states": _rand(g, pool, hkv, d, d), "q": _normal(g, R, hq, d),
         "k": _normal(g, R, hkv, d), "v": _normal(g, R, hkv, d)}
    if own:
        from prefix_tree_attention_attn_gb300 import linear

        s["slots"] = linear.StateSlots(into, out, pool)
    return s


def _prepare_copy(case, seed):
    g, P, L, hkv, d = _gen(seed), case["pool"], case["layers"], case["hkv"], case["d"]
    pages = np.random.default_rng(seed).permutation(P)[:2 * case["pages"]].astype(np.int32)
    codes = lambda *shape: (_normal(g, *shape) * 100).to(F8)  # noqa: E731
    scales = lambda: torch.exp2(torch.randint(-12, 3, (L, P, hkv), generator=g, device=DEV).float())  # noqa: E731
    s = {"case": case, "src": pages[:case["pages"]], "dst": pages[case["pages"]:], "k": codes(L, P, hkv, PAGE, d),
         "v": codes(L, P, hkv, d, PAGE), "ks": scales(), "vs": scales()}
    if own:
        from prefix_tree_attention_attn_gb300 import decode

        s["caches"] = [decode.TreeCache(s["k"][i], s["v"][i], s["ks"][i], s["vs"][i]) for i in range(L)]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

LOW, HIGH = 0.2, 0.28


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        from prefix_tree_attention_attn_gb300 import decode, linear, loss

        if op == "policy":
            r = loss.policy_loss(s["plan"], s["logits"], s["tokens"], s["old"], s["adv"], weights=s["weights"],
                                 ref_logprobs=s["ref"], per_token=case["per_token"], clip_low=LOW, clip_high=HIGH,
                                 kl_coef=case["kl"], entropy_coef=case["entropy"], grad=case["grad"])
            return {"loss": r.loss, "logprobs": r.logprobs, "entropy": r.entropy, "dlogits": r.dlogits}
        if op == "prefill":
            o = linear.tree_linear_prefill(s["plan"], s["states"], s["slots"], s["q"], s["k"], s["v"], s["decay"],
                                           s["scale"], workspace=s["workspace"])
            return {"o": o, "states": s["states"]}
        if op == "step":
            o = linear.tree_linear_step(s["states"], s["slots"], s["q"], s["k"], s["v"], s["decay"], s["scale"])
            return {"o": o, "states": s["states"]}
        decode.tree_cache_copy(s["caches"], s["src"], s["dst"])
        return {n: s[n] for n in ("k", "v", "ks", "vs")}
    if op == "policy":
        return _policy(s)
    if op == "prefill":
        return _prefill(s)
    if op == "step":
        return _step(s)
    src, dst = _cuda(s["src"], torch.int64), _cuda(s["dst"], torch.int64)
    for n in ("k", "v"):
        s[n].view(torch.uint8)[:, dst] = s[n].view(torch.uint8)[:, src]
    for n in ("ks", "vs"):
        s[n][:, dst] = s[n][:, src]
    return {n: s[n] for n in ("k", "v", "ks", "vs")}


def _policy(s):
    case, row, w = s["case"], s["row"], s["weights"].double()
    y = s["tokens"][s["target"]].long()
    N = len(s["tokens"])
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, dtype=torch.float64)
    lse = top[:, 0].double() + total.log()
    live = w != 0
    seen = torch.zeros(N, dtype=torch.bool, device=x.device).index_put_((row[live],), live[live])
    h = torch.where(seen, lse - (e * x).sum(1, dtype=torch.float64) / total, 0)
    # 64 bits per prediction: a ratio may stand next to the border of the clip
    lp = torch.where(live, x[row, y].double() - lse[row], 0)
    a = s["adv"].double() if case["per_token"] else s["adv"].double()[s["traj"]]
    ratio = torch.exp(lp - s["old"].double())
    clipped = ratio.clamp(1 - LOW, 1 + HIGH)
    each = -torch.minimum(ratio * a, clipped * a) - case["entropy"] * h[row]
    grad = torch.where(ratio * a <= clipped * a, -ratio * a, 0)
    if case["kl"]:
        far = s["ref"].double() - lp
        each = each + case["kl"] * (torch.exp(far) - far - 1)
        grad = grad + case["kl"] * (1 - torch.exp(far))
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    out = {"loss": torch.where(live, w * each, zero).sum().float(), "logprobs": lp.float(), "entropy": h.float(),
           "dlogits": None}
    if case["grad"]:
        grad = torch.where(live, w * grad, zero)
        by_row = lambda v: torch.zeros(N, dtype=torch.float64, device=x.device).index_add_(0, row, v)  # noqa: E731
        d = e * (-by_row(grad) / total).float()[:, None]
        if case["entropy"]:
            factor = (case["entropy"] * by_row(w) / total).float()[:, None]
            d += e * factor * (x + (h - lse).float()[:, None])
        d.index_put_((row, y), grad.float(), accumulate=True)
        out["dlogits"] = d.bfloat16()
    return out


def _prefill(s):
    hq, hkv = s["case"]["hq"], s["case"]["hkv"]
    pad = lambda t: torch.cat([t.float(), torch.zeros_like(t[:1], dtype=torch.float32)])[s["rows"]]  # noqa: E731
    q, k, v = pad(s["q"]), pad(s["k"]), pad(s["v"])                          # [chunk, 128, heads, d]
    C = len(q)
    # powers of the decay from exponents in 64 bits
    lg = s["decay"].double().log()[:, None, None]
    power = lambda n: torch.where(n >= 0, torch.exp(lg * n.clamp_min(0)), 0).float()  # noqa: E731
    i = torch.arange(CHUNK, device=q.device)
    left = power((s["count"][:, None] - 1 - i))                              # [hkv, chunk, 128]
    grown = torch.einsum("cmgk,cmgv->gckv", k * left.permute(1, 2, 0)[..., None], v).reshape(hkv, C, -1)
    entered = s["states"][0].reshape(hkv, 1, -1) if s["case"]["entered"] else 0
    start = power(s["start"][:, None])                                       # [hkv, chunk, 1]
    state = (torch.matmul(power(s["gap"]), grown) + start * entered).view(hkv, C, 128, 128)
    q = q.view(C, CHUNK, hkv, hq // hkv, 128) * s["scale"]
    o = torch.einsum("cmghk,gckv->cmghv", q, state) * power(i[None] + 1)[:, 0].t()[None, :, :, None, None]
    p = torch.einsum("cmghk,cngk->cghmn", q, k)
    p *= power(i[:, None] - i[None])[None, :, None]
    o += torch.einsum("cghmn,cngv->cmghv", p, v)
    flat = o.reshape(C * CHUNK, hq, 128)[(i[None] < s["count"][:, None]).reshape(-1)]
    order = s["rows"].reshape(-1)[(i[None] < s["count"][:, None]).reshape(-1)]
    out = torch.empty_like(s["q"])
    out[order] = flat.bfloat16()
    last = torch.matmul(power(s["end_gap"]), grown) + power(s["end"][:, None]) * entered
    s["states"][s["kept"]] = last.view(hkv, -1, 128, 128).transpose(0, 1)
    return {"o": out, "states": s["states"]}


def _step(s):
    hkv, d = s["k"].shape[1:]
    state = s["states"][s["into"]] * s["decay"][:, None, None] + s["k"].float()[..., None] * s["v"].float()[:, :, None]
    q = s["q"].float().view(len(state), hkv, -1, d)
    s["states"][s["out"]] = state
    return {"o": (torch.matmul(q, state) * s["scale"]).view(s["q"].shape).bfloat16(), "states": s["states"]}


# ---------------------------------------------------------------------------
# work, and the operators in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "step":
        R, hq, hkv, d = case["rows"], case["hq"], case["hkv"], case["d"]
        sources = R - case["forked"] + min(case["forked"], R // 4 + 1)       # forks of one state read it once
        return {"bytes": 4 * (R + sources) * hkv * d * d + 2 * R * (2 * hq + 2 * hkv) * d,
                "flops": R * d * d * (3 * hkv + 2 * hq)}
    if case["op"] == "copy":
        page = 2 * case["hkv"] * (PAGE * case["d"] + 4)
        return {"bytes": 2 * case["layers"] * case["pages"] * page, "flops": 0}
    parent, seg = _tree(case)
    N = sum(seg)
    if case["op"] == "prefill":
        hq, hkv, d = case["hq"], case["hkv"], 128
        leaves = len(parent) - len(set(parent) - {-1})
        return {"bytes": 4 * N * (hq + hkv) * d + 4 * (leaves + case["entered"]) * hkv * d * d,
                "flops": 2 * N * d * d * (hq + hkv)}
    inner = set(parent)
    ends = [v for v in range(len(parent)) if v not in inner]
    rows = N - len(ends) - (seg[0] - 1 if case["masked"] else 0)             # rows of some weight
    preds = sum(sum(seg[v] for v in _path(parent, u)) - 1 for u in ends)
    return {"bytes": 2 * rows * case["vocab"] + 2 * N * case["vocab"] * case["grad"] + 20 * preds + 8 * N,
            "flops": 6 * rows * case["vocab"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"policy": _exact_policy, "prefill": _exact_prefill, "step": _exact_step, "copy": _exact_copy}[case["op"]](s)


def _exact_policy(s):
    """The loss of each row from its own predictions, the gradient by the chain rule, 256 rows at a time."""
    case, N = s["case"], len(s["tokens"])
    y = s["tokens"][s["target"]].long()
    a = (s["adv"] if case["per_token"] else s["adv"][s["traj"]]).double()
    w, old = s["weights"].double(), s["old"].double()
    lp, h = torch.zeros_like(w), torch.zeros(N, dtype=torch.float64, device=w.device)
    d = torch.zeros(s["logits"].shape, dtype=torch.float64, device=w.device) if case["grad"] else None
    total = torch.zeros((), dtype=torch.float64, device=w.device)
    order = torch.argsort(s["row"], stable=True)
    order = order[w[order] != 0]
    bound = torch.searchsorted(s["row"][order], torch.arange(0, N + 256, 256, device=w.device)).tolist()
    for b, r0 in enumerate(range(0, N, 256)):
        at = order[bound[b]:bound[b + 1]]
        if not len(at):
            continue
        rows, place = torch.unique(s["row"][at], return_inverse=True)
        logp = torch.log_softmax(s["logits"][rows].double(), 1)
        p = logp.exp()
        ent = -(p * logp).sum(1)
        l = logp[place, y[at]]
        ratio = (l - old[at]).exp()
        free = torch.where(a[at] > 0, ratio <= 1 + HIGH, ratio >= 1 - LOW)
        held = torch.where(a[at] > 0, torch.full_like(ratio, 1 + HIGH), torch.full_like(ratio, 1 - LOW))
        each = -a[at] * torch.where(free, ratio, held) - case["entropy"] * ent[place]
        dl = torch.where(free, -a[at] * ratio, torch.zeros_like(ratio))
        if case["kl"]:
            far = s["ref"][at].double() - l
            each += case["kl"] * (torch.expm1(far) - far)
            dl -= case["kl"] * torch.expm1(far)
        total += (w[at] * each).sum()
        lp[at] = l
        h[rows] = ent
        if case["grad"]:
            dl *= w[at]
            sums = torch.zeros((2, len(rows)), dtype=torch.float64, device=w.device)
            sums[0].index_add_(0, place, dl)
            sums[1].index_add_(0, place, w[at])
            block = case["entropy"] * sums[1][:, None] * p * (logp + ent[:, None]) - sums[0][:, None] * p
            block.index_put_((place, y[at]), dl, accumulate=True)
            d[rows] = block
    return {"loss": total, "logprobs": lp, "entropy": h, "dlogits": d}


def _exact_prefill(s):
    """Node after node, 64 tokens at a time: outputs and state advance together."""
    case = s["case"]
    parent, seg = _tree(case)
    hq, hkv, d = case["hq"], case["hkv"], 128
    order, off = _packed(parent, seg)
    g = s["decay"].double()
    states, left = s["states"].double(), {}
    waiting = [0] * len(parent)
    for p in parent:
        if p >= 0:
            waiting[p] += 1
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=g.device)
    i = torch.arange(64, device=g.device)
    for u in order:
        p = parent[u]
        if p >= 0:
            S = left[p]
            waiting[p] -= 1
            if not waiting[p]:
                del left[p]
        else:
            S = states[s["slot_in"][u]] if s["slot_in"][u] >= 0 else torch.zeros((hkv, d, d), dtype=torch.float64, device=g.device)
        for t in range(off[u], off[u] + seg[u], 64):
            m = int(min(64, off[u] + seg[u] - t))
            q = s["q"][t:t + m].double().view(m, hkv, -1, d).permute(1, 2, 0, 3) * s["scale"]      # [hkv, G, m, d]
            k, v = (s[n][t:t + m].double().transpose(0, 1) for n in ("k", "v"))                       # [hkv, m, d]
            lag = (i[:m, None] - i[None, :m])
            w = torch.where(lag >= 0, g[:, None, None] ** lag.clamp_min(0), 0.0)
            y = (q @ k[:, None].transpose(-1, -2) * w[:, None]) @ v[:, None]
            y += (g[:, None] ** (i[:m] + 1))[:, None, :, None] * (q @ S[:, None])
            o[t:t + m] = y.permute(2, 0, 1, 3).reshape(m, hq, d)
            S = (g ** m)[:, None, None] * S + (k * (g[:, None] ** (m - 1 - i[:m]))[..., None]).transpose(1, 2) @ v
        if waiting[u]:
            left[u] = S
        if s["slot_out"][u] >= 0:
            states[s["slot_out"][u]] = S
    return {"o": o, "states": states}


def _exact_step(s):
    """Head by head, from states that no pass has changed."""
    R, hkv, d = s["k"].shape
    G = s["q"].shape[1] // hkv
    states = s["states"].double()
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=states.device)
    new = []
    for h in range(hkv):
        k, v = s["k"][:, h].double(), s["v"][:, h].double()
        S = float(s["decay"][h]) * states[s["into"], h] + torch.einsum("rk,rv->rkv", k, v)
        for j in range(G):
            o[:, h * G + j] = s["scale"] * torch.einsum("rk,rkv->rv", s["q"][:, h * G + j].double(), S)
        new.append(S)
    for h in range(hkv):
        states[s["out"], h] = new[h]
    return {"o": o, "states": states}


def _exact_copy(s):
    """Page by page."""
    out = {n: s[n].clone() for n in ("k", "v", "ks", "vs")}
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for n in out:
            t = out[n].view(torch.uint8) if n in ("k", "v") else out[n]
            t[:, b] = t[:, a]
    return {"k": out["k"].float(), "v": out["v"].float(), "ks": out["ks"].double(), "vs": out["vs"].double()}
