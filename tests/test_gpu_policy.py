"""The clipped policy loss and its gradient (include/tree_loss.h) against the oracle.

Tolerances, from the arithmetic.  e^(x - m) is within 2^-22 + |x - m| 2^-24 of itself (at most
2^-21 where it counts: e^-a a < 1), a sum of at most 8 * 10 terms in a row, then 9 pairwise, is within
89 * 2^-24; ln S is then within 2^-17 and its own rounding, and a log-prob within
2^-17 + 2^-23 |lp|, an entropy within 2^-16 (1 + H).  A ratio or e^(ref - lp) is within 2^-16 of
itself, so the loss is within 2^-15 of the sum of its terms' magnitudes.  A gradient is within
2^-15 of the magnitudes that make it up (the oracle's bound) before its one rounding to bf16, 2^-8 of
itself.  Ratios are drawn at least 0.05 away from the clip's borders."""
import numpy as np
import pytest
import torch

from oracle import layout as OL
from oracle import loss as OLS
from prefix_tree_attention_attn_gb300 import TreePlan, build as _build, device_status
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import loss as TL
from prefix_tree_attention_attn_gb300.sample import sample_tokens

pytestmark = pytest.mark.gpu

STAR40 = ([-1] + [0] * 40, [6] + [1 + i % 3 for i in range(40)])                  # 40 predictions a root row, 40 children
MIXED = ([-1, 0, 0, 1, 1, 3, -1], [4, 3, 2, 1, 2, 1, 3])                          # a forest, branches in branches
WIDE = ([-1, 0] + [1] * 35 + [0], [3, 4] + [1] * 35 + [2])                        # 35 through an inner node, one beside


@pytest.fixture(autouse=True)
def _lib(lib, cuda_device):
    yield
    torch.cuda.synchronize()
    assert device_status() == 0


def make(tree, V, seed, per_token=False, zero=0.5, masked=0.0, same=False):
    parent, seg = tree
    g = np.random.default_rng(seed)
    N, L = sum(seg), len(OL.leaves(parent))
    n = sum(len(i) for _, i in OL.trajectories(parent, seg)) - L
    tok = g.integers(0, min(V, 3) if same else V, N)
    x = torch.from_numpy(g.normal(size=(N, V)) * 2).bfloat16()
    if masked:
        hide = g.random((N, V)) < masked
        hide[:, tok] = False                              # (what is predicted keeps a probability)
        x[torch.from_numpy(hide)] = -float("inf")
    lp = OLS.traj_logprobs(parent, seg, x.double().numpy(), tok)
    f32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.float32))  # noqa: E731
    old = f32(lp - g.choice([-0.6, -0.1, 0.0, 0.1, 0.6], n))
    w = f32((g.random(n) - 0.2) * (g.random(n) >= zero))
    return x, torch.from_numpy(tok).int(), old, f32(g.normal(size=n if per_token else L)), w, f32(lp + 0.5 * g.normal(size=n))


def check(tree, data, got, per_token=False, use_old=True, use_w=True, scale=1.0, **kw):
    x, tok, old, adv, w, ref = data
    num = lambda t: t.double().cpu().numpy()  # noqa: E731
    loss, lp, ent, grad, bound = OLS.policy_loss(*tree, num(x), tok.numpy(), num(old) if use_old else None, num(adv),
                                                 weights=num(w) if use_w else None, ref=num(ref), per_token=per_token, **kw)
    H = ent.max(initial=0.0)
    assert np.abs(num(got.logprobs) - lp).max(initial=0) <= 2.0 ** -17 + 2.0 ** -23 * np.abs(lp).max(initial=0)
    assert np.abs(num(got.entropy) - ent).max() <= 2.0 ** -16 * (1 + H)
    # the magnitudes of the loss's terms: those of its gradient at the targets, and the penalties'
    ww = num(w) if use_w else np.full(len(lp), 1 / max(1, len(lp)))
    a = num(adv) if per_token else np.repeat(num(adv), [len(i) - 1 for _, i in OL.trajectories(*tree)])
    ratio = np.exp(lp - num(old)) if use_old else np.ones(len(lp))
    far = num(ref) - lp
    terms = np.abs(a) * np.maximum(ratio, 2) + kw.get("kl_coef", 0) * (np.exp(far) + np.abs(far) + 1) + kw.get("entropy_coef", 0) * (1 + H)
    assert abs(float(got.loss) - loss) <= 2.0 ** -15 * (np.abs(ww) * terms).sum() + 1e-30
    if got.dlogits is not None:
        e = np.abs(num(got.dlogits) - scale * grad)
        lim = 2.0 ** -8 * np.abs(scale * grad) + 2.0 ** -15 * abs(scale) * bound + 1e-38
        assert (e <= lim).all(), (np.unravel_index(np.argmax(e / lim), e.shape), (e / lim).max())


def run(tree, data, device, use_old=True, use_w=True, use_ref=True, plan=None, x=None, **kw):
    d = [t.to(device) for t in data]
    return TL.policy_loss(plan or TreePlan(*tree), d[0] if x is None else x, d[1], d[2] if use_old else None, d[3],
                          weights=d[4] if use_w else None, ref_logprobs=d[5] if use_ref else None, **kw)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 500, 1000, 4097, 20473, 20481, 50257])
def test_vocabularies(cuda_device, V):
    data = make(MIXED, V, V, zero=0.3)
    kw = dict(kl_coef=0.1, entropy_coef=0.02, clip_high=0.3)
    check(MIXED, data, run(MIXED, data, cuda_device, **kw), **kw)


@pytest.mark.parametrize("V", [152064, 262144])
def test_largest_vocabularies(cuda_device, V):
    tree = ([-1, 0, 0], [2, 2, 1])
    data = make(tree, V, 5, zero=0.0)
    kw = dict(kl_coef=0.1, entropy_coef=0.02)
    check(tree, data, run(tree, data, cuda_device, **kw), **kw)


@pytest.mark.parametrize("tree", [STAR40, MIXED, WIDE, ([-1], [1]), ([-1], [9]), ([-1, -1], [1, 1]), ([-1, 0, 0], [1, 1, 1])])
@pytest.mark.parametrize("same", [False, True])
def test_trees(cuda_device, tree, same):
    """Many predictions per row, many children per row, children with the same token."""
    for per_token in (False, True):
        data = make(tree, 300, 17 + per_token, per_token=per_token, same=same)
        check(tree, data, run(tree, data, cuda_device, per_token=per_token, kl_coef=0.05), per_token=per_token, kl_coef=0.05)


def test_options(cuda_device):
    data = make(WIDE, 700, 3)
    for use_old, use_w, kw in ((False, True, {}), (True, False, {}), (False, False, dict(entropy_coef=-0.1)),
                               (True, True, dict(clip_low=1.0, clip_high=float("inf"))),
                               (False, True, dict(clip_low=0.0, clip_high=0.0))):
        check(WIDE, data, run(WIDE, data, cuda_device, use_old=use_old, use_w=use_w, use_ref=False, **kw),
              use_old=use_old, use_w=use_w, **kw)
    got = run(WIDE, data, cuda_device, grad_scale=-0.25)
    check(WIDE, data, got, scale=-0.25)
    alone = run(WIDE, data, cuda_device, grad=False)
    assert alone.dlogits is None and torch.equal(alone.loss, got.loss)
    assert torch.equal(alone.logprobs, got.logprobs) and torch.equal(alone.entropy, got.entropy)


@pytest.mark.parametrize("V", [300, 30011])
def test_strides_alignments_and_in_place(cuda_device, V):
    """Rows that start anywhere, gradients that lie elsewhere in their vectors, or over the logits."""
    data = make(STAR40 if V < 1000 else MIXED, V, 8, same=True)
    tree = STAR40 if V < 1000 else MIXED
    N = sum(tree[1])
    want = run(tree, data, cuda_device, entropy_coef=0.01)
    check(tree, data, want, entropy_coef=0.01)
    for off, wide, d_off in ((1, V + 5, 0), (8, V + 16, 8), (3, V + 3, 6), (0, V + 1, 0)):
        room = torch.full((N, wide), 7.0, dtype=torch.bfloat16, device=cuda_device)
        x = room[:, off:off + V] if off + V <= wide else room[:, :V]
        x.copy_(data[0])
        back = torch.full((N, V + 9), 5.0, dtype=torch.bfloat16, device=cuda_device)
        out = back[:, d_off:d_off + V]
        got = run(tree, data, cuda_device, x=x, dlogits=out, entropy_coef=0.01)
        assert got.dlogits is out
        check(tree, data, got, entropy_coef=0.01)
        assert (back[:, :d_off] == 5).all() and (back[:, d_off + V:] == 5).all()
        got = run(tree, data, cuda_device, x=x, dlogits=x, entropy_coef=0.01)
        check(tree, data, got, entropy_coef=0.01)
        left = room.clone()
        left[:, off:off + V] = 7
        assert (left == 7).all()
    x = data[0].to(cuda_device)
    got = run(tree, data, cuda_device, x=x, dlogits=x, entropy_coef=0.01)
    assert torch.equal(x, want.dlogits) and torch.equal(got.loss, want.loss)


def test_masked_logits(cuda_device):
    for masked in (0.5, 0.999):
        data = make(MIXED, 5000, 4, masked=masked, zero=0.0)
        check(MIXED, data, run(MIXED, data, cuda_device, kl_coef=0.1, entropy_coef=0.1), kl_coef=0.1, entropy_coef=0.1)
    data[0][:, 1:] = torch.finfo(torch.bfloat16).min          # masks of the lowest value, the targets at -inf:
    data[1][:] = 0                                            # ratios of 0, nothing to learn from
    data[2][:] = 0
    data[0][:, 0] = -float("inf")
    got = run(MIXED, data, cuda_device, use_ref=False, entropy_coef=0.1)
    seen = got.entropy != 0
    assert (got.logprobs == -float("inf")).all() and (got.dlogits == 0).all() and seen.sum() == 12
    assert (got.entropy[seen] - np.log(4999)).abs().max() <= 2.0 ** -16 * 10
    w, a = data[4].double().numpy(), np.repeat(data[3].double().numpy(), [len(i) - 1 for _, i in OL.trajectories(*MIXED)])
    terms = w * (np.maximum(-0.8 * a, 0) - 0.1 * np.log(4999))
    assert abs(float(got.loss) - terms.sum()) <= 2.0 ** -15 * np.abs(terms).sum()


def test_one_token_left(cuda_device):
    """Masks of the lowest value everywhere else: probability 1, entropy 0, no gradient; and -inf likewise."""
    for low in (torch.finfo(torch.bfloat16).min, -float("inf")):
        data = make(MIXED, 5000, 4, zero=0.0)
        data[0][:, 1:] = low
        data[1][:] = 0
        data[2][:] = 0
        got = run(MIXED, data, cuda_device, use_ref=False, entropy_coef=0.1)
        assert (got.logprobs == 0).all() and (got.entropy == 0).all() and (got.dlogits == 0).all()


def test_rows_without_weight_are_not_read(cuda_device):
    """Whatever they hold: NaN logits, token ids, old log-probs and advantages of what has no weight."""
    tree = ([-1, 0, 0], [5, 4, 3])
    data = make(tree, 400, 9, zero=0.0)
    want = run(tree, data, cuda_device, kl_coef=0.1)
    x, tok, old, adv, w, ref = (t.clone() for t in data)
    n0 = 8                                                    # the first trajectory's predictions
    w[4:8] = 0                                                # its own rows: 5 .. 8 (the last predicts nothing)
    w[[0, n0 + 0]] = 0                                        # the root's first row, in both
    clean = run(tree, (x, tok, old, adv, w, ref), cuda_device, kl_coef=0.1)
    check(tree, (x, tok, old, adv, w, ref), clean, kl_coef=0.1)
    x[0] = float("nan")
    x[5:9] = float("inf")
    x[11] = float("nan")                                      # the second leaf's last token predicts nothing
    tok[[1, 6, 7, 8]] = torch.tensor([-1, 400, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    old[[0, 5, n0]] = float("nan")
    ref[[0, 6, n0]] = float("inf")
    got = run(tree, (x, tok, old, adv, w, ref), cuda_device, kl_coef=0.1)
    for a, b in zip(got, clean):
        assert torch.equal(a, b)
    assert not got.dlogits[[0, 5, 6, 7, 8, 11]].any() and want.dlogits[0].any()


def test_rows_without_a_distribution(cuda_device):
    """NaN, +inf or nothing but -inf in a row, and token ids out of range, give NaN there alone."""
    tree = ([-1], [8])
    data = make(tree, 3000, 10, zero=0.0)
    clean = run(tree, data, cuda_device)
    for how in range(4):
        x, tok = data[0].clone(), data[1].clone()
        if how == 3:
            tok[3] = 3000
        else:
            x[2, 2999 if how else slice(None)] = (-float("inf"), float("inf"), float("nan"))[how]
        got = run(tree, (x, tok, *data[2:]), cuda_device)
        assert torch.isnan(got.loss) and torch.isnan(got.logprobs[2]) and torch.isnan(got.dlogits[2]).all()
        keep = [0, 1, 3, 4, 5, 6, 7]
        assert torch.equal(got.dlogits[keep], clean.dlogits[keep])
        assert how == 3 or torch.isnan(got.entropy[2])


def test_gradient_against_differences(cuda_device):
    """Of the kernel's own loss, along random directions, steps of exact bf16 values."""
    g = torch.Generator().manual_seed(3)
    x, tok, old, adv, w, ref = make(WIDE, 40, 6, zero=0.0)
    x = (x * 8).round().clamp(-24, 24) / 8                    # multiples of 1/8: +-1/16 stays exact
    kw = dict(kl_coef=0.3, entropy_coef=0.2, clip_low=1.0, clip_high=float("inf"))
    data = (x, tok, old, adv, w, ref)
    d = run(WIDE, data, cuda_device, **kw).dlogits.double().cpu()
    h = 2.0 ** -4
    for _ in range(5):
        s = (torch.randint(0, 2, x.shape, generator=g) * 2 - 1) * (torch.rand(x.shape, generator=g) < 0.02)
        f = [float(run(WIDE, ((x + k * h * s).bfloat16(), *data[1:]), cuda_device, **kw).loss) for k in (2, 1, -1, -2)]
        slope = (8 * (f[1] - f[2]) - (f[0] - f[3])) / (12 * h)       # error of order h^4 times the fifth derivative
        exact = float((d * s).sum())
        size = float((d.abs() * s.abs()).sum())
        assert abs(slope - exact) <= 2.0 ** -7 * size + 2.0 ** -9 * float(w.abs().sum()), (slope, exact, size)


def test_reproducible_and_debug_build(cuda_device):
    data = make(STAR40, 20000, 12, same=True)
    a = run(STAR40, data, cuda_device, kl_coef=0.1, entropy_coef=0.01)
    for _ in range(3):
        b = run(STAR40, data, cuda_device, kl_coef=0.1, entropy_coef=0.01)
        assert all(torch.equal(u, v) for u, v in zip(a, b))
    with B.library(_build.build_library(debug=True)):
        b = run(STAR40, data, cuda_device, kl_coef=0.1, entropy_coef=0.01)
        torch.cuda.synchronize()
        assert device_status() == 0
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("V,N", [(300, 3000), (16001, 700), (33000, 900)])
def test_debug_build_of_many_rows(cuda_device, V, N):
    """Rows that share slots, with and without the gradient, in the build that checks its bounds."""
    g = torch.Generator(cuda_device).manual_seed(V)
    plan = TreePlan([-1, 0, 0], [N - 200, 100, 100])
    x = torch.randn((N, V), device=cuda_device, generator=g).bfloat16()
    tok = torch.randint(0, V, (N,), device=cuda_device, generator=g, dtype=torch.int32)
    adv = torch.tensor([1.0, -2.0], device=cuda_device)
    call = lambda grad: TL.policy_loss(plan, x, tok, None, adv, entropy_coef=0.1, grad=grad)  # noqa: E731
    want, alone = call(True), call(False)
    with B.library(_build.build_library(debug=True)):
        plan = TreePlan([-1, 0, 0], [N - 200, 100, 100])
        got, got_alone = call(True), call(False)
        torch.cuda.synchronize()
        assert device_status() == 0
    assert all(torch.equal(u, v) for u, v in zip(got, want)) and all(torch.equal(u, v) for u, v in zip(got_alone[:3], alone[:3]))
    assert all(torch.equal(u, v) for u, v in zip(alone[:3], want[:3]))


def test_on_sampled_tokens(cuda_device):
    """What sampling says of a token is its old log-prob: every ratio is 1, so the loss is minus the mean
    advantage and the gradient that of the log-probs."""
    tree = ([-1, 0, 0], [6, 5, 7])
    plan = TreePlan(*tree)
    x, tok, *_ = make(tree, 2000, 13)
    x = x.to(cuda_device)
    nxt, lp = sample_tokens(x, torch.rand(18, device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(6)), top_k=50)
    tok = tok.to(cuda_device)
    _, ptr, at = TL.trajectories(plan)
    rows = np.concatenate([at[ptr[i]:ptr[i + 1] - 1] for i in range(2)])
    targets = np.concatenate([at[ptr[i] + 1:ptr[i + 1]] for i in range(2)])
    keep = np.array([t != 11 for t in targets])               # the second child's first token is drawn beside the first's
    tok[torch.from_numpy(targets[keep]).long()] = nxt[torch.from_numpy(rows[keep]).long()]
    _, old = TL.traj_logprobs(plan, x, tok)
    drawn = lp[torch.from_numpy(rows).long().to(cuda_device)]
    assert (old - drawn)[torch.from_numpy(keep).to(cuda_device)].abs().max() <= 2.0 ** -13 * (1 + old.abs().max())
    adv = torch.tensor([1.0, -0.5], device=cuda_device)
    got = TL.policy_loss(plan, x, tok, old, adv)
    n = [10, 12]
    assert abs(float(got.loss) - -(n[0] - 0.5 * n[1]) / 22) <= 2.0 ** -10
    assert (got.logprobs - old).abs().max() <= 2.0 ** -12 * (1 + old.abs().max())


def test_capture_and_side_stream(cuda_device):
    data = [t.to(cuda_device) for t in make(WIDE, 9000, 14, same=True)]
    other = [t.to(cuda_device) for t in make(WIDE, 9000, 15, same=True)]
    plan, plan2 = TreePlan(*WIDE), TreePlan(*WIDE)
    call = lambda d, p=plan, **kw: TL.policy_loss(p, d[0], d[1], d[2], d[3], weights=d[4], ref_logprobs=d[5], kl_coef=0.1, **kw)  # noqa: E731
    want = [call(d) for d in (data, other)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(data, plan2, stream=side)                      # a plan's first call
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(got, want[0]))
    held = [t.clone() for t in data]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(held)
        again = call(held, grad=False)
    for d, w in ((other, want[1]), (data, want[0])):
        for a, b in zip(held, d):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(u, v) for u, v in zip(out, w))
        assert torch.equal(again.loss, w.loss)


def test_rows_behind_32_bit_offsets(cuda_device):
    """A row that starts beyond 2^32 bytes, element offsets beyond 2^31."""
    N, V = 17000, 152064
    tree = ([-1], [N])
    plan = TreePlan(*tree)
    x = torch.empty((N, V), dtype=torch.bfloat16, device=cuda_device)
    g = torch.Generator(cuda_device).manual_seed(2)
    for i in range(0, N, 2000):
        x[i:i + 2000] = torch.randn((min(2000, N - i), V), device=cuda_device, generator=g)
    tok = torch.randint(0, V, (N,), device=cuda_device, generator=g, dtype=torch.int32)
    w = torch.zeros(N - 1, device=cuda_device)
    rows = [0, 14123, 16998]
    w[rows] = 1
    adv = torch.tensor([2.0], device=cuda_device)
    d = TL.policy_loss(plan, x, tok, None, adv, weights=w).dlogits
    live = d.float().abs().amax(1) > 0
    assert torch.nonzero(live).flatten().tolist() == rows
    for r in rows:
        p = torch.softmax(x[r].double(), 0)
        p[int(tok[r + 1])] -= 1
        e = (d[r].double() - 2 * p).abs()
        assert (e <= 2.0 ** -8 * 2 * p.abs() + 2.0 ** -14 * p.abs()).all()


@pytest.mark.parametrize("V,stride,at", [(301, 301, 0), (301, 304, 0), (4001, 4100, 3), (300, 300, 5), (1000, 1013, 1)])
def test_new_gradients_of_padded_logits(cuda_device, V, stride, at):
    data = make(MIXED, V, 21)
    N = len(data[1])
    x = torch.empty(N * stride + at, dtype=torch.bfloat16, device=cuda_device).as_strided((N, V), (stride, 1), at)
    x.copy_(data[0])
    got, dense = run(MIXED, data, cuda_device, x=x, kl_coef=0.1), run(MIXED, data, cuda_device, kl_coef=0.1)
    check(MIXED, data, got, kl_coef=0.1)
    assert got.dlogits.shape == (N, V) and (got.dlogits.stride(0) - stride) % 8 == 0
    assert (got.dlogits.data_ptr() - x.data_ptr()) % 16 == 0
    assert (got.loss - dense.loss).abs() <= 2.0 ** -12


@pytest.mark.parametrize("V,N", [(1000, 20000), (6001, 9000), (9000, 6000), (33000, 4000), (100000, 1500), (152064, 2500)])
@pytest.mark.parametrize("branches", [False, True])
def test_many_rows(cuda_device, V, N, branches):
    """More rows than are under way at a time, by far; and the loss alone, its log-probs and its entropies are the
    same bits as with the gradient.  With a leaf at every third row: rows of two targets, most of them with more than 32
    predictions.  The same tolerances (ratios of 1: g is the advantage)."""
    if branches:
        N = min(N, 1500)
        parent = [-1] + [2 * (i // 2) for i in range(N // 3 * 2)]      # node 2 i has the children 2 i + 1, a leaf, and 2 i + 2
        tree = (parent, [2 - (i % 2) for i in range(len(parent))])
    else:
        tree = ([-1], [N])
    plan = TreePlan(*tree)
    N = plan.n_tokens
    g = torch.Generator(cuda_device).manual_seed(V + branches)
    x = torch.empty((N, V), dtype=torch.bfloat16, device=cuda_device)
    for i in range(0, N, 500):
        x[i:i + 500] = 2 * torch.randn((min(500, N - i), V), device=cuda_device, generator=g)
    tok = torch.randint(0, V, (N,), device=cuda_device, generator=g, dtype=torch.int32)
    _, ptr, at = TL.trajectories(plan)
    rows = torch.from_numpy(np.concatenate([at[a:b - 1] for a, b in zip(ptr, ptr[1:])])).long().to(cuda_device)
    to = torch.from_numpy(np.concatenate([at[a + 1:b] for a, b in zip(ptr, ptr[1:])])).long().to(cuda_device)
    n = len(rows)
    adv = torch.randn(n, device=cuda_device, generator=g)
    w = torch.rand(n, device=cuda_device, generator=g) * (rows % 5 != 3)       # (rows without any weight)
    ent = 0.01
    kw = dict(weights=w, per_token=True, entropy_coef=ent)
    got = TL.policy_loss(plan, x, tok, None, adv, **kw)
    alone = TL.policy_loss(plan, x, tok, None, adv, grad=False, **kw)
    assert all(torch.equal(u, v) for u, v in zip(got[:3], alone[:3]))

    W, A = w.double(), adv.double()
    each = torch.zeros(N, dtype=torch.float64, device=cuda_device)
    sum_w = each.clone().index_add_(0, rows, W)
    sum_g, size_g = each.clone().index_add_(0, rows, -W * A), each.clone().index_add_(0, rows, (W * A).abs())
    edge, edge_size = each.clone().index_add_(0, to, -W * A), each.clone().index_add_(0, to, (W * A).abs())
    parent_row = torch.full((N,), -1, dtype=torch.long, device=cuda_device)
    parent_row[to] = rows
    loss = terms = 0.0
    for i in range(0, N, 250):
        r = torch.arange(i, min(N, i + 250), device=cuda_device)
        logp = torch.log_softmax(x[r].double(), 1)
        p = logp.exp()
        H = -(p * logp).sum(1)
        H = torch.where(sum_w[r] != 0, H, 0.0)
        assert ((got.entropy[r] - H).abs() <= 2.0 ** -16 * (1 + H)).all()
        here = torch.nonzero((rows >= i) & (rows < i + 250)).flatten()
        lp = logp[rows[here] - i, tok[to[here]].long()] * (W[here] != 0)
        assert ((got.logprobs[here] - lp).abs() <= 2.0 ** -17 + 2.0 ** -23 * lp.abs()).all()
        loss += float((-W[here] * (A[here] + ent * H[rows[here] - i])).sum())
        terms += float((W[here] * (2 * A[here].abs() + ent * (1 + H[rows[here] - i]))).sum())
        want = -sum_g[r, None] * p + ent * sum_w[r, None] * p * (logp + H[:, None])
        bound = size_g[r, None] * p + ent * sum_w[r, None] * p * (logp.abs() + H[:, None])
        kids = torch.nonzero((parent_row >= i) & (parent_row < i + 250)).flatten()
        want.index_put_((parent_row[kids] - i, tok[kids].long()), edge[kids], accumulate=True)
        bound.index_put_((parent_row[kids] - i, tok[kids].long()), edge_size[kids], accumulate=True)
        e = (got.dlogits[r].double() - want).abs()
        assert (e <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * bound + 1e-38).all(), i
    assert abs(float(got.loss) - loss) <= 2.0 ** -15 * terms


@pytest.mark.parametrize("base", [3e2, 5e3, 2e4, 1e5, 1e6, 2.0 ** 24, 3e7, 1e9, 1e20, 1e31])
@pytest.mark.parametrize("entropy", [0.0, 0.05])
def test_rows_far_from_zero(cuda_device, base, entropy):
    """Logits around any number: several largest ones, among them every token that is predicted, the others up to three
    steps of bf16 below.  A shift changes nothing, and these differences are exact: the same tolerances."""
    for tree, V in ((([-1], [9]), 700), (MIXED, 700), (STAR40, 90), (([-1, 0, 0], [3, 2, 2]), 21000)):
        for sign in (1, -1):
            _, tok, _, adv, w, _ = make(tree, V, 23, zero=0.0)
            g = np.random.default_rng(abs(int(base) % 1000 + sign))
            steps = g.integers(0, 4, (len(tok), V)).astype(np.int16)
            steps[:, tok.numpy()] = 0
            top = torch.tensor(sign * base).bfloat16()
            x = (top.view(torch.int16) - sign * torch.from_numpy(steps)).view(torch.bfloat16)
            near = x.double() - top.double()
            lp = OLS.traj_logprobs(*tree, near.numpy(), tok)
            f32 = lambda a: torch.from_numpy(a.astype(np.float32))  # noqa: E731
            data = [near, tok, f32(lp - g.choice([-0.6, -0.1, 0.0, 0.1, 0.6], len(lp))), adv, w, f32(lp + 0.5 * g.normal(size=len(lp)))]
            got = run(tree, data, cuda_device, x=x.to(cuda_device), kl_coef=0.05, entropy_coef=entropy)
            check(tree, data, got, kl_coef=0.05, entropy_coef=entropy)


def rest_of(x, y):
    """(1 - p, p, H + ln p, sum of magnitudes of p_v (x_v - x_y)) of element y of a row, the first from the others alone."""
    others = torch.cat([x[:y], x[y + 1:]]) - x[y]
    e = others.exp()
    s, t = e.sum(), torch.where(e > 0, e * others, 0.0)
    return s / (1 + s), 1 / (1 + s), -t.sum() / (1 + s), t.abs().sum() / (1 + s)


@pytest.mark.parametrize("V", [2, 90, 301, 5000, 30011, 152064])
@pytest.mark.parametrize("entropy", [0.0, 0.05])
def test_confident_targets(cuda_device, V, entropy):
    """Targets of probability 1 - 10^-1 to 1 - 10^-9: their own element is g (1 - p), within the tolerances above of that, not
    of g (1 - p has the relative error of a sum and a ratio of sums, 2^-16); and the others' add up to its opposite."""
    N = 25
    g = torch.Generator().manual_seed(V)
    x = torch.randn((N, V), generator=g) * 2
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    tok[1:4] = torch.tensor([0, V - 1, V // 2])               # first, last: vectors that a row owns in part
    for r in range(N - 1):
        y = int(tok[r + 1])
        others = torch.cat([x[r, :y], x[r, y + 1:]])
        x[r, y] = torch.logsumexp(others.double(), 0).float() + 2.302585 * (0.3 + (r % 10) * 0.95)
    x = x.bfloat16()
    adv, w = torch.randn(N - 1, generator=g), torch.rand(N - 1, generator=g) + 0.5
    plan = TreePlan([-1], [N])
    room = torch.empty((N, V + 3), dtype=torch.bfloat16, device=cuda_device)
    for xd, over in ((x.to(cuda_device), False), (room[:, 1:V + 1], False), (room[:, 3:], True)):
        xd.copy_(x)
        d = TL.policy_loss(plan, xd, tok.to(cuda_device), None, adv.to(cuda_device), weights=w.to(cuda_device), per_token=True,
                           entropy_coef=entropy, dlogits=xd if over else None).dlogits.double().cpu()
        for r in range(N - 1):
            y, G = int(tok[r + 1]), -float(w[r]) * float(adv[r])
            q, p, h, size = rest_of(x[r].double(), y)
            want = G * q + entropy * float(w[r]) * p * h
            bound = abs(G) * q + entropy * float(w[r]) * p * size
            assert abs(d[r, y] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -16 * bound, (r, y, float(q), float(d[r, y] / want))
        assert not d[N - 1].any()


@pytest.mark.parametrize("V,kids", [(400, 3), (400, 20), (30011, 7), (152064, 40)])
def test_confident_targets_of_several(cuda_device, V, kids):
    """A row whose children begin with a certain token, some of them, or with others: the certain token's element is
    sum g (1 - p) of its children minus p times the others' sum, where those may be 0."""
    g = torch.Generator().manual_seed(V + kids)
    tree = ([-1] + [0] * kids, [2] + [1] * kids)
    N = 2 + kids
    x = torch.randn((N, V), generator=g)
    tok = torch.randint(0, V, (N,), generator=g, dtype=torch.int32)
    sure = V - 3
    tok[2::2] = sure                                          # every other child, the first among them
    plan = TreePlan(*tree)
    for gap in (2.0, 5.0, 9.0, 14.0, 19.0):
        x[1, sure] = -100.0
        x[1, sure] = torch.logsumexp(x[1].double(), 0).float() + gap
        xb = x.bfloat16()
        q, p, h, size = rest_of(xb[1].double(), sure)
        for others in (0.0, 1.0):
            adv = torch.randn(kids, generator=g) + 2
            adv[1::2] *= others
            r = TL.policy_loss(plan, xb.to(cuda_device), tok.to(cuda_device), None, adv.to(cuda_device), entropy_coef=0.01,
                               weights=torch.cat([torch.tensor([float(i % 3 == 0), 1.0]) for i in range(kids)]).to(cuda_device))
            d = r.dlogits.double().cpu()
            G = -adv.double()
            here = tok[2:] == sure
            want = G[here].sum() * q - p * G[~here].sum() + 0.01 * kids * p * h
            bound = G[here].abs().sum() * q + p * G[~here].abs().sum() + 0.01 * kids * p * size
            assert abs(d[1, sure] - want) <= 2.0 ** -8 * abs(want) + 2.0 ** -16 * bound, (gap, others, float(d[1, sure] / want))
            logp = torch.log_softmax(xb[1].double(), 0)
            H = -(logp.exp() * logp).sum()
            full = -G.sum() * logp.exp() + 0.01 * kids * logp.exp() * (logp + H)
            full.index_add_(0, tok[2:].long(), G)
            size_full = G.abs().sum() * logp.exp() + 0.01 * kids * logp.exp() * (logp.abs() + H)
            size_full.index_add_(0, tok[2:].long(), G.abs())
            assert ((d[1] - full).abs() <= 2.0 ** -8 * full.abs() + 2.0 ** -15 * size_full).all()


@pytest.mark.parametrize("V,kids,distinct", [(600, 6000, 600), (600, 3000, 3), (7001, 5000, 7001), (40000, 3000, 900), (152064, 1500, 5)])
def test_many_children(cuda_device, V, kids, distinct):
    """A row of thousands of children, many of which begin alike: the sum of their g in each element.  n terms in a row are
    within n 2^-24 of the sum of their magnitudes, at most 2^-12 here with the pairwise sums behind it; else as above."""
    tree = ([-1] + [0] * kids, [2] + [1] * kids)
    N = 2 + kids
    g = torch.Generator(cuda_device).manual_seed(V + kids)
    x = torch.randn((N, V), device=cuda_device, generator=g).bfloat16()
    tok = torch.randint(0, distinct, (N,), device=cuda_device, generator=g, dtype=torch.int32) * (V // distinct)
    adv = torch.randn(kids, device=cuda_device, generator=g)
    w = torch.rand(2 * kids, device=cuda_device, generator=g) * (torch.rand(2 * kids, device=cuda_device, generator=g) < 0.8)
    call = lambda: TL.policy_loss(plan, x, tok, None, adv, weights=w, entropy_coef=0.01)  # noqa: E731
    plan = TreePlan(*tree)
    got = call()
    again = call()
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for row, here, to in ((0, slice(0, None, 2), tok[1:2].expand(kids)), (1, slice(1, None, 2), tok[2:])):
        G, W = -(w.double() * adv.double().repeat_interleave(2))[here], w.double()[here]
        logp = torch.log_softmax(x[row].double(), 0)
        p, H = logp.exp(), -(logp.exp() * logp).sum()
        want = -G.sum() * p + 0.01 * W.sum() * p * (logp + H)
        size = G.abs().sum() * p + 0.01 * W.sum() * p * (logp.abs() + H)
        want.index_add_(0, to.long(), G)
        size.index_add_(0, to.long(), G.abs())
        e = (got.dlogits[row].double() - want).abs()
        assert (e <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * size).all()
    assert not got.dlogits[2:].any()


def test_time_of_many_children(cuda_device):
    """Eight times the children of a row, at most twenty times the time (what goes with their square: some thirty)."""
    def once(kids):
        plan, N = TreePlan([-1] + [0] * kids, [2] + [1] * kids), kids + 2
        g = torch.Generator(cuda_device).manual_seed(kids)
        x = torch.randn((N, 600), device=cuda_device, generator=g).bfloat16()
        tok = torch.randint(0, 600, (N,), device=cuda_device, generator=g, dtype=torch.int32)
        adv, took = torch.randn(kids, device=cuda_device, generator=g), []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            TL.policy_loss(plan, x, tok, None, adv)
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b))
        return min(took)

    assert once(16000) <= 20 * once(2000)


@pytest.mark.parametrize("kids", [31, 32, 33, 64, 127, 128, 129, 130, 257])
@pytest.mark.parametrize("V", [50, 701])
def test_children_around_the_sizes_of_a_pass(cuda_device, kids, V):
    """Whatever way the targets of a row are added up in, some with the same token: the oracle's, within the same tolerances."""
    tree = ([-1] + [0] * kids, [2] + [1] * kids)
    for same in (False, True):
        data = make(tree, V, kids + V, same=same)
        check(tree, data, run(tree, data, cuda_device, kl_coef=0.05, entropy_coef=0.01), kl_coef=0.05, entropy_coef=0.01)
