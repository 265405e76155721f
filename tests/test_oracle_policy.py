"""Pins of the policy loss's oracle (CPU): its gradient against central differences of its loss
and against autograd of the plain formula on the expanded trajectories, and hand-worked values."""
import numpy as np
import pytest
import torch

from oracle import layout as OL
from oracle import loss as OLS

TREES = [([-1], [5]), ([-1, 0, 0], [3, 2, 1]), ([-1, 0, 0, 1, -1], [2, 3, 1, 2, 4]), ([-1, 0, 1], [1, 1, 1])]


def make(parent, seg, V, seed, per_token):
    g = np.random.default_rng(seed)
    N, L = sum(seg), len(OL.leaves(parent))
    n = sum(len(i) for _, i in OL.trajectories(parent, seg)) - L
    x, tok = g.normal(size=(N, V)) * 2, g.integers(0, V, N)
    lp = OLS.traj_logprobs(parent, seg, x, tok)
    # ratios away from the clip's borders
    old = lp - g.choice([-0.6, -0.1, 0.05, 0.5], n)
    return x, tok, old, g.normal(size=n if per_token else L), g.random(n) * (g.random(n) < 0.7), lp + g.normal(size=n) * 0.3


@pytest.mark.parametrize("per_token", [False, True])
@pytest.mark.parametrize("k", range(len(TREES)))
def test_gradient_against_differences_and_autograd(k, per_token):
    parent, seg = TREES[k]
    x, tok, old, adv, w, ref = make(parent, seg, 6, k, per_token)
    kw = dict(weights=w, ref=ref, per_token=per_token, clip_low=0.2, clip_high=0.3, kl_coef=0.1, entropy_coef=0.05)
    loss, lp, ent, grad, bound = OLS.policy_loss(parent, seg, x, tok, old, adv, **kw)
    h = 1e-5
    for at in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        d = (OLS.policy_loss(parent, seg, up, tok, old, adv, **kw)[0] -
             OLS.policy_loss(parent, seg, down, tok, old, adv, **kw)[0]) / (2 * h)
        assert abs(d - grad[at]) <= 1e-8
    assert (np.abs(grad) <= bound + 1e-15).all()
    t = torch.tensor(x, requires_grad=True)
    logp = torch.log_softmax(t, 1)
    total, i = 0.0, 0
    for l, (_, idx) in enumerate(OL.trajectories(parent, seg)):
        for q in range(len(idx) - 1):
            a, lpk = adv[i if per_token else l], logp[idx[q], int(tok[idx[q + 1]])]
            ratio = torch.exp(lpk - old[i])
            far = ref[i] - lpk
            e = -(logp[idx[q]].exp() * logp[idx[q]]).sum()
            total = total + w[i] * (-torch.minimum(ratio * a, ratio.clamp(0.8, 1.3) * a) +
                                    0.1 * (torch.exp(far) - far - 1) - 0.05 * e)
            i += 1
    if i:
        total.backward()
        assert abs(float(total.detach()) - loss) <= 1e-12 and np.abs(t.grad.numpy() - grad).max() <= 1e-12


def test_hand_worked():
    # two tokens, two logits equal: lp = -ln 2, entropy ln 2; ratio 2 of an advantage of 1 is clipped at 1.2
    x = np.zeros((2, 2))
    loss, lp, ent, grad, _ = OLS.policy_loss([-1], [2], x, [0, 1], [-2 * np.log(2)], [1.0])
    assert abs(loss + 1.2) < 1e-15 and abs(lp[0] + np.log(2)) < 1e-15 and not grad.any()
    assert abs(ent[0] - np.log(2)) < 1e-15 and ent[1] == 0
    # an advantage of -1 is not held from above: loss 2, slope 2 (1[v = 1] - 1/2)
    loss, _, _, grad, _ = OLS.policy_loss([-1], [2], x, [0, 1], [-2 * np.log(2)], [-1.0])
    assert abs(loss - 2) < 1e-15 and np.allclose(grad[0], [-1, 1]) and not grad[1].any()
    # a ratio of 1 with a clip of nothing: the border belongs to the free side
    loss, _, _, grad, _ = OLS.policy_loss([-1], [2], x, [0, 1], None, [3.0], clip_low=0.0, clip_high=0.0)
    assert loss == -3 and np.allclose(grad[0], [1.5, -1.5])
