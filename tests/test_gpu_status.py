"""Notices about a call's data -- a token for a full node, a row's invalid sampling
parameters, a decay outside (0, 1] -- stay with their call: with one of them recorded and not
read, every other call gives the bits it gives without, and the status still tells."""
import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan, device_status, tree_attn_bwd, tree_attn_fwd
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import decode as TD
from prefix_tree_attention_attn_gb300.linear import tree_linear_fwd
from prefix_tree_attention_attn_gb300.sample import sample_tokens

pytestmark = pytest.mark.gpu


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=g.device).bfloat16()


def full_node(dev):
    plan = TD.DecodePlan([-1], [64], [0], 2, 2, 64)
    cache = TD.TreeCache.empty(plan.n_pages, 2, 64, dev)
    k = torch.zeros((64, 2, 64), dtype=torch.bfloat16, device=dev)
    TD.tree_cache_write(plan, cache, k, k)
    lens = plan.lens()
    TD.tree_cache_append(plan, cache, lens, k[:1], k[:1])
    assert lens.tolist() == [64]


def bad_row(dev):
    x = torch.zeros((3, 50), dtype=torch.bfloat16, device=dev)
    t = torch.tensor([1.0, -1.0, 1.0], device=dev)
    tok, _ = sample_tokens(x, torch.zeros(3, device=dev), temperature=t)
    assert tok.tolist() == [0, -1, 0]


def bad_decay(dev):
    plan = TreePlan([-1, 0], [150, 60])
    x = torch.zeros((210, 2, 128), dtype=torch.bfloat16, device=dev)
    tree_linear_fwd(plan, x, x, x, torch.tensor([0.9, 1.5], device=dev), 0.1)


NOTICES = {"full node": (full_node, TD.ERR_CACHE_FULL), "bad row": (bad_row, -15), "bad decay": (bad_decay, -12)}


@pytest.mark.parametrize("name", list(NOTICES))
def test_notices_do_not_reach_other_calls(lib, cuda_device, name):
    cause, code = NOTICES[name]
    g = torch.Generator(cuda_device).manual_seed(3)
    # both kinds of items of the attention over the cache: leaves of long segments and their prefix
    seg = [6000] + [1500 + 37 * i for i in range(40)]
    plan = TD.DecodePlan([-1] + [0] * 40, seg, range(1, 41), 16, 2, 128)
    cache, lens = TD.TreeCache.empty(plan.n_pages, 2, 128, cuda_device), plan.lens()
    TD.tree_cache_write(plan, cache, randn(g, sum(seg), 2, 128), randn(g, sum(seg), 2, 128))
    q1 = randn(g, 40, 16, 128)
    # the training side
    train = TreePlan([-1] + [0] * 8, [4000] + [700] * 8)
    n = train.n_tokens
    q, do = randn(g, n, 8, 128), randn(g, n, 8, 128)
    k, v = randn(g, n, 2, 128), randn(g, n, 2, 128)
    decay = torch.tensor([0.99, 1.0], device=cuda_device)
    logits, u = randn(g, 33, 50000), torch.rand(33, generator=g, device=cuda_device)

    def calls():
        out = list(TD.tree_decode(plan, cache, lens, q1, 0.09))
        o, lse = tree_attn_fwd(train, q, k, v, 0.09)
        _, dk, dv = tree_attn_bwd(train, q, k, v, o, lse, do, 0.09)
        return out + [o, lse, dk, dv, tree_linear_fwd(train, q, k, v, decay, 0.1), *sample_tokens(logits, u, 0.9, 0, 0.95)]

    clean = calls()
    assert device_status() == 0 and all(torch.isfinite(x.float()).all() for x in clean)
    cause(cuda_device)
    for _ in range(10):
        for a, b in zip(calls(), clean):
            assert torch.equal(a, b)
    assert device_status() == code and device_status() == 0


def test_a_failure_is_not_hidden_by_a_notice(lib, cuda_device):
    """A wait that runs out after a notice is recorded and told first."""
    bad_row(cuda_device)
    full_node(cuda_device)                          # the first notice is kept
    assert B.load().tree_attn_selftest_wait_timeout(50, None) == 0
    assert device_status() == -10 - 1000 * 99
    assert device_status() == -15
    assert device_status() == 0


def test_abandoned_items_leave_nothing_in_flight(lib, cuda_device):
    """With a failure recorded, the attention over the cache gives its waits up early and
    returns, its copies and products ended; the status read, the same calls give their bits
    again."""
    g = torch.Generator(cuda_device).manual_seed(4)
    for d, hkv in ((128, 2), (64, 1)):
        seg = [9000] + [700 + 137 * i for i in range(40)]
        plan = TD.DecodePlan([-1] + [0] * 40, seg, range(1, 41), 8 * hkv, hkv, d)
        kinds = plan.export()["items"][:, 0, 5]
        assert kinds.any() and not kinds.all()                  # CTAs' items and warps' items
        cache, lens = TD.TreeCache.empty(plan.n_pages, hkv, d, cuda_device), plan.lens()
        TD.tree_cache_write(plan, cache, randn(g, sum(seg), hkv, d), randn(g, sum(seg), hkv, d))
        q = randn(g, 40, 8 * hkv, d)
        clean = TD.tree_decode(plan, cache, lens, q, 0.09)
        assert device_status() == 0
        for _ in range(3):
            assert B.load().tree_attn_selftest_wait_timeout(10, None) == 0
            for _ in range(4):
                TD.tree_decode(plan, cache, lens, q, 0.09)      # incomplete
            assert device_status() == -10 - 1000 * 99
            for _ in range(4):
                for a, b in zip(TD.tree_decode(plan, cache, lens, q, 0.09), clean):
                    assert torch.equal(a, b)
        assert device_status() == 0
