"""The forward and backward calls captured in a CUDA graph.

Once a plan's tables are on the device (its first call there, or
tree_attn_plan_upload), tree_attn_fwd and tree_attn_bwd allocate nothing and
do not synchronise, so a whole step can be captured once and replayed -- what
launch-bound small trees want (five launches per step become one).  Replays
must give the eager results: O, LSE, dK and dV bit for bit (dQ sums fp32
partials with atomics, so within 1e-3)."""
import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan, device_status, tree_attn_bwd, tree_attn_fwd
from workloads import tensors as WX
from workloads import trees as WT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["tiny_binary", "grpo_star"])
def test_graph_replay_matches_eager(lib, cuda_device, name):
    t = WT.load_tree(name)
    heads, rec, xc = WX.workload_inputs(name, t.n_tokens)
    x = {k: v.to(cuda_device) for k, v in xc.items()}
    plan = TreePlan(t.parent, t.seg_len)
    plan.upload()
    o, lse = torch.empty_like(x["q"]), torch.empty((heads.hq, t.n_tokens), dtype=torch.float32, device=cuda_device)
    dq, dk, dv = torch.empty_like(x["q"]), torch.empty_like(x["k"]), torch.empty_like(x["v"])
    ws = torch.empty(plan.workspace_size(heads.hq, heads.hkv, heads.d)[1], dtype=torch.uint8, device=cuda_device)

    def step():
        tree_attn_fwd(plan, x["q"], x["k"], x["v"], rec.scale, o=o, lse=lse)
        tree_attn_bwd(plan, x["q"], x["k"], x["v"], o, lse, x["do"], rec.scale, dq=dq, dk=dk, dv=dv, workspace=ws)

    step()
    torch.cuda.synchronize()
    eager = [a.clone() for a in (o, lse, dq, dk, dv)]
    for a in (o, lse, dq, dk, dv):
        a.fill_(float("nan"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert device_status() == 0
    for nm, a, b in zip(("O", "LSE", "dQ", "dK", "dV"), (o, lse, dq, dk, dv), eager):
        assert torch.isfinite(a.float()).all(), nm
        if nm == "dQ":
            assert float((a.float() - b.float()).norm() / b.float().norm()) <= 1e-3
        else:
            assert torch.equal(a, b), nm


def test_plans_dropped_while_a_graph_is_captured(lib, cuda_device):
    """Plans may be dropped at any time, during a capture too: the captured calls of other plans
    stand and replay."""
    from prefix_tree_attention_attn_gb300 import decode as TD
    make = lambda: TD.DecodePlan([-1, 0], [700, 5], [1], 4, 2, 64)  # noqa: E731
    kept, dropped, train = make(), make(), TreePlan([-1, 0], [200, 30])
    for p in (kept, dropped, train):
        p.upload()
    g = torch.Generator(cuda_device).manual_seed(2)
    draw = lambda *s: torch.randn(s, device=cuda_device, generator=g).bfloat16()  # noqa: E731
    cache, lens = TD.TreeCache.empty(kept.n_pages, 2, 64, cuda_device), kept.lens()
    TD.tree_cache_write(kept, cache, draw(705, 2, 64), draw(705, 2, 64))
    q = draw(1, 4, 64)
    want = TD.tree_decode(kept, cache, lens, q, 0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        TD.tree_decode(kept, cache, lens, q, 0.1)
        dropped.close()
        train.close()
        got = TD.tree_decode(kept, cache, lens, q, 0.1)
    for _ in range(3):
        got[0].zero_(), got[1].zero_()
        graph.replay()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert device_status() == 0


def test_a_refused_launch_is_its_own_calls_error(lib, cuda_device):
    """A plan's first call does not belong into a capture: it and the calls after it in the lost
    capture are refused; the calls after that are not taken for failed."""
    from prefix_tree_attention_attn_gb300 import _binding as B
    from prefix_tree_attention_attn_gb300 import decode as TD
    from prefix_tree_attention_attn_gb300.sample import sample_tokens
    make = lambda: TD.DecodePlan([-1, 0], [70, 5], [1], 4, 2, 64, capacity=[70, 60])  # noqa: E731
    kept, late = make(), make()
    kept.upload()
    k = torch.ones((75, 2, 64), dtype=torch.bfloat16, device=cuda_device)
    q, x, u = torch.ones((1, 4, 64), dtype=torch.bfloat16, device=cuda_device), k.view(75, 128), torch.zeros(75, device=cuda_device)
    for refused in ("append", "decode", "sample"):
        cache, lens = TD.TreeCache.empty(kept.n_pages, 2, 64, cuda_device), kept.lens()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError):
            with torch.cuda.graph(graph):
                with pytest.raises(B.TreeAttnError):
                    TD.tree_decode(late, cache, lens, q, 0.1)
                with pytest.raises(B.TreeAttnError):
                    if refused == "append":
                        TD.tree_cache_append(kept, cache, lens, k[:1], k[:1])
                    elif refused == "decode":
                        TD.tree_decode(kept, cache, lens, q, 0.1)
                    else:
                        sample_tokens(x, u)
        TD.tree_cache_write(kept, cache, k, k)              # reports launches by the runtime's last error
        o, _ = TD.tree_decode(kept, cache, lens, q, 0.1)
        assert (o == 1).all() and device_status() == 0
