"""Refusals of the linear attention's state calls on the host (CPU only; nothing is launched)."""
import ctypes as C

import numpy as np
import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan
from prefix_tree_attention_attn_gb300 import linear as TL


def test_slots():
    for args in (([0, 1], [0], 2), ([[0]], [[0]], 1), ([0], [1], 1), ([1], [0], 1), ([-2], [0], 1), ([0], [-2], 1),
                 ([0, 1], [1, 1], 2), ([0.5], [0], 1), ([0], [0], -1), ([2 ** 31], [0], 2 ** 31 - 1), ([0], [0], 2 ** 31)):
        with pytest.raises(ValueError):
            TL.StateSlots(*args)
    assert len(TL.StateSlots([], [], 0)) == 0
    apart = lambda a, b, n=9: TL.StateSlots(a, b, n)._rows_apart  # noqa: E731
    assert apart([0, 1], [0, 1]) and apart([3, 3, 3], [0, 1, 2]) and apart([-1, -1], [0, 1]) and apart([], [])
    assert apart([1, 1], [0, -1]) and apart([0, 1], [-1, 0])           # a padding row reads nothing
    assert not apart([0, 1], [1, 0]) and not apart([0, 0], [0, 1]) and not apart([5, 2], [2, 5])
    assert apart([2 ** 31 - 2], [0], 2 ** 31 - 1)                      # (nothing of the pool's size on the host)
    a = np.array([0, 1], np.int32)
    s = TL.StateSlots(a, a, 2)
    a[:] = 7
    assert s.slot_in.tolist() == [0, 1] and s.slot_out.tolist() == [0, 1]


def test_slots_of_a_plan(lib):
    forest = TreePlan([-1, 0, 0, -1, 3], [2, 1, 1, 2, 1])
    ok = lambda a, b: TL.StateSlots(a, b, 9)._check_plan(forest)  # noqa: E731
    ok([0, -1, -1, 1, -1], [-1, 0, 2, -1, 1])                          # each tree's own slot
    ok([0, 5, 5, 0, 5], [-1, 1, 2, 3, 5])                              # a fork; other nodes' slot_in is not read
    ok([-1] * 5, [0, 1, 2, 3, 4])
    for a, b in (([0, -1, -1, 1, -1], [-1, 1, 2, -1, 0]), ([0, -1, -1, 0, -1], [0, 1, 2, 3, 4]),
                 ([0, -1, -1, -1, -1], [-1, -1, -1, -1, 0])):
        with pytest.raises(ValueError):
            ok(a, b)
    with pytest.raises(ValueError):
        TL.StateSlots([0], [0], 1)._check_plan(forest)


def test_bad_arguments(lib):
    fake, odd, p = C.c_void_p(0x1000), C.c_void_p(0x1008), TreePlan([-1, 0], [100, 60])

    def prefill(q=fake, k=fake, v=fake, o=fake, states=fake, n=4, decay=fake, hq=4, hkv=2, d=128, scale=1.0, ws=fake,
                ws_bytes=1 << 40, plan=p.handle, a=fake, b=fake):
        return lib.tree_attn_linear_prefill(plan, q, k, v, o, states, n, a, b, decay, hq, hkv, d, scale, ws, ws_bytes, None)

    def step(states=fake, n=4, a=fake, b=fake, q=fake, k=fake, v=fake, qs=512, ks=256, vs=256, o=fake, decay=fake, rows=3,
             hq=4, hkv=2, d=128, scale=1.0):
        return lib.tree_attn_linear_step(states, n, a, b, q, k, v, qs, ks, vs, o, decay, rows, hq, hkv, d, scale, None)

    for name in ("q", "k", "v", "o", "decay", "plan", "states"):
        assert prefill(**{name: None}) == -1, name
    for name in ("q", "k", "v", "o", "states"):
        assert prefill(**{name: odd}) == -5, name
    assert prefill(a=C.c_void_p(0x1002)) == -5 and prefill(b=C.c_void_p(0x1001)) == -5 and prefill(ws=odd) == -5
    assert prefill(hq=3) == -1 and prefill(hkv=0) == -1 and prefill(n=-1) == -1 and prefill(d=64) == -4
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert prefill(scale=s) == -1
    for name in ("a", "b", "q", "k", "v", "o", "decay", "states"):
        assert step(**{name: None}) == -1, name
    for name in ("q", "k", "v", "o", "states"):
        assert step(**{name: odd}) == -5, name
    assert step(hq=5) == -1 and step(hkv=-2) == -1 and step(rows=-1) == -1 and step(n=-1) == -1 and step(d=96) == -4
    assert step(qs=508) == -1 and step(qs=504) == -1 and step(ks=248) == -1 and step(vs=250) == -1
    assert step(scale=float("nan")) == -1 and step(rows=2 ** 40) == -3
    assert step(rows=0, a=None, q=None) == 0


def test_binding_refuses_before_the_library(lib, monkeypatch):
    monkeypatch.setattr(TL, "_current_device", lambda: 0)
    x, states = torch.zeros((2, 4, 128), dtype=torch.bfloat16), torch.zeros((2, 2, 128, 128))
    with pytest.raises(ValueError, match="rows"):
        TL.tree_linear_step(states, TL.StateSlots([0], [0], 2), x, x[:, :2], x[:, :2], None, 1.0)
    with pytest.raises(ValueError, match="another row"):
        TL.tree_linear_step(states, TL.StateSlots([0, 1], [1, 0], 2), x, x[:, :2], x[:, :2], None, 1.0)
    with pytest.raises(ValueError, match="q: expected"):
        TL.tree_linear_step(states, TL.StateSlots([0, 1], [0, 1], 2), x, x[:, :2], x[:, :2], None, 1.0)
    with pytest.raises(ValueError, match="q: expected"):
        TL.tree_linear_prefill(TreePlan([-1], [2]), states, TL.StateSlots([0], [1], 2), x, x[:, :2], x[:, :2], None, 1.0)


def test_workspace_holds_what_is_written(lib):
    """The states that enter the chunks, in bf16, and the end states of the nodes with children, in fp32: nothing for leaves."""
    for parent, seg, chunks, inner in (([-1] * 1024, [300] * 1024, 3072, 0), ([-1] + [0] * 40, [128] * 41, 41, 1),
                                       ([-1, 0, 1, 2, 0, 0, 0, 0, 0, 0, 0], [129] * 11, 22, 3)):
        for hkv in (1, 8):
            assert TL.prefill_workspace(TreePlan(parent, seg), hkv, 128) == hkv * 128 * 128 * (2 * chunks + 4 * inner)


@pytest.mark.parametrize("hkv", [39, 77, 2 ** 20, 2 ** 29, 2 ** 30, 2 ** 31 - 1])
def test_any_number_of_heads_is_answered(lib, hkv):
    """A size, or a refusal of the call."""
    p, fake = TreePlan([-1, 0], [2000, 60]), C.c_void_p(0x1000)
    assert TL.prefill_workspace(p, hkv, 128) >= hkv * 128 * 128 * (2 * 17 + 4)
    assert lib.tree_attn_linear_prefill(p.handle, fake, fake, fake, fake, fake, 4, fake, fake, fake, hkv, hkv, 128, 1.0, fake,
                                        256, None) < 0
