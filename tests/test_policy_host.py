"""Refusals of the policy loss on the host (CPU only; nothing is launched)."""
import ctypes as C

import pytest
import torch

from prefix_tree_attention_attn_gb300 import TreePlan
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import loss as TL

FAKE, ODD2, ODD1 = 0x1000, 0x1002, 0x1001


def status(lib, plan, logits=FAKE, stride=100, vocab=100, tokens=FAKE, policy=(), loss=FAKE, logprobs=FAKE, entropy=FAKE,
           dlogits=FAKE * 4, d_stride=100, ws=FAKE, ws_bytes=1 << 20, **fields):
    s = B.Policy(FAKE, FAKE, FAKE, FAKE, 0, 0.2, 0.2, 0.1, 0.0, 1.0)
    for k, v in fields.items():
        setattr(s, k, v)
    p = lambda x: C.c_void_p(x)  # noqa: E731
    return lib.tree_attn_policy_loss(plan.handle if plan else None, p(logits), stride, vocab, p(tokens),
                                     C.byref(s) if policy is not None else None, p(loss), p(logprobs), p(entropy),
                                     p(dlogits), d_stride, p(ws), ws_bytes, None)


def test_bad_arguments(lib):
    plan = TreePlan([-1, 0, 0], [5, 3, 2])
    bad = -1
    assert status(lib, None) == bad
    for name in ("logits", "tokens", "loss"):
        assert status(lib, plan, **{name: None}) == bad
    assert status(lib, plan, policy=None) == bad
    assert status(lib, plan, vocab=0) == bad and status(lib, plan, vocab=-5) == bad
    assert status(lib, plan, stride=99) == bad and status(lib, plan, d_stride=99) == bad
    assert status(lib, plan, dlogits=FAKE, stride=104) == bad               # over the logits with another stride
    assert status(lib, plan, vocab=262145, stride=1 << 20, d_stride=1 << 20) == -3
    nan, inf = float("nan"), float("inf")
    for fields in (dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_low=nan), dict(clip_high=-0.1), dict(clip_high=nan),
                   dict(kl_coef=inf), dict(kl_coef=nan), dict(entropy_coef=inf), dict(grad_scale=nan), dict(per_token=2)):
        assert status(lib, plan, **fields) == bad, fields
    assert status(lib, plan, logits=ODD1) == -5 and status(lib, plan, dlogits=ODD1) == -5
    for name in ("tokens", "loss", "logprobs", "entropy"):
        assert status(lib, plan, **{name: ODD2}) == -5
    for name in ("old_logprobs", "advantages", "weights", "ref_logprobs"):
        assert status(lib, plan, **{name: ODD2}) == -5
    assert status(lib, plan, ws=0x1010) == -5
    need = TL.policy_workspace(plan)
    assert status(lib, plan, ws_bytes=need - 1) == -6 and status(lib, plan, ws=None) == -6
    n = C.c_size_t()
    assert lib.tree_attn_policy_loss_workspace(None, C.byref(n)) == bad
    assert lib.tree_attn_policy_loss_workspace(plan.handle, None) == bad


def test_binding_refuses_before_the_library(lib, monkeypatch):
    """Tensors on the CPU, of the wrong shape or type: refused before anything is launched."""
    monkeypatch.setattr(TL, "_current_device", lambda: 0)
    plan = TreePlan([-1, 0, 0], [5, 3, 2])
    x, tok, adv = torch.zeros((10, 50), dtype=torch.bfloat16), torch.zeros(10, dtype=torch.int32), torch.zeros(2)
    for args in ((x, tok), (x.float(), tok), (x[:9], tok), (x[0], tok)):
        with pytest.raises(ValueError, match="logits"):
            TL.policy_loss(plan, *args, None, adv)
