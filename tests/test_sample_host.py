"""Host-side checks of the sampling call and its reference (CPU only)."""
import ctypes as C

import numpy as np

from oracle import sample as OS
from prefix_tree_attention_attn_gb300 import _binding as B


def test_the_call_validates_before_touching_the_device(lib):
    f, odd2, odd4 = C.c_void_p(0x1000), C.c_void_p(0x1001), C.c_void_p(0x1002)
    s = B.Sampling()
    s.temperature = 1.0
    call = lib.tree_attn_sample
    ok = (f, 100, 2, 100, f, C.byref(s), f, f, None)

    def with_(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return call(*a)
    assert with_(_0=None) == -1 and with_(_4=None) == -1 and with_(_5=None) == -1 and with_(_6=None) == -1
    assert with_(_2=-1) == -1 and with_(_3=0) == -1 and with_(_1=99) == -1
    assert with_(_1=262145, _3=262145) == -3
    assert with_(_0=odd2) == -5 and with_(_4=odd4) == -5 and with_(_6=odd4) == -5 and with_(_7=odd4) == -5
    bad = B.Sampling()
    bad.top_ks = 0x1002
    assert with_(_5=C.byref(bad)) == -5
    assert with_(_2=0) == 0                                   # no rows: nothing to do
    assert lib.tree_attn_strerror(-15).decode() == "invalid sampling parameters of a row"


def test_reference_draw_against_plain_formulas():
    """The exact reference against cumulated fp64 softmax shares, away from borders."""
    rng = np.random.default_rng(0)
    for _ in range(50):
        x = np.round(rng.standard_normal(40) * 8) / 4
        T, u = float(rng.choice([0.5, 1.0, 2.0])), float(np.float32(rng.random()))
        order = np.lexsort((np.arange(40), -x))
        w = np.exp((x[order] - x.max()) / T)
        c = np.cumsum(w)
        n = int((c < 0.8 * c[-1]).sum()) + 1
        share = c[:n] / c[n - 1]
        if np.abs(share - u).min() < 1e-9 or np.abs(c / c[-1] - 0.8).min() < 1e-6:
            continue
        t, lp = OS.draw(x, u, T, 0, 0.8, 0.0)
        assert t == order[int((share <= u).sum())]
        assert abs(lp - (x[t] - np.log(np.exp(x).sum()))) < 1e-12
    assert OS.weights([0.0], 0.0, 1.0) == [OS.ONE] and OS.weights([-100.0], 0.0, 1.0) == [0]
    assert OS.draw([1.0, 3.0, 3.0], 0.9, 0.0)[0] == 1
