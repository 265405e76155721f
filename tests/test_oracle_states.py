"""Pins of the linear attention oracle that starts from given states (CPU): zero states give the other
formulas, a tree cut at a node and continued from its state gives the whole tree's outputs, and a
hand-worked token."""
import numpy as np

from oracle import layout as OL
from oracle import linear as OLN


def draw(seed, N, hq, hkv, d):
    g = np.random.default_rng(seed)
    return g.normal(size=(N, hq, d)), g.normal(size=(N, hkv, d)), g.normal(size=(N, hkv, d))


def test_zero_states_are_the_other_formulas():
    parent, seg = [-1, 0, 0, 1, -1], [3, 2, 4, 1, 2]
    q, k, v = draw(1, sum(seg), 4, 2, 5)
    o, end, size, mass = OLN.from_states(parent, seg, q, k, v, [0.9, 1.0], 0.3, [None] * 5, chunk=2)
    want = OLN.forward_parallel(parent, seg, q, k, v, [0.9, 1.0], 0.3)
    assert np.abs(o - want).max() <= 1e-12
    assert (np.abs(o) <= size + 1e-12).all() and all((np.abs(end[u]) <= mass[u] + 1e-12).all() for u in end)


def test_continuing_a_cut_tree():
    parent, seg = [-1, 0, 1, 1], [4, 3, 2, 5]
    q, k, v = draw(2, sum(seg), 2, 1, 4)
    _, off, _ = OL.packed_layout(parent, seg)
    o, end, _, _ = OLN.from_states(parent, seg, q, k, v, [0.8], 1.0, [None] * 4)
    rows = np.r_[off[2]:off[2] + 2, off[3]:off[3] + 5]
    o2, end2, _, _ = OLN.from_states([-1, -1], [2, 5], q[rows], k[rows], v[rows], [0.8], 1.0, [end[1], end[1]])
    assert np.abs(o2 - o[rows]).max() <= 1e-12
    assert np.abs(end2[0] - end[2]).max() <= 1e-12 and np.abs(end2[1] - end[3]).max() <= 1e-12


def test_hand_worked():
    S0 = np.array([[[1.0, 2.0], [3.0, 4.0]]])
    q, k, v = np.array([[[1.0, 0.0], [0.0, 2.0]]]), np.array([[[1.0, -1.0]]]), np.array([[[2.0, 3.0]]])
    o, end, _, _ = OLN.from_states([-1], [1], q, k, v, [0.5], 10.0, [S0])
    assert np.allclose(end[0], [[[2.5, 4.0], [-0.5, -1.0]]]) and np.allclose(o[0], [[25.0, 40.0], [-10.0, -20.0]])
