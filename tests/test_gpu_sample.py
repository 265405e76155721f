"""Token sampling on the GPU against the exact reference.

Tokens must be equal.  The reference holds the same weights, integers of 2^45 for the
largest, from 40-digit arithmetic; a weight of the kernel may be one unit off (its
exponent carries about 2^-44), so a cut or a draw may differ only where a border lies
within a few units of the sums -- for random u, less than 1 row in 10^6 here.

Log-probs: logprob = (x - top) - log1p(rest), rest = the others' weight over the
largest's.  x - top is exact to fp32's half step; rest is a sum of V integers, each within
one unit of 2^-45, rounded to fp32; log1p has slope at most 1 and is within 2 units: an
absolute error of V * 2^-45 and a relative one below 2^-21 (both terms are at most
|logprob|).
"""
import numpy as np
import pytest
import torch

from oracle import sample as OS
from prefix_tree_attention_attn_gb300 import _binding as B
from prefix_tree_attention_attn_gb300 import build as _build
from prefix_tree_attention_attn_gb300 import device_status
from prefix_tree_attention_attn_gb300.sample import ERR_INVALID_SAMPLING, sample_tokens

pytestmark = pytest.mark.gpu


def bf16(x, dev):
    return torch.as_tensor(np.asarray(x, dtype=np.float32)).bfloat16().to(dev)


def check(logits, u, T=1.0, k=0, p=1.0, m=0.0, **kw):
    """Runs the rows, compares every one with the reference; parameters may be lists."""
    R, dev = logits.shape[0], logits.device
    arg = {}
    for name, x, dt in (("temperature", T, torch.float32), ("top_k", k, torch.int32), ("top_p", p, torch.float32),
                        ("min_p", m, torch.float32)):
        arg[name] = torch.tensor(x, dtype=dt, device=dev) if isinstance(x, (list, np.ndarray)) else x
    tok, lp = sample_tokens(logits, torch.as_tensor(np.asarray(u, np.float32)).to(dev), **arg, **kw)
    tok, lp = tok.cpu().numpy(), lp.cpu().numpy().astype(np.float64)
    x = logits.float().cpu().numpy().astype(np.float64)
    at = lambda a, r: a[r] if isinstance(a, (list, np.ndarray)) else a  # noqa: E731
    for r in range(R):
        t, want = OS.draw(x[r], u[r], at(T, r), at(k, r), at(p, r), at(m, r))
        assert tok[r] == t, (r, tok[r], t, u[r], at(T, r), at(k, r), at(p, r), at(m, r))
        if t < 0:
            assert np.isnan(lp[r])
        else:
            assert abs(lp[r] - want) <= 2.0 ** -21 * abs(want) + x.shape[1] * 2.0 ** -45, (r, lp[r], want)
    return tok, lp


@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 8192, 32003, 152064, 262144])
def test_random_rows_every_filter(lib, cuda_device, V):
    """Vocabularies from one token to the largest, every row another mix of filters."""
    rng = np.random.default_rng(V)
    R = 24 if V < 40000 else 6
    x = rng.standard_normal((R, V)) * rng.choice([0.01, 2.0, 6.0, 30.0], size=(R, 1))
    T = rng.choice([0.0, 0.3, 0.7, 1.0, 1.0, 3.0, 40.0], size=R)
    k = rng.choice([0, 0, 1, 2, 5, 50, 1000, V, V + 5], size=R)
    p = rng.choice([1.0, 1.0, 0.95, 0.5, 0.01, 0.0], size=R)
    m = rng.choice([0.0, 0.0, 0.01, 0.2, 1.0, 2.0], size=R)
    u = rng.random(R).astype(np.float32)
    u[0], u[-1] = 0.0, np.nextafter(np.float32(1), np.float32(0))
    check(bf16(x, cuda_device), u, list(T), list(map(int, k)), list(p), list(m))
    assert device_status() == 0


@pytest.mark.parametrize("rows", [1, 77, 160, 310])
def test_row_counts(lib, cuda_device, rows):
    """Every split of a row over CTAs (8, 4, 2, 1), scalar parameters, odd row starts."""
    rng = np.random.default_rng(rows)
    V = 33001
    wide = bf16(rng.standard_normal((rows, V + 4)) * 3, cuda_device)
    u = rng.random(rows).astype(np.float32)
    sub = list(rng.permutation(rows)[:12])
    full = wide[:, 3:3 + V]                                # rows start on odd elements
    tok, lp = sample_tokens(full, torch.from_numpy(u).to(cuda_device), 0.9, 40, 0.9, 0.01)
    pick = full[sub].contiguous()
    t2, l2 = check(pick, u[sub], 0.9, 40, 0.9, 0.01)
    assert np.array_equal(tok.cpu().numpy()[sub], t2) and np.array_equal(lp.cpu().numpy()[sub].astype(np.float64), l2)
    tok3, lp3 = sample_tokens(full, torch.from_numpy(u).to(cuda_device), 0.9, 40, 0.9, 0.01)
    assert torch.equal(tok, tok3) and torch.equal(lp, lp3)


def test_ties_and_borders(lib, cuda_device):
    """Equal logits: ties go to the lowest index; cuts and draws that fall exactly on a
    border.  Eight equal tokens have cumulated shares of exactly 1/8."""
    x = np.zeros((1, 8))
    for i in range(8):
        for frac, want in ((0.0, i), (0.5, i), (np.float32(1) - 2.0 ** -20, i)):
            tok, _ = check(bf16(x, cuda_device), [np.float32((i + float(frac)) / 8)])
            assert tok[0] == want
    assert check(bf16(x, cuda_device), [0.999], p=0.5)[0][0] == 3           # four reach exactly half
    assert check(bf16(x, cuda_device), [0.999], p=float(np.float32(0.5) + 2.0 ** -24))[0][0] == 4
    assert check(bf16(x, cuda_device), [0.999], k=3)[0][0] == 2
    assert check(bf16(x, cuda_device), [0.999], m=1.0)[0][0] == 7
    assert check(bf16(x, cuda_device), [0.3], T=0.0)[0][0] == 0
    y = np.array([[1.0, -0.0, 3.0, 0.0, 3.0, -0.0, 1.0]])                    # -0 and 0 are equal
    for u in np.linspace(0, 0.999, 40):
        check(bf16(y, cuda_device), [u], T=7.0)
        check(bf16(y, cuda_device), [u], T=7.0, k=6)
    for u in (-1.0, 0.0, 1.0, 5.0):                                          # out of [0, 1)
        check(bf16(y, cuda_device), [u], k=4)


def test_masks_and_lost_rows(lib, cuda_device):
    """-inf and the type's lowest value as masks; rows without a distribution."""
    rng = np.random.default_rng(2)
    low = float(torch.finfo(torch.bfloat16).min)
    V, inf = 9000, float("inf")
    x = rng.standard_normal((12, V)) * 3
    x[0, 10:] = -inf
    x[1, :-1] = -inf                                   # one token left
    x[2, 5:] = low
    x[3, :] = low                                      # all masked alike: uniform
    x[4, :] = -inf                                     # nothing left
    x[5, 77] = float("nan")
    x[6, 78] = inf
    x[7, 20:] = -1e4
    x[8, ::2] = low
    x[9, ::2] = -inf
    x[9, 1::2] = low                                   # -inf beside the lowest value
    x[10] = -60000 - 1000 * np.abs(x[10])              # a row far below the short range
    x[11, 100:] = -70000
    u = rng.random(12).astype(np.float32)
    for T, k, p in ((1.0, 0, 1.0), (0.5, 30, 0.9), (2000.0, 0, 0.99), (0.0, 0, 1.0)):
        tok, lp = check(bf16(x, cuda_device), u, T, k, p)
        assert (tok[4:7] == -1).all()
    assert device_status() == 0


def test_values_outside_the_short_range(lib, cuda_device):
    """Tiny, huge and mixed logits take the full range and stay exact."""
    rng = np.random.default_rng(3)
    V = 5000
    x = np.stack([rng.standard_normal(V) * 1e-20, rng.standard_normal(V) * 1e-39, rng.standard_normal(V) * 1e6,
                  rng.standard_normal(V) * 2.0 ** rng.integers(-130, 127, V), rng.standard_normal(V) * 1e30,
                  np.where(rng.random(V) < 0.01, 1e-15, rng.standard_normal(V)), np.full(V, -1e20),
                  np.full(V, 3e38)])
    u = rng.random(len(x)).astype(np.float32)
    for T, k, p, m in (([1e-20, 1e-39, 1e6, 1e10, 1e30, 1.0, 1.0, 1e38], 0, 1.0, 0.0), (1.0, 700, 0.9, 0.0),
                       ([3e-20, 5e-39, 3e5, 1e30, 1e29, 0.2, 1e-3, 1.0], 64, 0.7, 0.05), (0.0, 0, 1.0, 0.0),
                       (1e38, 0, 0.5, 0.999)):
        check(bf16(x, cuda_device), u, T, k, p, m)


def test_peaked_rows_keep_their_logprob(lib, cuda_device):
    """A token of almost all the mass: its log-prob is small and still exact."""
    x = np.full((3, 4000), -20.0)
    x[0, 17], x[1, 5], x[2, 3] = 0.0, -4.0, 10.0
    for T in (0.0, 1.0, 0.5):
        check(bf16(x, cuda_device), [0.2, 0.3, 0.4], T)


def test_invalid_parameters_mark_their_row(lib, cuda_device):
    x = bf16(np.random.default_rng(4).standard_normal((6, 100)), cuda_device)
    nan = float("nan")
    tok, lp = sample_tokens(x, torch.full((6,), 0.5, device=cuda_device),
                            torch.tensor([1.0, -1.0, nan, float("inf"), 1.0, 1.0], device=cuda_device), 0,
                            torch.tensor([0.9, 1, 1, 1, nan, 1], device=cuda_device),
                            torch.tensor([0, 0, 0, 0, 0, nan], device=cuda_device))
    assert tok[0] >= 0 and (tok[1:] == -1).all() and torch.isnan(lp[1:]).all() and torch.isfinite(lp[0])
    assert device_status() == ERR_INVALID_SAMPLING and device_status() == 0
    tok, _ = sample_tokens(x[:1], torch.full((1,), nan, device=cuda_device))
    assert tok[0] == -1 and device_status() == ERR_INVALID_SAMPLING


def test_frequencies(lib, cuda_device):
    """A regular grid of u draws each token in proportion: with n grid points, every
    token's count is within one of n times its share of the kept tokens."""
    rng = np.random.default_rng(6)
    x = bf16(rng.standard_normal((1, 300)) * 2, cuda_device)
    n = 1 << 14
    u = (torch.arange(n, device=cuda_device) + 0.5) / n
    tok, _ = sample_tokens(x.expand(n, 300).contiguous(), u, 0.8, 60, 1.0, 0.0)
    w = np.exp((x[0].float().cpu().numpy().astype(np.float64)) / np.float32(0.8))
    keep = np.argsort(-w, kind="stable")[:60]
    share = np.zeros(300)
    share[keep] = w[keep] / w[keep].sum()
    got = np.bincount(tok.cpu().numpy(), minlength=300)
    assert (np.abs(got - n * share) <= 1.001).all()


def test_graph_streams_and_outputs(lib, cuda_device):
    rng = np.random.default_rng(7)
    x = bf16(rng.standard_normal((5, 40000)) * 2, cuda_device)
    u = torch.zeros(5, device=cuda_device)
    tok, lp = torch.empty(5, dtype=torch.int32, device=cuda_device), torch.empty(5, device=cuda_device)
    sample_tokens(x, u, tokens=tok, logprobs=lp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sample_tokens(x, u, 0.9, 0, 0.95, 0.0, tokens=tok, logprobs=lp)
    side = torch.cuda.Stream()
    for _ in range(4):
        new = torch.rand(5, device=cuda_device)
        u.copy_(new)
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        t2, l2 = sample_tokens(x, new, 0.9, 0, 0.95, 0.0, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(tok, t2) and torch.equal(lp, l2)
    e = sample_tokens(x[:0], u[:0])
    assert e[0].shape == (0,)


def test_refusals(lib, cuda_device):
    x, u = torch.zeros((2, 64), dtype=torch.bfloat16, device=cuda_device), torch.zeros(2, device=cuda_device)
    for bad in (lambda: sample_tokens(x.float(), u), lambda: sample_tokens(x.cpu(), u), lambda: sample_tokens(x[0], u),
                lambda: sample_tokens(x, u[:1]), lambda: sample_tokens(x, u.double()), lambda: sample_tokens(x[:, ::2], u),
                lambda: sample_tokens(x[:1].expand(2, 64), u), lambda: sample_tokens(x, u, top_k=u),
                lambda: sample_tokens(x, u, temperature=u[:1]), lambda: sample_tokens(x, u, tokens=u),
                lambda: sample_tokens(torch.zeros((1, 262145), dtype=torch.bfloat16, device=cuda_device), u[:1]),
                lambda: sample_tokens(torch.zeros((1, 0), dtype=torch.bfloat16, device=cuda_device), u[:1])):
        with pytest.raises((ValueError, RuntimeError)):
            bad()


@pytest.mark.parametrize("k", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1])
def test_top_k_that_is_no_int32_is_refused(lib, cuda_device, k):
    x, u = torch.zeros((2, 64), dtype=torch.bfloat16, device=cuda_device), torch.zeros(2, device=cuda_device)
    with pytest.raises(ValueError):
        sample_tokens(x, u, top_k=k)


def test_rows_behind_32_bit_offsets(lib, cuda_device):
    """The last of 8,200 rows of 262,144 logits (2^31 elements and more before them) draw what
    they draw alone."""
    R, V = 8200, 262144
    g = torch.Generator(cuda_device).manual_seed(7)
    x = torch.zeros((R, V), dtype=torch.bfloat16, device=cuda_device)
    x[-4:] = torch.randn((4, V), device=cuda_device, generator=g).bfloat16()
    u = torch.rand(R, device=cuda_device, generator=g)
    tok, lp = sample_tokens(x, u, temperature=0.9, top_p=0.8)
    t2, l2 = sample_tokens(x[-4:].clone(), u[-4:].clone(), temperature=0.9, top_p=0.8)
    assert torch.equal(tok[-4:], t2) and torch.equal(lp[-4:], l2)
    assert (tok[:-4] >= 0).all() and (tok[:-4] < 0.81 * V).all()       # equal logits: the first 80 %


@pytest.mark.parametrize("offset", [0, 1, 3, 6])
@pytest.mark.parametrize("ctas,rows", [(8, 7), (4, 23), (2, 55), (1, 120)])
def test_rows_split_over_ctas(lib, cuda_device, ctas, rows, offset):
    """A row's slices start anywhere: 8, 4, 2 and 1 CTAs a row at 33,001 logits (by the model in
    the call), rows 33,008 elements apart that begin on odd elements, twice each in a row and
    with a tie that reaches over every slice."""
    rng = np.random.default_rng([ctas, offset])
    V, stride = 33001, 33008
    x = rng.standard_normal((rows, V)) * 3
    x[1::2] = np.round(x[1::2])                            # thousands of equal logits
    flat = torch.zeros(offset + rows * stride, dtype=torch.bfloat16, device=cuda_device)
    full = flat[offset:].view(rows, stride)[:, :V]
    full.copy_(bf16(x, cuda_device))
    u = rng.random(rows).astype(np.float32)
    ud = torch.from_numpy(u).to(cuda_device)
    outs = [sample_tokens(full, ud, 0.9, 500, 0.95, 0.001) for _ in range(50)]
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs)
    sub = [int(r) for r in rng.permutation(rows)[:7]]
    want = [OS.draw(full[r].float().cpu().numpy().astype(np.float64), u[r], 0.9, 500, 0.95, 0.001) for r in sub]
    assert [int(outs[0][0][r]) for r in sub] == [t for t, _ in want]
    for r, (_, lp) in zip(sub, want):
        assert abs(float(outs[0][1][r]) - lp) <= 2.0 ** -21 * abs(lp) + V * 2.0 ** -45
    assert device_status() == 0


@pytest.mark.parametrize("rows,V", [(1, 152064), (30, 33001), (60, 9000), (200, 4097)])
def test_debug_build_is_clean_and_gives_the_same_bits(lib, cuda_device, rows, V):
    """Every split, the short and the full range, few and many equal logits through the
    bounds-checked build."""
    rng = np.random.default_rng([rows, V])
    x = rng.standard_normal((rows, V)) * 4
    x[1::4] = np.round(x[1::4])                            # many ties, zeros of both signs
    x[2::8, ::3] = -np.inf
    x[3::8] *= 1e6                                         # the full range
    x[5::8, 0] = 1e-20
    x[6::16] = 0
    x[7::16] = np.nan
    logits, u = bf16(x, cuda_device), torch.from_numpy(rng.random(rows).astype(np.float32)).to(cuda_device)
    T = torch.from_numpy(rng.choice([0.0, 0.7, 1.0, 2.0], rows).astype(np.float32)).to(cuda_device)
    out = []
    for path in (_build.LIB, _build.build_library(debug=True)):
        with B.library(path):
            out.append(sample_tokens(logits, u, T, 300, 0.9, 0.001) + sample_tokens(logits, u, T))
            assert device_status() == 0, path
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(*out))
