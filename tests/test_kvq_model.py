"""CPU pins of the 64-bit models that the GPU tests of the 4-bit cache and of the acceptance compare with."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import kvq_model as m


def exact_row(x):
    """Codes, scale and zero of one row in rational arithmetic (differences and quotients are exact here)."""
    v = [Fraction(float(t)) for t in x]
    z = min(v)
    want = (max(v) - z) / 15
    cands = [Fraction(float(c)) for c in m.from_bits(np.arange(0x7F80, dtype=np.uint16))]
    lo, hi = 0, len(cands) - 1
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if cands[mid] <= want else (lo, mid - 1)
    s = lo
    if lo + 1 < len(cands):
        a, b = want - cands[lo], cands[lo + 1] - want
        s = lo + 1 if a > b or (a == b and lo & 1) else lo
    if cands[s] == 0:
        return [0] * len(v), s
    out = []
    for t in v:
        y = (t - z) / cands[s]
        c = int(y)
        f = y - c
        c += f > Fraction(1, 2) or (f == Fraction(1, 2) and c % 2 == 1)
        out.append(min(15, max(0, c)))
    return out, s


@pytest.mark.parametrize("seed", range(4))
def test_quantise_is_the_rational_definition(seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((8, 64), generator=g) * torch.exp(torch.randn((8, 1), generator=g) * 4)
    x[0] = 0.0
    x[1] = 3.25                       # constant
    x[2] = torch.arange(64) / 2       # ties
    x[3, 1:] = x[3, :1] * 1e-3
    x = x.bfloat16()
    c, s, z = m.quantise(x)
    for i in range(8):
        ref, rs = exact_row(x[i].float().numpy())
        assert list(c[i]) == ref and int(s[i]) == rs, i
        assert m.from_bits(z[i:i + 1])[0] == x[i].float().min().item()


def test_rounding_to_bf16_is_torch_rounding_where_fp32_is_exact():
    g = np.random.default_rng(0)
    f = np.abs(g.standard_normal(4096)).astype(np.float32)
    want = m.bits(torch.from_numpy(f).bfloat16())
    assert np.array_equal(m.to_bf16_bits(f.astype(np.float64)), want)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_every_code_has_a_place_of_its_own(d):
    seen = np.zeros((m.rec_bytes(d), 2), int)
    for is_v in (False, True):
        for r in range(64):
            at, sh = m._addr(d, is_v, r)
            seen[at, sh // 4] += 1
    assert (seen[: 64 * d] == 1).all() and (seen[64 * d:] == 0).all()


def test_store_and_held_agree_and_leave_other_positions():
    g = torch.Generator().manual_seed(1)
    data = torch.randint(0, 256, (2, 1, 2, m.rec_bytes(64)), generator=g, dtype=torch.uint8).numpy()
    before = m.held(data, None, 1, 0, 100, True)
    k = torch.randn((2, 5, 1, 64), generator=g).bfloat16()
    v = torch.randn((2, 5, 1, 64), generator=g).bfloat16()
    m.store(data, None, [3, 67], k, v)
    c, s, z = m.quantise(v)
    got = m.held(data, None, 1, 0, 100, True)
    assert (got[0][62:67] == c[1, :, 0]).all() and (got[1][62:67] == m.from_bits(s[1, :, 0])).all()
    keep = np.r_[0:62, 67:100]
    assert (got[0][keep] == before[0][keep]).all()
    assert (m.held(data, None, 0, 0, 3, False)[0] == m.quantise(k)[0][0, 2:, 0]).all()  # two tokens of padding


def test_attention_of_one_key_and_of_equal_keys():
    data = np.zeros((1, 1, 1, m.rec_bytes(64)), np.uint8)
    g = torch.Generator().manual_seed(2)
    v = torch.randn((1, 4, 1, 64), generator=g).bfloat16()
    m.store(data, None, [4], torch.ones((1, 4, 1, 64)).bfloat16(), v)
    q = torch.randn((1, 4, 1, 64), generator=g).bfloat16()
    out, lse, _ = m.attend(data, None, [4], q, 0.5)
    c, s, z = m.held(data, None, 0, 0, 4, True)
    val = s[:, None] * c + z[:, None]
    logit = m.from_bits(m.bits(q))[0, :, 0].sum(-1) * 0.5
    for i in range(4):
        assert np.allclose(out[0, i, 0], val[: i + 1].mean(0), atol=1e-12)
        assert np.isclose(lse[0, i, 0], logit[i] + np.log(i + 1))


def test_acceptance_follows_the_target_distribution():
    """Over many uniforms the first emitted token has the target's distribution (speculative sampling's invariant)."""
    rng = np.random.default_rng(3)
    v, n = 6, 40000
    p = rng.dirichlet(np.ones(v), size=2)
    q = rng.dirichlet(np.ones(v))
    x = rng.choice(v, size=(n, 1), p=q)
    tok, acc = m.accept(np.broadcast_to(p, (n, 2, v)), np.broadcast_to(q, (n, 1, v)), x,
                        rng.random((n, 1)), rng.random(n))
    freq = np.bincount(tok[:, 0], minlength=v) / n
    # five standard deviations of a frequency
    assert (np.abs(freq - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / n)).all()
    second = np.bincount(tok[acc == 1, 1], minlength=v) / (acc == 1).sum()
    assert (np.abs(second - p[1]) < 5 * np.sqrt(p[1] * (1 - p[1]) / (acc == 1).sum())).all()


def test_acceptance_edges():
    p = np.zeros((1, 3, 4))
    p[0, :, 2] = 1.0
    u, w = np.array([[0.999, 0.0]]), np.array([0.0])
    assert m.accept(p, None, np.array([[2, 2]]), u, w)[0].tolist() == [[2, 2, 2]]      # greedy, all accepted
    assert m.accept(p, None, np.array([[2, 1]]), u, w)[0].tolist() == [[2, 2, -1]]     # greedy, second refused
    assert m.accept(p, None, np.array([[7, 1]]), u, w)[0].tolist() == [[2, -1, -1]]    # no such token
    assert m.accept(p, None, np.array([[2, 2]]), u, w, n=np.array([0]))[0].tolist() == [[2, -1, -1]]
    assert m.accept(0 * p, None, np.array([[2, 2]]), u, w)[0].tolist() == [[-1, -1, -1]]
    q = p[:, :2].copy()                                                               # p = q, refused by u = 1
    assert m.accept(p, q, np.array([[2, 2]]), np.array([[1.0, 0.0]]), w)[0].tolist() == [[2, -1, -1]]
