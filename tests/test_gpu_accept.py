"""Acceptance of drafted tokens on the GPU against the 64-bit model: whole numbers, equal."""
import numpy as np
import pytest
import torch

import kvq_model as m
from parity import gpu
from speculative_decoding_attention_gb300 import wm

pytestmark = pytest.mark.gpu

BAD_LENGTH, BAD_TOKEN, BAD_PROB = 1, 5, 6


def make(b, k, v, gen, noise=1.0, sharp=2.5):
    logits = torch.randn((b, k + 1, v), generator=gen) * sharp
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :k] + noise * torch.randn((b, k, v), generator=gen), -1)
    x = torch.multinomial(q.reshape(b * k, v), 1, generator=gen).view(b, k).to(torch.int32)
    return p, q, x, torch.rand((b, k), generator=gen), torch.rand((b,), generator=gen)


def run(p, q, x, u, w, n=None, lens=None):
    dev = gpu()
    d = lambda t: None if t is None else t.to(dev)  # noqa: E731
    return wm.spec_accept(d(p), d(q), d(x), d(u), d(w), n_draft=d(n), seq_lens=d(lens))


def check(p, q, x, u, w, n=None):
    lens = torch.arange(p.shape[0]) + 1000
    tok, acc, new = run(p, q, x, u, w, n, lens)
    rt, ra = m.accept(p.numpy(), None if q is None else q.numpy(), x.numpy(), u.numpy(), w.numpy(),
                      None if n is None else n.numpy())
    assert acc.cpu().numpy().tolist() == ra.tolist()
    assert tok.cpu().numpy().tolist() == rt.tolist()
    assert new.cpu().numpy().tolist() == (lens.numpy() - x.shape[1] + ra).tolist()
    return tok, acc


@pytest.mark.parametrize("v", [1, 2, 31, 33, 1000, 4097, 50001, 131072])
@pytest.mark.parametrize("b,k", [(1, 1), (3, 4), (33, 7)])
@pytest.mark.parametrize("probs", [True, False])
def test_matches_the_model(v, b, k, probs):
    gen = torch.Generator().manual_seed(v + b + k)
    p, q, x, u, w = make(b, k, v, gen)
    check(p, q if probs else None, x, u, w)
    assert wm.get_device_error() == 0


@pytest.mark.parametrize("noise", [0.0, 0.1, 3.0])
def test_ragged_drafts(noise):
    gen = torch.Generator().manual_seed(1)
    p, q, x, u, w = make(64, 6, 777, gen, noise)
    n = torch.randint(0, 7, (64,), generator=gen).to(torch.int32)
    # what lies past a sequence's drafts is not read
    for b in range(64):
        x[b, n[b]:] = -5
        q[b, n[b]:] = float("nan")
        p[b, n[b] + 1:] = float("nan")
        u[b, n[b]:] = float("nan")
    tok, acc = check(p, q, x, u, w, n)
    assert wm.get_device_error() == 0
    if noise == 0.0:
        assert acc.cpu().tolist() == n.tolist()  # p = q: every draft is accepted


@pytest.mark.parametrize("b", [60, 77, 153, 305, 700])
@pytest.mark.parametrize("probs", [True, False])
def test_batches_of_every_cluster_size(b, probs):
    """8 CTAs per sequence down to one, and more sequences than are resident at once."""
    gen = torch.Generator().manual_seed(b)
    p, q, x, u, w = make(b, 2, 1301, gen)
    check(p, q if probs else None, x, u, w)


def test_smallest_probabilities_are_compared_exactly():
    gen = torch.Generator().manual_seed(5)
    b = 512
    tiny = lambda lo, hi: torch.randint(lo, hi, (b,), generator=gen).double() * 2.0 ** -149  # noqa: E731
    p, q = torch.zeros((b, 2, 3)), torch.zeros((b, 1, 3))
    p[:, 0, 0], q[:, 0, 0] = tiny(0, 6).float(), tiny(1, 9).float()
    p[:, 0, 1], p[:, 1, 2], q[:, 0, 1] = 1.0, 1.0, 1.0
    u = torch.randint(0, 1 << 24, (b, 1), generator=gen).float() * 2.0 ** -24
    u[::4] = 0.5 + 2.0 ** -24
    u[1::4] = 0.5
    u[2::4] = 0.5 - 2.0 ** -25
    check(p, q, torch.zeros((b, 1), dtype=torch.int32), u, torch.rand((b,), generator=gen))


def test_more_drafts_than_a_warp():
    gen = torch.Generator().manual_seed(2)
    p, q, x, u, w = make(5, 70, 300, gen, noise=0.0)
    u[1, 40], q[1, 40] = 0.9, 1.0
    u[2, 0], q[2, 0] = 0.9, 1.0
    check(p, q, x, u, w)


def test_thresholds_at_the_ends_and_on_borders():
    """w = 0, w next to 1, and rows of equal exact entries, whose running sums meet the threshold exactly."""
    gen = torch.Generator().manual_seed(3)
    b, v = 64, 4096
    p, q, x, u, w = make(b, 2, v, gen)
    w[:8], w[8:16] = 0.0, 1.0 - 2.0 ** -24
    p[16:] = 1.0 / v
    u[16:] = 0.0
    w[16:] = torch.arange(b - 16) / 64
    check(p, q, x, u, w)


def test_greedy_verification():
    """One-hot target rows: drafts are accepted while they are the target's choice, and the next choice follows."""
    gen = torch.Generator().manual_seed(4)
    b, k, v = 40, 5, 1003
    best = torch.randint(0, v, (b, k + 1), generator=gen)
    p = torch.nn.functional.one_hot(best, v).float()
    x = best[:, :k].clone().to(torch.int32)
    miss = torch.rand((b, k), generator=gen) < 0.3
    x[miss] = (x[miss] + 1) % v
    tok, acc = check(p, None, x, torch.rand((b, k), generator=gen), torch.rand((b,), generator=gen))
    for i in range(b):
        a = int(acc[i])
        assert tok[i, : a + 1].cpu().tolist() == best[i, : a + 1].tolist()


def test_zero_residual_falls_back_to_the_target():
    gen = torch.Generator().manual_seed(5)
    p, q, x, u, w = make(6, 2, 500, gen)
    q = p[:, :2].clone()
    u[:] = 1.0  # refused although p = q
    check(p, q, x, u, w)
    # a small residual, far below the row's own weight
    q[:, 0] = p[:, 0] * (1 + 2.0 ** -22)
    q[:, 0, 77] = p[:, 0, 77] * 0.5
    x[:, 0] = 5
    check(p, q, x, u, w)


def test_bad_values_count_as_documented():
    gen = torch.Generator().manual_seed(6)
    p, q, x, u, w = make(8, 3, 640, gen)
    p[:, :, 3::50], q[:, :, 9::60], p[:, :, 11] = float("nan"), -1.0, float("-inf")
    p[0, :, 12] = float("inf")
    w[1], w[2], u[3] = float("nan"), -2.0, 3.0
    check(p, q, x, u, w)


def test_bad_tokens_counts_and_empty_rows_are_recorded():
    gen = torch.Generator().manual_seed(7)
    p, q, x, u, w = make(4, 3, 100, gen)
    x[1, 1], u[1] = 100, 0.0
    x[2, 0] = -1
    check(p, q, x, u, w)
    assert wm.get_device_error() == BAD_TOKEN
    x = x.clamp(0, 99)
    check(p, q, x, u, w, torch.tensor([3, -1, 9, 2], dtype=torch.int32))
    assert wm.get_device_error() == BAD_LENGTH
    p[3] = 0.0
    tok, acc = check(p, q, x, u, w)
    assert wm.get_device_error() == BAD_PROB and int(acc[3]) == 0 and int(tok[3, 0]) == -1


def test_lengths_in_place_streams_and_graphs():
    dev = gpu()
    gen = torch.Generator().manual_seed(8)
    p, q, x, u, w = (t.to(dev) for t in make(9, 3, 5000, gen))
    lens = torch.full((9,), 50, dtype=torch.int64, device=dev)
    tok, acc, new = wm.spec_accept(p, q, x, u, w, seq_lens=lens)
    assert torch.equal(new, lens - 3 + acc)
    assert wm.spec_accept(p, q, x, u, w)[2] is None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t2, a2, _ = wm.spec_accept(p, q, x, u, w, stream=side)
    side.synchronize()
    assert torch.equal(t2, tok) and torch.equal(a2, acc)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t3, a3, _ = wm.spec_accept(p, q, x, u, w, seq_lens=lens, new_len=lens)
    u.zero_()
    g.replay()
    torch.cuda.synchronize()
    rt, ra = m.accept(p.cpu().numpy(), q.cpu().numpy(), x.cpu().numpy(), u.cpu().numpy(), w.cpu().numpy())
    assert t3.cpu().numpy().tolist() == rt.tolist()
    assert lens.cpu().numpy().tolist() == (50 - 3 + ra).tolist()


def test_tensors_of_the_wrong_type_or_shape_are_refused():
    dev = gpu()
    gen = torch.Generator().manual_seed(9)
    p, q, x, u, w = (t.to(dev) for t in make(2, 3, 50, gen))
    for bad in (dict(target_probs=p.double()), dict(target_probs=p[:, :3].contiguous()), dict(draft_probs=q[:, :2]),
                dict(draft_tokens=x.long()), dict(u_accept=u.cpu()), dict(u_sample=u),
                dict(target_probs=p.transpose(0, 1)), dict(new_len=torch.zeros(2, dtype=torch.int64, device=dev))):
        args = {**dict(target_probs=p, draft_probs=q, draft_tokens=x, u_accept=u, u_sample=w), **bad}
        with pytest.raises(ValueError):
            wm.spec_accept(**args)
