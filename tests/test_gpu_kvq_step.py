"""The 4-bit cache and the acceptance as a speculative step uses them: draft over the ring, append the proposed
tokens' K/V, verify over the 4-bit cache, accept, roll the ring back -- eagerly and as one captured graph replayed --
and the bounded waits of the attention."""
import math

import numpy as np
import pytest
import torch

import kvq_model as m
from parity import gpu
from speculative_decoding_attention_gb300 import wm

pytestmark = pytest.mark.gpu

TIMEOUT = 3


class Step:
    """Buffers of one step: B sequences, k drafts, a random 'model' that turns hidden rows into probabilities."""

    def __init__(self, dev, seed, lens, hkv, g, d, k, vocab, page):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.dev, self.gen, self.k, self.vocab = dev, gen, k, vocab
        b, per = len(lens), -(-max(lens) // page) + 2
        n_pages = b * per
        table = torch.randperm(n_pages, generator=gen, device=dev).view(b, per).to(torch.int32)
        data = torch.randint(0, 256, (n_pages, hkv, page // 64, wm.kvq_record_bytes(d)), generator=gen, device=dev,
                             dtype=torch.uint8)
        self.cache = wm.KVQCache(data, torch.zeros(b, dtype=torch.int64, device=dev), table)
        self.ring = wm.Ring.create(b, hkv, d, 4, 96, dev)
        self.ws, self.dws = wm.kvq_workspace(self.cache, hkv * g, k + 1), wm.step_workspace(self.ring, hkv * g)
        rnd = lambda *s: torch.randn(s, generator=gen, device=dev).bfloat16()  # noqa: E731
        self.rnd, self.shape = rnd, (b, hkv, g, d)
        self.lens = torch.tensor(lens, dtype=torch.int64, device=dev)
        # the prompt: every sequence's first positions, padded in front
        n = max(lens)
        k0, v0 = rnd(b, n, hkv, d), rnd(b, n, hkv, d)
        self.cache.seq_lens.copy_(self.lens)
        wm.kvq_append(self.cache, k0, v0)
        # the draft's ring from the tail that the cache holds
        kt, vt = wm.kvq_read(self.cache, n)
        hist = wm.KVCache(*(torch.stack([t[i].roll(lens[i] - n, 0) for i in range(b)]).transpose(1, 2).contiguous()
                            for t in (kt, vt)), self.lens.clone())
        wm.ring_fill(self.ring, hist)
        self.head = torch.randn((hkv * g * d, vocab), generator=gen, device=dev) / math.sqrt(hkv * g * d)
        self.new = torch.empty(b, dtype=torch.int64, device=dev)
        self.inputs()
        self.tokens = self.accepted = None

    def inputs(self):
        """Fresh values in the same buffers."""
        b, hkv, g, d = self.shape
        new = dict(kn=self.rnd(b, self.k + 1, hkv, d), vn=self.rnd(b, self.k + 1, hkv, d),
                   q=self.rnd(b, self.k + 1, hkv * g, d), kd=self.rnd(b, hkv, d), vd=self.rnd(b, hkv, d),
                   qd=self.rnd(b, hkv * g, d),
                   u=torch.rand((b, self.k), generator=self.gen, device=self.dev),
                   w=torch.rand((b,), generator=self.gen, device=self.dev),
                   noise=torch.randn((b, self.k, self.vocab), generator=self.gen, device=self.dev))
        for name, t in new.items():
            if hasattr(self, name):
                getattr(self, name).copy_(t)
            else:
                setattr(self, name, t)

    def run(self):
        self.draft_out, _ = wm.draft_step(self.ring, self.kd, self.vd, self.qd, 0.1, self.dws)
        self.cache.seq_lens.copy_(self.lens + self.k + 1)
        wm.kvq_append(self.cache, self.kn, self.vn)
        self.out, self.lse = wm.verify_attn_kvq(self.cache, self.q, 0.1, workspace=self.ws)
        logits = self.out.flatten(2).float() @ self.head * 20
        self.p = torch.softmax(logits, -1)
        self.qp = torch.softmax(logits[:, :-1] + self.noise, -1)
        self.x = (self.qp.cumsum(-1) < 0.5).sum(-1).clamp(max=self.vocab - 1).to(torch.int32)
        self.tokens, self.accepted, _ = wm.spec_accept(self.p, self.qp, self.x, self.u, self.w,
                                                       seq_lens=self.cache.seq_lens, new_len=self.new)
        wm.ring_rollback(self.ring, self.new)
        self.lens.copy_(self.new)

    def check(self, data, lens):
        """Against the models, from the cache's bytes and lengths before the step; returns both after it."""
        full = [n + self.k + 1 for n in lens]
        table = self.cache.block_table.cpu().numpy()
        m.store(data, table, full, self.kn.cpu(), self.vn.cpu())
        assert np.array_equal(self.cache.data.cpu().numpy(), data)
        ref, _, size = m.attend(data, table, full, self.q.cpu(), 0.1)
        err = np.abs(self.out.float().cpu().numpy() - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * size).all()  # see test_gpu_kvq.py
        rt, ra = m.accept(self.p.cpu().numpy(), self.qp.cpu().numpy(), self.x.cpu().numpy(), self.u.cpu().numpy(),
                          self.w.cpu().numpy())
        assert self.tokens.cpu().numpy().tolist() == rt.tolist()
        assert self.accepted.cpu().numpy().tolist() == ra.tolist()
        lens = [n + 1 + int(a) for n, a in zip(lens, ra)]
        assert self.lens.cpu().tolist() == lens
        seen = [min(s + 1, n) for s, n in zip(self.seen, lens)]  # one draft entry, then the rollback
        assert self.ring.n_seen.cpu().tolist() == seen
        self.seen = seen
        assert wm.get_device_error() == 0
        return data, lens


@pytest.mark.parametrize("hkv,g,d,k,page", [(2, 4, 128, 3, 64), (1, 8, 64, 2, 128), (2, 2, 256, 5, 64)])
def test_speculative_steps(hkv, g, d, k, page):
    dev = gpu()
    lens = [130, 61, 200]
    s = Step(dev, d + k, lens, hkv, g, d, k, 300, page)
    s.seen = list(lens)
    data = s.cache.data.cpu().numpy()
    for _ in range(4):
        s.inputs()
        s.run()
        data, lens = s.check(data, lens)
    # the same step as a graph: replayed on fresh inputs and grown lengths, among eager steps
    s.inputs()
    keep = [t.clone() for t in (s.lens, s.cache.data, s.ring.k, s.ring.v, s.ring.pos_tag, s.ring.n_seen)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for t, c in zip((s.lens, s.cache.data, s.ring.k, s.ring.v, s.ring.pos_tag, s.ring.n_seen), keep):
        t.copy_(c)
    for _ in range(4):
        s.inputs()
        graph.replay()
        torch.cuda.synchronize()
        data, lens = s.check(data, lens)


@pytest.mark.parametrize("d,g", [(64, 4), (128, 4), (128, 24), (256, 32), (256, 64)])
@pytest.mark.parametrize("tile", [0, 1, 3])
def test_attention_wait_times_out_then_next_call_is_clean(d, g, tile):
    """The copies stop at the run's 128-position tile `tile`: every role gives up, and the next call is as before."""
    dev = gpu()
    n = 152 * 512  # at least four such tiles for every CTA
    gen = torch.Generator(device=dev).manual_seed(d + g)
    cache = wm.KVQCache.create(1, 1, d, n, dev)
    cache.seq_lens.fill_(n)
    x = torch.randn((1, n, 1, d), generator=gen, device=dev).bfloat16()
    wm.kvq_append(cache, x, x.flip(1))
    q = torch.randn((1, 1, g, d), generator=gen, device=dev).bfloat16()
    ref, ref_lse = wm.verify_attn_kvq(cache, q, 0.1)
    assert wm.get_device_error() == 0
    wm.set_test_stall(tile, 4000)
    try:
        wm.verify_attn_kvq(cache, q, 0.1)
        torch.cuda.synchronize()
    finally:
        wm.set_test_stall(-1)
    assert wm.get_device_error() == TIMEOUT
    out, lse = wm.verify_attn_kvq(cache, q, 0.1)
    assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
    assert wm.get_device_error() == 0


@pytest.mark.parametrize("d,t", [(64, 1), (128, 3), (128, 6), (256, 2), (256, 4)])
def test_replays_are_bit_identical(d, t):
    """A race shows as a replay that differs: 100 replays over a ragged batch."""
    dev = gpu()
    gen = torch.Generator(device=dev).manual_seed(d + t)
    lens = [5000, 1, 300, 0, 2049, 700]
    cache = wm.KVQCache.create(6, 2, d, 5000, dev)
    cache.seq_lens.copy_(torch.tensor(lens))
    k, v = (torch.randn((6, 5000, 2, d), generator=gen, device=dev).bfloat16() for _ in range(2))
    wm.kvq_append(cache, k, v)
    q = torch.randn((6, t, 16, d), generator=gen, device=dev).bfloat16()
    ref, ref_lse = wm.verify_attn_kvq(cache, q, 0.1)
    out, lse = torch.empty_like(ref), torch.empty_like(ref_lse)
    ws = wm.kvq_workspace(cache, 16, t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        wm.verify_attn_kvq(cache, q, 0.1, out=out, lse=lse, workspace=ws)
    for _ in range(100):
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, ref_lse)
