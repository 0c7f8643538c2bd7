"""Attention over the 4-bit KV cache where one CTA's part of a sequence is long.

The cache is paged, and its block tables name the same eight pages again and again, so
millions of positions have a model of 512: each held row with the number of times that
it is seen.  Bounds as in test_gpu_kvq.py, and one more, for the tensor cores' sums:
an addition that cuts off loses less than one unit in the last of 24 bits, 2^-23 of
the sum; over the 32 tiles of one accumulator, 32 additions each, the sum is half its
last value on average, so at most 1024 x 2^-23 / 2 = 2^-14 of the magnitudes is lost.
(A single accumulator over 1028 tiles was seen to lose 2^-9.8 of them.)
"""
import numpy as np
import pytest
import torch

import kvq_model as m
from parity import gpu
from speculative_decoding_attention_gb300 import wm

pytestmark = pytest.mark.gpu

PAGES, LONG, LONGEST = 8, 4_999_999, 20_000_001


def model(data, bt, lens, q, scale):
    """(out, lse, size, spread): as kvq_model.attend, by counting; spread = sum_j w_j s_j |c_jd - 8|."""
    b_n, t, hq, d = q.shape
    hkv = data.shape[1]
    g = hq // hkv
    out, size, spread = (np.zeros((b_n, t, hq, d)) for _ in range(3))
    lse = np.full((b_n, t, hq), -np.inf)
    qf = m.from_bits(m.bits(q))
    every = np.arange(PAGES, dtype=np.int32)[None]
    for h in range(hkv):
        ck, sk, zk = m.held(data, every, 0, h, 64 * PAGES, False)
        cv, sv, zv = m.held(data, every, 0, h, 64 * PAGES, True)
        keys = sk[:, None] * ck + zk[:, None]
        vals = sv[:, None] * cv + zv[:, None]
        for b in range(b_n):
            at = (bt[b, :, None] * 64 + np.arange(64)).reshape(-1)  # page row of every position
            for i in range(t):
                n = int(lens[b]) - t + i + 1
                if n <= 0:
                    continue
                times = np.bincount(at[:n], minlength=64 * PAGES).astype(np.float64)
                for r in range(h * g, (h + 1) * g):
                    x = keys @ qf[b, i, r] * scale
                    top = x[times > 0].max()
                    w = np.where(times > 0, times * np.exp(x - top), 0.0)
                    lse[b, i, r] = top + np.log(w.sum())
                    w /= w.sum()
                    out[b, i, r] = w @ vals
                    size[b, i, r] = w @ (sv[:, None] * cv + np.abs(zv)[:, None])
                    spread[b, i, r] = w @ (sv[:, None] * np.abs(cv - 8))
    return out, lse, size, spread


def setup(kind, lens, hkv, g, t, d, gen, dev):
    """The cache, its host copy, the queries and their scale."""
    k = torch.randn((1, 64 * PAGES, hkv, d), generator=gen)
    v = torch.randn((1, 64 * PAGES, hkv, d), generator=gen)
    q = torch.randn((len(lens), t, hkv * g, d), generator=gen)
    scale = d ** -0.5
    entries = -(-max(lens) // 64)
    if kind == "level":
        # Equal weights, and values whose codes are far from the middle while their mean is near 0:
        # about step s from -13 s, codes 12 to 15 and a single 0 in every row.  s is at most 1/4,
        # and 1/4 in every page's first row: the weights that meet the codes, 512 s, then have
        # bf16's 8 bits and are exact in fp16.
        c = torch.randint(12, 16, v.shape, generator=gen)
        c[:, :, :, 0] = 15
        c.view(-1, d)[torch.arange(c.numel() // d), 1 + torch.arange(c.numel() // d) % (d - 1)] = 0
        s = 0.03 + 0.21 * torch.rand(v.shape[:3], generator=gen)
        s[:, ::64] = 0.25
        v, q = (c - 13) * s[..., None], torch.zeros_like(q)
    if kind == "rising":
        # Logits of page p near 5.8 p: each next page raises the maxima by more than 8 in log2 units.
        u = torch.full((d,), d ** -0.5)
        k = 0.1 * k + torch.arange(PAGES).repeat_interleave(64).view(1, -1, 1, 1) * u
        q, scale = 5.8 * u + 0.1 * q * u, 1.0
        page = torch.arange(entries) // 300 % PAGES
    else:
        page = torch.randint(0, PAGES, (entries,), generator=gen)
    bt = torch.stack([page.roll(7 * b) for b in range(len(lens))]).to(torch.int32)
    data = np.zeros((PAGES, hkv, 1, m.rec_bytes(d)), np.uint8)
    every = torch.arange(PAGES, dtype=torch.int32)[None]
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    m.store(data, every.numpy(), [64 * PAGES], k, v)
    pool = torch.from_numpy(data).to(dev)
    return wm.KVQCache(pool, torch.tensor(lens, device=dev), bt.to(dev)), data, bt.numpy(), q, scale


@pytest.mark.parametrize("kind", ["random", "level", "rising"])
@pytest.mark.parametrize("lens,hkv,g,t,d", [
    ([LONG], 2, 4, 1, 64),               # 257 tiles a part; up to 16 rows
    ([LONGEST], 2, 4, 1, 64),            # 1028
    ([LONG], 2, 8, 3, 64),               # 32
    ([LONG, 0, 130], 1, 16, 3, 128),     # 48; the long one, an empty one and a short one
    ([LONG], 2, 4, 4, 128),
    ([LONG // 2, 70_001], 2, 8, 4, 256),
    ([LONG // 2], 2, 4, 2, 256),
    ([LONG], 2, 16, 4, 64),              # 64
])
def test_long_parts(kind, lens, hkv, g, t, d):
    dev = gpu()
    gen = torch.Generator().manual_seed(d + g + t)
    cache, data, bt, q, scale = setup(kind, lens, hkv, g, t, d, gen, dev)
    out, lse = wm.verify_attn_kvq(cache, q.to(dev), scale)
    again = wm.verify_attn_kvq(cache, q.to(dev), scale)
    assert wm.get_device_error() == 0
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    ref, ref_lse, size, spread = model(data, bt, lens, q, scale)
    got, got_lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    # level: the weights are exact
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * spread + (0 if kind == "level" else 3 * 2.0 ** -11 * size)
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), (np.unravel_index((err - bound).argmax(), err.shape), err.max(), (err / bound).max())
    fin = np.isfinite(ref_lse)
    assert np.array_equal(fin, np.isfinite(got_lse)) and (got[~fin] == 0).all()
    assert (np.abs(got_lse[fin] - ref_lse[fin]) <= 2.0 ** -12).all()
