"""The 4-bit KV cache on the GPU against the 64-bit model (tests/kvq_model.py).

Append and read are bit-exact.  Attention: the output is a weighted mean of
held values; what separates it from the model is
  - the rounding of the result to bf16: at most 2^-8 of it;
  - the rounding of the weights to fp16 for the tensor cores: at most 2^-11 of
    each, so at most 2^-11 of `size` = sum_j w_j (s_j c_jd + |z_j|), twice (numerator
    and normaliser);
  - fp32 arithmetic of the logits: a logit of magnitude up to 64 in log2 units is
    off by at most D additions' 2^-24 of it and the exponential by 2^-22, below
    2^-11 together at these sizes (|logit| < 40).
lse: fp32 logits and logarithm, within 2^-12 here (values below 64).
"""
import numpy as np
import pytest
import torch

import kvq_model as m
from parity import gpu
from speculative_decoding_attention_gb300 import wm

pytestmark = pytest.mark.gpu

BAD_LENGTH, BAD_PAGE, TIMEOUT = 1, 2, 3


def table(batch, max_pages, extra, gen):
    n = batch * max_pages + extra
    return n, torch.randperm(n, generator=gen)[: batch * max_pages].view(batch, max_pages).to(torch.int32)


def empty_cache(lens, hkv, d, page, gen, dev, cap=None):
    """A cache of random bytes (stale contents) and its host copy."""
    cap = max(lens + [1]) if cap is None else cap
    if page:
        outer, bt = table(len(lens), -(-cap // page), 2, gen)
        blocks = page // 64
    else:
        outer, bt, blocks = len(lens), None, -(-cap // 64)
    data = torch.randint(0, 256, (outer, hkv, blocks, m.rec_bytes(d)), generator=gen, dtype=torch.uint8)
    cache = wm.KVQCache(data.to(dev), torch.tensor(lens, dtype=torch.int64, device=dev),
                        None if bt is None else bt.to(dev))
    return cache, data.numpy(), None if bt is None else bt.numpy()


def rows(shape, gen, gain=1.0):
    return (torch.randn(shape, generator=gen) * gain).bfloat16()


def filled(lens, hkv, d, page, gen, dev, gain=1.0, cap=None):
    """A cache whose positions 0..lens[b]-1 were appended on the GPU, checked bit for bit against the model."""
    cache, data, bt = empty_cache(lens, hkv, d, page, gen, dev, cap)
    n = max(lens + [1])
    k, v = rows((len(lens), n, hkv, d), gen, gain), rows((len(lens), n, hkv, d), gen)
    wm.kvq_append(cache, k.to(dev), v.to(dev))
    m.store(data, bt, lens, k, v)
    assert np.array_equal(cache.data.cpu().numpy(), data)
    return cache, data, bt


def check_attn(cache, data, bt, lens, t, g, gen, dev, scale=None, q_gain=1.0, q=None):
    d = cache.head_dim
    scale = d ** -0.5 if scale is None else scale
    q = rows((len(lens), t, cache.n_kv_heads * g, d), gen, q_gain) if q is None else q
    out, lse = wm.verify_attn_kvq(cache, q.to(dev), scale)
    assert wm.get_device_error() == 0
    ref, ref_lse, size = m.attend(data, bt, lens, q, scale)
    got, got_lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    bound = 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * size
    err = np.abs(got - ref)
    assert (err <= bound).all(), (np.unravel_index((err - bound).argmax(), err.shape), err.max())
    fin = np.isfinite(ref_lse)
    assert np.array_equal(fin, np.isfinite(got_lse))
    assert (np.abs(got_lse[fin] - ref_lse[fin]) <= 2.0 ** -12).all()
    assert (got_lse[~fin] == -np.inf).all() and (got[~fin] == 0).all()
    return out, lse, q


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [0, 64, 192])
@pytest.mark.parametrize("lens,n", [([1], 1), ([64, 65, 128], 1), ([5, 0, 130, 67], 3), ([200, 77], 77),
                                    ([63, 1, 300], 64)])
def test_append_is_bit_exact(d, page, lens, n):
    dev = gpu()
    gen = torch.Generator().manual_seed(d + page + n)
    cache, data, bt = empty_cache(lens, 3, d, page, gen, dev)
    k = rows((len(lens), n, 3, d), gen) * torch.exp(torch.randn((1, 1, 3, d), generator=gen)).bfloat16()
    v = rows((len(lens), n, 3, d), gen, 1e-3)
    wm.kvq_append(cache, k.to(dev), v.to(dev))
    m.store(data, bt, lens, k, v)
    assert np.array_equal(cache.data.cpu().numpy(), data)  # other positions and pages keep their bytes
    assert wm.get_device_error() == 0


@pytest.mark.parametrize("kind", ["constant", "zero", "ties", "tiny", "huge", "outlier", "border", "offset"])
def test_append_of_special_rows(kind):
    dev = gpu()
    gen = torch.Generator().manual_seed(7)
    x = torch.randn((1, 64, 2, 128), generator=gen)
    if kind == "constant":
        x[:] = -2.5
    elif kind == "zero":
        x[:] = 0
    elif kind == "ties":  # quotients that end in a half
        x = torch.randint(0, 31, x.shape, generator=gen).float() / 2
        x[..., 0], x[..., 1] = 0, 15
    elif kind == "tiny":
        x = x * 1e-38
    elif kind == "huge":
        x = x.clamp(-3, 3) * 1e38
    elif kind == "outlier":
        x[..., 5] *= 1e4
    elif kind == "border":  # -z / s a half, and values a hair off it
        x = torch.randint(-1, 2, x.shape, generator=gen).float() * 1e-30
        x[..., 0], x[..., 1] = -7.5, 7.5
    else:
        x = x * 2 ** -7 + 4
    x = x.bfloat16()
    cache, data, bt = empty_cache([64], 2, 128, 0, gen, dev)
    wm.kvq_append(cache, x.to(dev), (-x).to(dev))
    m.store(data, bt, [64], x, -x)
    assert np.array_equal(cache.data.cpu().numpy(), data)


def test_rows_with_nan_or_infinity_become_nan():
    dev = gpu()
    gen = torch.Generator().manual_seed(8)
    x = torch.randn((1, 4, 1, 64), generator=gen).bfloat16()
    x[0, 1, 0, 9], x[0, 2, 0, 3] = float("nan"), float("-inf")
    cache, data, _ = empty_cache([4], 1, 64, 0, gen, dev)
    wm.kvq_append(cache, x.to(dev), x.to(dev))
    k, v = wm.kvq_read(cache, 4)
    for y in (k, v):
        assert torch.isnan(y[0, 1:3]).all() and torch.isfinite(y[0, ::3]).all()


def test_append_one_by_one_equals_append_at_once():
    dev = gpu()
    gen = torch.Generator().manual_seed(9)
    k, v = rows((2, 70, 2, 128), gen).to(dev), rows((2, 70, 2, 128), gen).to(dev)
    a = wm.KVQCache.create(2, 2, 128, 70, dev)
    a.seq_lens.fill_(70)
    wm.kvq_append(a, k, v)
    b = wm.KVQCache.create(2, 2, 128, 70, dev)
    for i in range(70):
        b.seq_lens.fill_(i + 1)
        wm.kvq_append(b, k[:, i:i + 1].contiguous(), v[:, i:i + 1].contiguous())
    assert torch.equal(a.data, b.data)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [0, 128])
@pytest.mark.parametrize("n", [1, 3, 64, 150])
def test_read_gives_the_held_values(d, page, n):
    dev = gpu()
    gen = torch.Generator().manual_seed(d + n)
    lens = [150, 1, 64, 0, 97]
    cache, data, bt = filled(lens, 2, d, page, gen, dev)
    k, v = wm.kvq_read(cache, n)
    for is_v, got in ((False, k), (True, v)):
        want = np.zeros((len(lens), n, 2, d))
        for b, ln in enumerate(lens):
            for h in range(2):
                c, s, z = m.held(data, bt, b, h, ln, is_v)
                val = s[:, None] * c + z[:, None]
                take = min(n, ln)
                want[b, n - take:, h] = val[ln - take:]
        # one rounding to bf16 (2^-8) after fp32's
        err = np.abs(got.float().cpu().numpy() - want)
        assert (err <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want)).all()
    assert wm.get_device_error() == 0


def test_bad_lengths_and_pages_are_recorded_and_skipped():
    dev = gpu()
    gen = torch.Generator().manual_seed(11)
    cache, data, bt = empty_cache([100, 100, 100], 1, 64, 64, gen, dev)
    cache.seq_lens.copy_(torch.tensor([-1, 129, 100]))
    k = rows((3, 2, 1, 64), gen)
    wm.kvq_append(cache, k.to(dev), k.to(dev))
    assert wm.get_device_error() == BAD_LENGTH
    want = data.copy()
    m.store(want, bt[2:], [100], k[2:], k[2:])
    assert np.array_equal(cache.data.cpu().numpy(), want)
    cache.seq_lens.fill_(100)
    cache.block_table[0, 1] = 99
    cache.block_table[1, 1] = -1
    wm.kvq_append(cache, k.to(dev), k.to(dev))
    assert wm.get_device_error() == BAD_PAGE
    assert np.array_equal(cache.data.cpu().numpy(), want)
    kr, vr = wm.kvq_read(cache, 2)
    assert wm.get_device_error() == BAD_PAGE
    assert (kr[:2] == 0).all() and (vr[:2] == 0).all() and (kr[2] != 0).any()


# ------------------------------------------------------------------ attention

SHAPES = [(64, 1, 1), (64, 4, 3), (64, 8, 8), (128, 1, 1), (128, 4, 1), (128, 8, 4), (128, 8, 5), (128, 16, 4),
          (256, 2, 3), (256, 8, 4), (256, 8, 6), (256, 8, 8)]


@pytest.mark.parametrize("d,g,t", SHAPES)
@pytest.mark.parametrize("page", [0, 64, 256])
def test_attention_over_ragged_batches(d, g, t, page):
    dev = gpu()
    gen = torch.Generator().manual_seed(d + g + t + page)
    lens = [700, 0, 130, 128, 1, 129, 64, 2, 333]
    cache, data, bt = filled(lens, 2, d, page, gen, dev)
    check_attn(cache, data, bt, lens, t, g, gen, dev)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 1000, 4097])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_of_one_sequence(n, d):
    dev = gpu()
    gen = torch.Generator().manual_seed(n + d)
    cache, data, bt = filled([n], 1, d, 0, gen, dev)
    check_attn(cache, data, bt, [n], 2, 4, gen, dev)


@pytest.mark.parametrize("d,t", [(64, 1), (128, 5), (256, 2)])
def test_many_short_sequences(d, t):
    """More units than CTAs: a CTA's run crosses many units."""
    dev = gpu()
    gen = torch.Generator().manual_seed(d)
    lens = torch.randint(0, 40, (300,), generator=gen).tolist()
    cache, data, bt = filled(lens, 2, d, 64, gen, dev)
    check_attn(cache, data, bt, lens, t, 2, gen, dev)


def test_one_long_sequence_among_tiny_ones():
    dev = gpu()
    gen = torch.Generator().manual_seed(3)
    lens = [1] * 30 + [6000] + [0] * 20 + [2] * 13
    cache, data, bt = filled(lens, 1, 128, 64, gen, dev)
    check_attn(cache, data, bt, lens, 3, 4, gen, dev)


def test_empty_batch():
    dev = gpu()
    gen = torch.Generator().manual_seed(4)
    cache, data, bt = empty_cache([0, 0, 0], 2, 128, 64, gen, dev, cap=128)
    check_attn(cache, data, bt, [0, 0, 0], 2, 2, gen, dev)


@pytest.mark.parametrize("kind", ["uniform", "peaked", "sink", "offset", "constant_v", "mixed_v"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_of_special_distributions(kind, d):
    """Weights that are all equal, one key far above the rest, values whose zero is large beside their step, rows of
    constant values (scale 0) beside others."""
    dev = gpu()
    gen = torch.Generator().manual_seed(5)
    n = 2000
    k, v = torch.randn((1, n, 1, d), generator=gen), torch.randn((1, n, 1, d), generator=gen)
    q = torch.randn((1, 2, 4, d), generator=gen)
    if kind == "uniform":
        q[:] = 0
    elif kind == "peaked":
        k[:, ::97] *= 8
    elif kind == "sink":  # one key 14 above a mass of equal ones
        k[:] = 0
        k[0, 0, 0] = q[0, 0, 0] * 14 / (q[0, 0, 0] ** 2).sum() * d ** 0.5
    elif kind == "offset":
        v = v * 2 ** -6 + 3
    elif kind == "constant_v":
        v[:] = torch.randn((1, n, 1, 1), generator=gen)
    else:
        v[:, ::2] = torch.randn((1, n // 2, 1, 1), generator=gen)
        v[:, 1::4] *= 1e-3
    k, v = k.bfloat16(), v.bfloat16()
    cache, data, bt = empty_cache([n], 1, d, 0, gen, dev)
    wm.kvq_append(cache, k.to(dev), v.to(dev))
    m.store(data, bt, [n], k, v)
    check_attn(cache, data, bt, [n], 2, 4, gen, dev, q=q.bfloat16())


@pytest.mark.parametrize("gain", [1e-12, 1e-3, 1e3, 1e12])
def test_scales_of_values_and_queries(gain):
    """Outputs follow the values' magnitude; logits do not depend on how q and the scale share theirs."""
    dev = gpu()
    gen = torch.Generator().manual_seed(6)
    lens = [300]
    cache, data, bt = empty_cache(lens, 1, 128, 0, gen, dev)
    k, v = rows((1, 300, 1, 128), gen), rows((1, 300, 1, 128), gen, gain)
    wm.kvq_append(cache, k.to(dev), v.to(dev))
    m.store(data, bt, lens, k, v)
    check_attn(cache, data, bt, lens, 1, 4, gen, dev, scale=128 ** -0.5 / gain, q_gain=gain)


def test_bytes_past_the_length_do_not_matter():
    """NaN scales past the end and, for a row, past its causal boundary."""
    dev = gpu()
    gen = torch.Generator().manual_seed(12)
    lens = [100, 128, 190]
    cache, data, bt = filled(lens, 1, 128, 64, gen, dev, cap=256)
    d = 128
    q = rows((3, 4, 2, d), gen)
    ref, _ = wm.verify_attn_kvq(cache, q.to(dev), 0.1)
    for b, n in enumerate(lens):
        for pos in list(range(n - 1, 256)):
            rec, r = m.record(data, bt, b, 0, pos // 64), pos % 64
            rec[64 * d:].view(np.uint16).reshape(2, 64, 2)[:, r] = 0x7FFF  # NaN
            at, sh = m._addr(d, True, r)
            rec[at] |= (0xF << sh).astype(np.uint8)
    cache.data.copy_(torch.from_numpy(data))
    out, _ = wm.verify_attn_kvq(cache, q.to(dev), 0.1)
    assert torch.isnan(out[:, 3]).all()                # its own key is NaN
    assert torch.equal(out[:, :3], ref[:, :3])         # the rows before do not see it


def test_nan_queries_stay_in_their_rows():
    dev = gpu()
    gen = torch.Generator().manual_seed(13)
    lens = [300]
    cache, data, bt = filled(lens, 1, 128, 0, gen, dev)
    q = rows((1, 2, 4, 128), gen)
    ref, _ = wm.verify_attn_kvq(cache, q.to(dev), 0.1)
    q[0, 1, 2, 7] = float("nan")
    out, lse = wm.verify_attn_kvq(cache, q.to(dev), 0.1)
    assert torch.isnan(out[0, 1, 2]).all() and torch.isnan(lse[0, 1, 2])
    keep = torch.ones((2, 4), dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[0][keep.to(dev)], ref[0][keep.to(dev)])


def test_attention_reports_bad_lengths_and_pages():
    dev = gpu()
    gen = torch.Generator().manual_seed(14)
    lens = [100, 100]
    cache, data, bt = filled(lens, 1, 64, 64, gen, dev)
    q = rows((2, 1, 2, 64), gen).to(dev)
    cache.seq_lens[0] = 129
    wm.verify_attn_kvq(cache, q, 0.1)
    assert wm.get_device_error() == BAD_LENGTH
    cache.seq_lens[0] = 100
    cache.block_table[0, 1] = 77
    out, _ = wm.verify_attn_kvq(cache, q, 0.1)
    assert wm.get_device_error() == BAD_PAGE
    ref, _, size = m.attend(data, bt[1:], lens[1:], q[1:].cpu(), 0.1)
    assert (np.abs(out[1:].float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * size).all()


def test_workspace_needs_no_contents_and_calls_repeat_bit_for_bit():
    dev = gpu()
    gen = torch.Generator().manual_seed(15)
    lens = [900, 17, 300]
    cache, data, bt = filled(lens, 2, 128, 64, gen, dev)
    q = rows((3, 2, 8, 128), gen).to(dev)
    ws = wm.kvq_workspace(cache, 8, 2)
    ref = None
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out, lse = wm.verify_attn_kvq(cache, q, 0.1, workspace=ws)
        if ref is None:
            ref = (out, lse)
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])


def test_other_streams_and_graphs():
    """A call on another stream than the current one, and a captured call replayed after the lengths and the contents
    changed on the device; two graphs with workspaces of their own."""
    dev = gpu()
    gen = torch.Generator().manual_seed(16)
    lens = [500, 20]
    cache, data, bt = filled(lens, 1, 128, 64, gen, dev, cap=640)
    q = rows((2, 2, 4, 128), gen).to(dev)
    ref, ref_lse = wm.verify_attn_kvq(cache, q, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = wm.verify_attn_kvq(cache, q, 0.1, stream=side)
    out2, _ = wm.verify_attn_kvq(cache, q, 0.1, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(out2, ref)
    graphs, outs = [], []
    k1, v1 = rows((2, 3, 1, 128), gen), rows((2, 3, 1, 128), gen)
    kd, vd = k1.to(dev), v1.to(dev)
    for i in range(2):
        ws = wm.kvq_workspace(cache, 4, 2)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wm.kvq_append(cache, kd, vd)
            outs.append(wm.verify_attn_kvq(cache, q, 0.1, workspace=ws))
        graphs.append((g, ws))
    lens = [503, 23]
    cache.seq_lens.copy_(torch.tensor(lens))
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    m.store(data, bt, lens, k1, v1)
    assert np.array_equal(cache.data.cpu().numpy(), data)
    r, _, size = m.attend(data, bt, lens, q.cpu(), 0.1)
    for o, _ in outs:
        assert (np.abs(o.float().cpu().numpy() - r) <= 2.0 ** -8 * np.abs(r) + 3 * 2.0 ** -11 * size).all()
    assert torch.equal(outs[0][0], outs[1][0])


def test_records_past_four_gigabytes():
    """Offsets beyond 32 bits: pages at the far end of a 5 GB pool."""
    dev = gpu()
    gen = torch.Generator().manual_seed(17)
    d, n_pages = 256, 320000
    data = torch.zeros((n_pages, 1, 1, m.rec_bytes(d)), dtype=torch.uint8, device=dev)
    bt = torch.tensor([[n_pages - 1, 3, n_pages - 2]], dtype=torch.int32, device=dev)
    cache = wm.KVQCache(data, torch.tensor([150], device=dev), bt)
    k, v = rows((1, 150, 1, d), gen), rows((1, 150, 1, d), gen)
    wm.kvq_append(cache, k.to(dev), v.to(dev))
    small = np.zeros((3, 1, 1, m.rec_bytes(d)), np.uint8)
    m.store(small, np.array([[0, 1, 2]]), [150], k, v)
    assert np.array_equal(data[bt[0].long()].cpu().numpy(), small)
    q = rows((1, 1, 4, d), gen)
    out, _ = wm.verify_attn_kvq(cache, q.to(dev), 0.06)
    ref, _, size = m.attend(small, np.array([[0, 1, 2]]), [150], q, 0.06)
    assert (np.abs(out.float().cpu().numpy() - ref) <= 2.0 ** -8 * np.abs(ref) + 3 * 2.0 ** -11 * size).all()


def test_pages_shared_by_two_sequences_can_be_read():
    dev = gpu()
    gen = torch.Generator().manual_seed(18)
    cache, data, bt = filled([192, 192], 1, 64, 64, gen, dev)
    bt[1, :2] = bt[0, :2]
    cache.block_table.copy_(torch.from_numpy(bt))
    check_attn(cache, data, bt, [192, 192], 2, 2, gen, dev)
