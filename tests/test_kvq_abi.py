"""Refusals of the 4-bit cache's and the acceptance's entry points (no GPU needed): every bad argument is reported on
the host, before anything is enqueued."""
import ctypes

import pytest
import torch

from speculative_decoding_attention_gb300 import build as wm_build
from speculative_decoding_attention_gb300 import wm

P = ctypes.c_void_p
INV, UNS, WSP = wm.WM_ERR_INVALID_ARG, wm.WM_ERR_UNSUPPORTED, wm.WM_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    wm_build.build()
    return wm.load()


def kvq(paged=False, **over):
    c = wm._KVQ()
    c.data, c.seq_lens = 1 << 20, 2 << 20
    c.batch, c.n_kv_heads, c.head_dim = 2, 4, 128
    if paged:
        c.block_table, c.n_pages, c.page_size, c.max_pages = 3 << 20, 10, 64, 4
    else:
        c.n_cap = 256
    for k, v in over.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(data=None), INV), (dict(seq_lens=None), INV), (dict(batch=0), INV), (dict(n_kv_heads=0), INV),
    (dict(head_dim=96), UNS), (dict(data=(1 << 20) + 8), INV), (dict(seq_lens=(2 << 20) + 4), INV),
    (dict(n_cap=0), INV), (dict(n_cap=100), UNS), (dict(n_cap=1 << 31), UNS),
    (dict(batch=65536, n_kv_heads=1), UNS),
    (dict(paged=True, page_size=32), UNS), (dict(paged=True, page_size=0), INV), (dict(paged=True, n_pages=0), INV),
    (dict(paged=True, max_pages=0), INV), (dict(paged=True, block_table=(3 << 20) + 2), INV),
    (dict(paged=True, n_pages=1 << 31), UNS), (dict(paged=True, max_pages=1 << 26), UNS),
]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(lib, over, status):
    c = kvq(**over)
    r = ctypes.byref(c)
    assert lib.wm_kvq_append(r, P(16), P(16), 1, None) == status
    assert lib.wm_kvq_read(r, 1, P(16), P(16), None) == status
    assert lib.wm_verify_attn_kvq(r, P(16), 1, 8, 1.0, P(16), None, P(256), 1 << 40, None) == status


def test_null_cache_is_refused(lib):
    assert lib.wm_kvq_append(None, P(16), P(16), 1, None) == INV
    assert lib.wm_kvq_read(None, 1, P(16), P(16), None) == INV
    assert lib.wm_verify_attn_kvq(None, P(16), 1, 8, 1.0, P(16), None, P(256), 1 << 40, None) == INV


@pytest.mark.parametrize("k,v,n", [(None, 16, 1), (16, None, 1), (8, 16, 1), (16, 8, 1), (16, 16, 0), (16, 16, -3)])
def test_bad_rows_are_refused(lib, k, v, n):
    r = ctypes.byref(kvq())
    assert lib.wm_kvq_append(r, P(k), P(v), n, None) == INV
    assert lib.wm_kvq_read(r, n, P(k), P(v), None) == INV


def test_bad_attention_arguments_are_refused(lib):
    r = ctypes.byref(kvq())
    need = wm.kvq_workspace_size(2, 4, 8, 3, 128)

    def call(q=16, n_q=3, hq=8, scale=1.0, out=16, lse=None, ws=256, size=need):
        return lib.wm_verify_attn_kvq(r, P(q), n_q, hq, scale, P(out), P(lse), P(ws), size, None)

    assert call(q=None) == INV and call(out=None) == INV and call(q=8) == INV and call(out=8) == INV
    assert call(n_q=0) == INV and call(hq=0) == INV and call(hq=6) == INV and call(lse=2) == INV
    assert call(scale=float("nan")) == INV and call(scale=float("inf")) == INV
    assert call(n_q=33) == UNS                      # 66 rows per KV head
    assert call(ws=None) == WSP and call(ws=128) == WSP and call(size=need - 1) == WSP
    big = kvq(paged=True, batch=65535, n_kv_heads=1, max_pages=1 << 24, n_pages=1 << 24)
    assert lib.wm_verify_attn_kvq(ctypes.byref(big), P(16), 1, 1, 1.0, P(16), None, P(256), 1 << 60, None) == UNS


def test_sizes(lib):
    assert [lib.wm_kvq_record_bytes(d) for d in (64, 128, 256, 0, 96, -1)] == [4608, 8704, 16896, 0, 0, 0]
    bad = ctypes.c_size_t(-1).value
    for args in ((0, 4, 8, 1, 128), (1, 0, 8, 1, 128), (1, 4, 6, 1, 128), (1, 4, 8, 0, 128), (1, 4, 8, 1, 96),
                 (1, 1, 65, 1, 128), (65536, 1, 1, 1, 64)):
        assert lib.wm_kvq_workspace_size(*args) == bad, args
    assert 0 < lib.wm_kvq_workspace_size(1, 4, 8, 1, 128) < lib.wm_kvq_workspace_size(64, 4, 8, 1, 128)


def test_bad_acceptance_arguments_are_refused(lib):
    names = ["p", "q", "x", "n", "u", "w", "lens", "batch", "k", "vocab", "tok", "acc", "new"]
    good = dict(p=16, q=16, x=16, n=16, u=16, w=16, lens=16, batch=2, k=3, vocab=100, tok=16, acc=16, new=16)

    def call(**over):
        a = {**good, **over}
        return lib.wm_spec_accept(*[a[n] if n in ("batch", "k", "vocab") else P(a[n]) for n in names], None)

    for n in ("p", "x", "u", "w", "tok", "acc"):
        assert call(**{n: None}) == INV, n
    for n in ("p", "q", "x", "n", "u", "w", "tok", "acc"):
        assert call(**{n: 18}) == INV, n
    assert call(lens=12) == INV and call(new=12) == INV and call(lens=None) == INV  # new_len without seq_lens
    assert call(batch=0) == INV and call(k=0) == INV and call(vocab=0) == INV
    assert call(batch=65536) == UNS and call(vocab=(1 << 30) + 1) == UNS


def test_binding_checks_types_and_shapes():
    with pytest.raises(ValueError):
        wm.kvq_record_bytes(96)
    with pytest.raises(ValueError, match="record|64"):
        wm.KVQCache(torch.zeros((1, 1, 1, 100), dtype=torch.uint8), torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="contiguous CUDA"):
        wm.KVQCache(torch.zeros((1, 1, 1, 4608), dtype=torch.uint8), torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="per sequence"):
        wm.KVQCache(torch.zeros((1, 1, 1, 4608), dtype=torch.uint8), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="block_table"):
        wm.KVQCache(torch.zeros((1, 1, 1, 4608), dtype=torch.uint8), torch.zeros(2, dtype=torch.int64),
                    torch.zeros((1, 1), dtype=torch.int32))
