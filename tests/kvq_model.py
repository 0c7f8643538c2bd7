"""64-bit models of the 4-bit KV cache and of the acceptance of drafted
tokens, written from their definitions (include/wm_api.h) for the tests: one
byte address per code, plain sums, no splits and no running maxima."""
from __future__ import annotations

import numpy as np
import torch

RK = 64  # positions per record


def rec_bytes(d: int) -> int:
    return 64 * d + 512


def bits(x: torch.Tensor) -> np.ndarray:
    return x.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def from_bits(u: np.ndarray) -> np.ndarray:
    """bf16 bit patterns to float64."""
    return (u.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16_bits(x: np.ndarray) -> np.ndarray:
    """float64 (non-negative, finite) to bf16 bit patterns, one rounding to nearest even: the candidates are the
    truncation and its successor."""
    lo = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint32)
    lo = np.where(from_bits(lo.astype(np.uint16)) > x, lo - 1, lo)
    a, b = from_bits(lo.astype(np.uint16)), from_bits((lo + 1).astype(np.uint16))
    up = (x - a > b - x) | ((x - a == b - x) & (lo & 1 == 1))
    return np.where(up, lo + 1, lo).astype(np.uint16)


def quantise(x: torch.Tensor):
    """(codes uint8, scale bits, zero bits) of rows x [..., D] bf16."""
    u = bits(x)
    y = from_bits(u)
    bad = ~np.isfinite(y).all(-1)
    y = np.where(bad[..., None], 0.0, y)
    z = y.min(-1)
    s_bits = to_bf16_bits((y.max(-1) - z) / 15.0)
    s = from_bits(s_bits)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = (y - z[..., None]).astype(np.float32).astype(np.float64)  # the difference is fp32's
        c = np.where(s[..., None] > 0, np.rint(t / s[..., None]), 0.0)
    c = np.clip(c, 0, 15).astype(np.uint8)
    z_bits = (z.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return c, np.where(bad, 0x7FFF, s_bits).astype(np.uint16), np.where(bad, 0x7FFF, z_bits).astype(np.uint16)


def _addr(d: int, is_v: bool, r: int) -> tuple[np.ndarray, np.ndarray]:
    """Byte offset in the record and bit shift of every channel's code at row r."""
    ch = np.arange(d)
    e = np.full(d, r % 32) if is_v else ch % 32
    unit = 32 * d + (r // 32) * 16 * d + ch * 16 if is_v else (ch // 32) * 1024 + r * 16
    bit = 4 * (e % 8 // 2 + 4 * (e % 2))
    return unit + e // 8 * 4 + bit // 8, bit % 8


def record(data: np.ndarray, table, b: int, h: int, blk: int) -> np.ndarray:
    per = data.shape[2]
    outer = b if table is None else int(table[b, blk // per])
    return data[outer, h, blk % per]


def store(data: np.ndarray, table, lens, k: torch.Tensor, v: torch.Tensor) -> None:
    """Append k, v [B, n, Hkv, D] at the last n positions of lens."""
    n, hkv, d = k.shape[1:]
    for is_v, x in ((False, k), (True, v)):
        c, s, z = quantise(x)
        for b in range(k.shape[0]):
            for i in range(n):
                pos = int(lens[b]) - n + i
                if pos < 0:
                    continue
                for h in range(hkv):
                    rec, r = record(data, table, b, h, pos // RK), pos % RK
                    at, sh = _addr(d, is_v, r)
                    # one nibble after the other: two channels of one position share a K byte
                    np.bitwise_and.at(rec, at, (~(15 << sh) & 255).astype(np.uint8))
                    np.bitwise_or.at(rec, at, (c[b, i, h].astype(np.int64) << sh).astype(np.uint8))
                    sz = rec[64 * d + 256 * is_v:][: 256].view(np.uint16).reshape(64, 2)
                    sz[r] = s[b, i, h], z[b, i, h]


def held(data: np.ndarray, table, b: int, h: int, n: int, is_v: bool):
    """(codes, scale, zero) of positions 0..n-1 in float64: [n, D], [n], [n]."""
    d = (data.shape[3] - 512) // 64
    codes, s, z = np.empty((n, d)), np.empty(n), np.empty(n)
    for pos in range(n):
        rec, r = record(data, table, b, h, pos // RK), pos % RK
        at, sh = _addr(d, is_v, r)
        codes[pos] = (rec[at] >> sh) & 15
        s[pos], z[pos] = from_bits(rec[64 * d + 256 * is_v:][: 256].view(np.uint16).reshape(64, 2)[r])
    return codes, s, z


def attend(data: np.ndarray, table, lens, q: torch.Tensor, scale: float):
    """(out, lse, size): size[...] = sum_j w_j (s_j c_jd + |z_j|), the magnitude that roundings of the weights act on."""
    b_n, t, hq, d = q.shape
    hkv = data.shape[1]
    g = hq // hkv
    out, size = np.zeros((b_n, t, hq, d)), np.zeros((b_n, t, hq, d))
    lse = np.full((b_n, t, hq), -np.inf)
    qf = from_bits(bits(q))
    for b in range(b_n):
        n = int(lens[b])
        for h in range(hkv):
            ck, sk, zk = held(data, table, b, h, n, False)
            cv, sv, zv = held(data, table, b, h, n, True)
            k = sk[:, None] * ck + zk[:, None]
            v, a = sv[:, None] * cv + zv[:, None], sv[:, None] * cv + np.abs(zv)[:, None]
            for i in range(t):
                m = n - t + i + 1  # visible keys
                if m <= 0:
                    continue
                for x in range(h * g, h * g + g):
                    s = (k[:m] @ qf[b, i, x]) * scale
                    top = s.max()
                    w = np.exp(s - top)
                    tot = w.sum()
                    out[b, i, x] = w @ v[:m] / tot
                    size[b, i, x] = w @ a[:m] / tot
                    lse[b, i, x] = top + np.log(tot)
    return out, lse, size


def accept(p, q, x, u, w, n=None):
    """(tokens, accepted) of target rows p [B, k + 1, V], draft rows q [B, k, V] or None, drafts x [B, k]."""
    p = np.clip(np.nan_to_num(p.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)
    if q is not None:
        q = np.clip(np.nan_to_num(q.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)
    clamp = lambda y: np.clip(np.nan_to_num(y.astype(np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)  # noqa: E731
    u, w = clamp(u), clamp(w)
    b_n, k = x.shape
    v = p.shape[2]
    tokens, acc = np.full((b_n, k + 1), -1, np.int32), np.zeros(b_n, np.int32)
    for b in range(b_n):
        nb = k if n is None else int(min(max(n[b], 0), k))
        a = 0
        while a < nb:
            t = int(x[b, a])
            if not 0 <= t < v:
                break
            if not u[b, a] * (1.0 if q is None else q[b, a, t]) < p[b, a, t]:
                break
            tokens[b, a] = t
            a += 1
        acc[b] = a
        r = p[b, a].copy()
        if a < nb:
            if q is not None:
                r = np.maximum(r - q[b, a], 0)
            elif 0 <= int(x[b, a]) < v:
                r[int(x[b, a])] = 0
            if not r.sum() > 0:
                r = p[b, a].copy()
        c = np.cumsum(r)
        if c[-1] > 0:
            past = np.nonzero((c > w[b] * c[-1]) & (r > 0))[0]
            tokens[b, a] = past[0] if len(past) else np.nonzero(r > 0)[0][-1]
    return tokens, acc
