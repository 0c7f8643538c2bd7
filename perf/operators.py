"""Cases of the 4-bit KV cache (append, attention) and of the acceptance of
drafted tokens, with the operators' plain forms in elementary torch operations.

The 4-bit cache is an array of records, one per 64 positions of one KV head:
  K codes  [D/32][64][16] bytes   16 bytes = 32 channels of one position
  V codes  [2][D][16] bytes       16 bytes = 32 positions of one channel
  K scale and zero  [64][2] bf16, V scale and zero  [64][2] bf16
Eight codes share a 32-bit word: element e at bits 4 * (e / 2 + 4 * (e % 2)).
A code c of a position with scale s and zero z stands for s * c + z.
"""
import math

import torch

own = False

BLOCK = 64
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _attn(name, batch, ctx, hq, hkv, d, t, page=0, lo=0, peaked=0.0):
    """lo > 0: lengths spread over lo..ctx; peaked: share of keys scaled by 8."""
    return {"name": name, "op": "attn", "batch": batch, "ctx": ctx, "lo": lo, "hq": hq, "hkv": hkv, "d": d, "t": t,
            "page": page, "peaked": peaked}


def _append(name, batch, ctx, hkv, d, n, page=0, lo=0):
    return {"name": name, "op": "append", "batch": batch, "ctx": ctx, "lo": lo, "hkv": hkv, "d": d, "n": n,
            "page": page}


def _accept(name, batch, k, vocab, noise, probs=True, ragged=False):
    """noise: how far the draft's logits are from the target's; probs: the draft gives its probabilities."""
    return {"name": name, "op": "accept", "batch": batch, "k": k, "vocab": vocab, "noise": noise, "probs": probs,
            "ragged": ragged}


def listed():
    return [
        # one sequence, one token: the smallest call, where latency counts
        _attn("attn_decode_4k", 1, 4096, 8, 2, 128, 1),
        # 128K context, three drafted tokens
        _attn("attn_verify_128k", 1, 131072, 32, 4, 128, 4),
        # a hybrid model's full-attention layer at 1M context, peaked keys
        _attn("attn_verify_1m_d256", 1, 1048576, 16, 2, 256, 4, peaked=0.01),
        # two sequences of 1M, 40 query rows per KV head: the largest
        _attn("attn_verify_2x1m", 2, 1048576, 64, 8, 128, 5),
        # a ragged batch in 64-position pages
        _attn("attn_ragged_paged_b8", 8, 524288, 32, 8, 128, 3, page=64, lo=32768),
        # a serving batch of many short sequences, small heads, one token each
        _attn("attn_decode_b64_d64", 64, 8192, 16, 4, 64, 1, page=128, lo=1),
        # the step's new tokens of a serving batch
        _append("append_decode_b64", 64, 8192, 8, 128, 1, page=64, lo=1),
        # proposed tokens of a few sequences, which straddle a page's end
        _append("append_verify_b8_d256", 8, 32768, 2, 256, 6, page=64, lo=4096),
        # a prompt
        _append("append_prefill_32k", 1, 32768, 8, 128, 32768),
        # one sequence: latency
        _accept("accept_b1", 1, 3, 32000, 1.0),
        # a serving batch, drafts of different lengths, an odd vocabulary
        _accept("accept_b64", 64, 5, 131071, 0.7, ragged=True),
        # a large batch whose draft gives no probabilities (n-gram or retrieval drafts)
        _accept("accept_b256_greedy_draft", 256, 4, 131072, 0.5, probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "append", "accept"])
    d = rng.choice([64, 128, 256])
    page = rng.choice([0, 64, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "attn":
        t = rng.randint(1, 8)
        group = rng.randint(1, min(16, 64 // t))
        batch = _log(rng, 1, 64)
        ctx = _log(rng, 128, max(256, min(1048576, (1 << 31) // (batch * hkv * d))))
        c = _attn("", batch, ctx, hkv * group, hkv, d, t, page, rng.choice([0, 1, max(1, ctx // 8)]),
                  rng.choice([0.0, 0.01]))
    elif op == "append":
        batch = _log(rng, 1, 64)
        n = _log(rng, 1, 32768 // batch)
        ctx = n + _log(rng, 1, 32768)
        c = _append("", batch, ctx, hkv, d, n, page, rng.choice([0, n]))
    else:
        c = _accept("", _log(rng, 1, 256), rng.randint(1, 8), _log(rng, 1000, 131072), rng.uniform(0.2, 1.5),
                    rng.random() < 0.7, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lengths(case, g):
    """Positions of each sequence, the new ones included."""
    if case["lo"]:
        lens = torch.randint(case["lo"], case["ctx"] + 1, (case["batch"],), generator=g, device=DEV)
        lens[0] = case["ctx"]
    else:
        lens = torch.full((case["batch"],), case["ctx"], device=DEV)
    return lens.to(torch.int64)


def _table(case, lens, g):
    """Pages of the pool and the block table: a permuted pool with a few pages more than the lengths need."""
    page = case["page"]
    per = (lens + page - 1) // page
    most = -(-case["ctx"] // page)
    pool = case["batch"] * most + 3
    perm = torch.randperm(pool, generator=g, device=DEV)[: case["batch"] * most].view(case["batch"], most)
    used = torch.arange(most, device=DEV)[None, :] < per[:, None]
    return pool, torch.where(used, perm, torch.zeros_like(perm)).to(torch.int32)


def _quantise(x):
    """Codes (64-bit floats), scale and zero (bf16) of x [..., D] bf16, in 64 bits."""
    y = x.double()
    z, top = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    # one rounding from 64 bits to bf16: through 32 bits, rounded to odd, so that it is not rounded twice
    s64 = (top - z) / 15
    s32 = s64.float()
    down = torch.where(s32.double() > s64, torch.nextafter(s32, torch.zeros_like(s32)), s32)
    odd = (down.view(torch.int32) | (down.double() != s64).int()).view(torch.float32)
    s = odd.to(torch.bfloat16)
    safe = torch.where(s > 0, s, torch.ones_like(s)).double()
    c = ((y - z) / safe).round().clamp(0, 15) * (s > 0)
    return c, s, z.to(torch.bfloat16)


def _pack(codes):
    """Codes [..., 8 m] -> bytes [..., 4 m]: element e of 8 at bits 4 * (e / 2 + 4 * (e % 2)) of its word."""
    n = codes.to(torch.uint8).unflatten(-1, (-1, 4, 2)).transpose(-1, -2).flatten(-2).unflatten(-1, (4, 2))
    return (n[..., 0] | (n[..., 1] << 4)).flatten(-2)


def _records(k, v):
    """Records [blocks, 64 D + 512] bytes of k, v [blocks, 64, D] bf16."""
    d = k.shape[-1]
    out = torch.empty((k.shape[0], 64 * d + 512), dtype=torch.uint8, device=k.device)
    ck, sk, zk = _quantise(k)
    out[:, : 32 * d] = _pack(ck).unflatten(-1, (d // 32, 16)).transpose(1, 2).flatten(1)
    out[:, 64 * d: 64 * d + 256] = torch.cat([sk, zk], -1).view(torch.uint8).flatten(1)
    del ck
    cv, sv, zv = _quantise(v)
    out[:, 32 * d: 64 * d] = _pack(cv.transpose(1, 2)).unflatten(-1, (2, 16)).transpose(1, 2).flatten(1)
    out[:, 64 * d + 256:] = torch.cat([sv, zv], -1).view(torch.uint8).flatten(1)
    return out


def _cache(case, g):
    lens = _lengths(case, g)
    page, hkv, d = case["page"], case["hkv"], case["d"]
    if page:
        outer, table = _table(case, lens, g)
        blocks = page // BLOCK
    else:
        outer, table, blocks = case["batch"], None, -(-case["ctx"] // BLOCK)
    data = torch.empty((outer, hkv, blocks, 64 * d + 512), dtype=torch.uint8, device=DEV)
    flat = data.view(-1, 64 * d + 512)
    step = max(1, (1 << 27) // (BLOCK * d))
    for at in range(0, flat.shape[0], step):
        n = min(step, flat.shape[0] - at)
        k = torch.randn((n, BLOCK, d), generator=g, device=DEV)
        if case.get("peaked"):
            k = k * torch.where(torch.rand((n, BLOCK, 1), generator=g, device=DEV) < case["peaked"], 8.0, 1.0)
        v = torch.randn((n, BLOCK, d), generator=g, device=DEV)
        flat[at: at + n] = _records(k.bfloat16(), v.bfloat16())
    return {"data": data, "seq_lens": lens, "block_table": table}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "attn":
        st.update(_cache(case, g))
        st["scale"] = case["d"] ** -0.5
        st["q"] = torch.randn((case["batch"], case["t"], case["hq"], case["d"]), generator=g, device=DEV).bfloat16()
    elif case["op"] == "append":
        st.update(_cache(case, g))
        shape = (case["batch"], case["n"], case["hkv"], case["d"])
        # channels of different size, as keys have them
        gain = torch.exp(0.5 * torch.randn((case["hkv"], case["d"]), generator=g, device=DEV))
        st["k_new"] = (torch.randn(shape, generator=g, device=DEV) * gain).bfloat16()
        st["v_new"] = torch.randn(shape, generator=g, device=DEV).bfloat16()
    else:
        b, k, n = case["batch"], case["k"], case["vocab"]
        logits = torch.randn((b, k + 1, n), generator=g, device=DEV).mul_(2.5)
        st["target_probs"] = torch.softmax(logits, -1)
        logits[:, :k] += case["noise"] * torch.randn((b, k, n), generator=g, device=DEV)
        q = torch.softmax(logits[:, :k], -1)
        # the draft's tokens are drawn from its probabilities
        u = torch.rand((b, k, 1), generator=g, device=DEV)
        st["draft_tokens"] = (torch.cumsum(q, -1) < u).sum(-1).clamp(max=n - 1).to(torch.int32)
        st["draft_probs"] = q if case["probs"] else None
        st["u_accept"] = torch.rand((b, k), generator=g, device=DEV)
        st["u_sample"] = torch.rand((b,), generator=g, device=DEV)
        st["n_draft"] = (torch.randint(0, k + 1, (b,), generator=g, device=DEV).to(torch.int32)
                         if case["ragged"] else None)
        st["seq_lens"] = torch.randint(k + 1, 100000, (b,), generator=g, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _unpack(b):
    """Bytes [..., 4 m] -> codes [..., 8 m] in 32-bit floats."""
    n = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (-1, 2, 4))
    return n.transpose(-1, -2).flatten(-3).float()


def _values(rec, d):
    """K and V [..., 64, D] in 32 bits of records [..., 64 D + 512]."""
    k = _unpack(rec[..., : 32 * d].unflatten(-1, (d // 32, 64, 16)).transpose(-3, -2).flatten(-2))
    v = _unpack(rec[..., 32 * d: 64 * d].unflatten(-1, (2, d, 16)).transpose(-3, -2).flatten(-2)).transpose(-1, -2)
    sz = rec[..., 64 * d:].contiguous().view(torch.bfloat16).unflatten(-1, (2, 64, 2)).float()
    k = k * sz[..., 0, :, 0:1] + sz[..., 0, :, 1:2]
    v = v * sz[..., 1, :, 0:1] + sz[..., 1, :, 1:2]
    return k, v


def _plain_attn(st):
    c, lens = st["case"], st["seq_lens"]
    b, t, hq, hkv, d = c["batch"], c["t"], c["hq"], c["hkv"], c["d"]
    rec = st["data"]
    if st["block_table"] is not None:
        rec = rec[st["block_table"].long()].transpose(1, 2).flatten(2, 3)  # [B, Hkv, blocks, record]
    k, v = _values(rec, d)
    k, v = k.flatten(2, 3), v.flatten(2, 3)  # [B, Hkv, N, D]
    q = st["q"].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, T G, D]
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    last = lens[:, None] - t + torch.arange(t, device=DEV)  # [B, T]
    seen = torch.arange(k.shape[2], device=DEV) <= last[:, :, None]
    seen = seen.repeat_interleave(hq // hkv, 1)[:, None]
    s = torch.where(seen, s, -torch.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top)[..., 0]
    back = lambda x: x.unflatten(2, (t, hq // hkv)).transpose(1, 2).flatten(2, 3)  # noqa: E731
    return back(out).bfloat16(), back(lse)


def _plain_append(st):
    """The values that the cache holds for the new positions."""
    out = []
    for x in (st["k_new"], st["v_new"]):
        code, s, z = _quantise(x)
        out.append((code.float() * s.float() + z.float()).bfloat16())
    return tuple(out)


def _plain_accept(st):
    p, q, x = st["target_probs"], st["draft_probs"], st["draft_tokens"].long()
    b, k = x.shape
    n = st["n_draft"].long() if st["n_draft"] is not None else torch.full((b,), k, device=DEV)
    p_at = p[:, :k].gather(2, x[..., None])[..., 0].double()
    q_at = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(p_at)
    ok = (st["u_accept"].double() * q_at < p_at) & (torch.arange(k, device=DEV) < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    row = torch.arange(b, device=DEV)
    target = p[row, a].double()
    at = a.clamp(max=k - 1)
    if q is not None:
        rest = (target - q[row, at].double()).clamp(min=0)
    else:
        rest = target.scatter(1, x[row, at][:, None], 0.0)
    rest = torch.where((a < n)[:, None], rest, target)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, target)
    total = rest.cumsum(1)
    token = (total <= st["u_sample"].double()[:, None] * total[:, -1:]).sum(1).clamp(max=p.shape[2] - 1)
    place = torch.arange(k + 1, device=DEV)
    tokens = torch.where(place < a[:, None], torch.cat([x, x[:, :1]], 1), -1)
    tokens = torch.where(place == a[:, None], token[:, None], tokens)
    return tokens.to(torch.int32), a.to(torch.int32), st["seq_lens"] - k + a


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        return {"attn": _plain_attn, "append": _plain_append, "accept": _plain_accept}[op](st)
    from speculative_decoding_attention_gb300 import wm

    if op == "accept":
        return wm.spec_accept(st["target_probs"], st["draft_probs"], st["draft_tokens"], st["u_accept"],
                              st["u_sample"], n_draft=st["n_draft"], seq_lens=st["seq_lens"])
    if "cache" not in st:  # the handle and the workspace that a decode loop keeps
        st["cache"] = wm.KVQCache(st["data"], st["seq_lens"], st["block_table"])
        if op == "attn":
            st["workspace"] = wm.kvq_workspace(st["cache"], st["case"]["hq"], st["case"]["t"])
    if op == "append":
        wm.kvq_append(st["cache"], st["k_new"], st["v_new"])
        return wm.kvq_read(st["cache"], st["case"]["n"])
    return wm.verify_attn_kvq(st["cache"], st["q"], st["scale"], workspace=st["workspace"])


# ------------------------------------------------------------------ from the definition, in 64 bits

def _held(st, b, h, lo, hi, base, zero_at, along_d):
    """Values of positions lo..hi-1 of one head in 64 bits, by the address of each code."""
    d, data = st["case"]["d"], st["data"]
    pos = torch.arange(lo, hi, device=DEV)
    blk, r = pos // 64, pos % 64
    per = data.shape[2]
    outer = st["block_table"][b].long()[blk // per] if st["block_table"] is not None else torch.full_like(blk, b)
    flat = data.view(-1)
    rec = ((outer * data.shape[1] + h) * per + blk % per) * data.shape[3]
    ch = torch.arange(d, device=DEV)
    if along_d:
        e, byte = ch[None, :] % 32, (ch // 32 * 1024)[None, :] + r[:, None] * 16
    else:
        e, byte = (r % 32)[:, None], (r // 32 * 16 * d)[:, None] + ch[None, :] * 16
    bit = 4 * (e % 8 // 2 + 4 * (e % 2))
    addr = rec[:, None] + base + byte + e // 8 * 4 + bit // 8
    code = (flat[addr].int() >> (bit % 8).int()) & 15
    both = flat[(rec + zero_at + 4 * r)[:, None] + torch.arange(4, device=DEV)].view(torch.bfloat16).double()
    return code.double() * both[:, :1] + both[:, 1:]


def exact(case, seed):
    if case["op"] == "accept":
        return None  # whole numbers
    st = prepare(case, seed)
    if case["op"] == "append":
        return tuple(_exact_store(x) for x in (st["k_new"], st["v_new"]))
    b_n, t, hq, hkv, d = case["batch"], case["t"], case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros((b_n, t, hq, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b_n, t, hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(st["seq_lens"].tolist()):
        for h in range(hkv):
            q = st["q"][b, :, h * g: (h + 1) * g].double().reshape(t * g, d)
            limit = (n - t + torch.arange(t, device=DEV)).repeat_interleave(g)[:, None]
            top = torch.full((t * g, 1), -math.inf, dtype=torch.float64, device=DEV)
            total, acc = torch.zeros_like(top), torch.zeros((t * g, d), dtype=torch.float64, device=DEV)
            for lo in range(0, n, 1 << 17):
                hi = min(n, lo + (1 << 17))
                k = _held(st, b, h, lo, hi, 0, 64 * d, True)
                s = (q @ k.T) * st["scale"]
                s = s.masked_fill(torch.arange(lo, hi, device=DEV)[None, :] > limit, -math.inf)
                new = torch.maximum(top, s.amax(1, keepdim=True))
                base = torch.where(new == -math.inf, torch.zeros_like(new), new)
                w = torch.exp(s - base)
                keep = torch.exp(top - base)
                total = total * keep + w.sum(1, keepdim=True)
                acc = acc * keep + w @ _held(st, b, h, lo, hi, 32 * d, 64 * d + 256, False)
                top = new
            some = total[:, 0] > 0
            o = torch.where(some[:, None], acc / total, torch.zeros_like(acc))
            out[b, :, h * g: (h + 1) * g] = o.view(t, g, d)
            lse[b, :, h * g: (h + 1) * g] = (top + torch.log(total))[:, 0].view(t, g)
    return out, lse


def _exact_store(x):
    """Each row's least value, its step (an 8-bit significand nearest to a fifteenth of the range) and its codes."""
    y = x.double()
    low = y.amin(-1, keepdim=True)
    frac, exp = torch.frexp((y.amax(-1, keepdim=True) - low) / 15)
    step = torch.ldexp(torch.round(frac * 256) / 256, exp)
    code = torch.where(step > 0, torch.round((y - low) / torch.where(step > 0, step, torch.ones_like(step))),
                       torch.zeros_like(y))
    return low + step * code.clamp(0, 15)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "attn":
        # mean length of the spread
        tokens = case["batch"] * ((case["lo"] + case["ctx"]) / 2 if case["lo"] else case["ctx"])
        rows = case["batch"] * case["t"] * case["hq"]
        return {"bytes": tokens * case["hkv"] * (case["d"] + 8) + rows * (4 * case["d"] + 4),
                "flops": 4.0 * tokens * case["hq"] * case["t"] * case["d"]}
    if case["op"] == "append":
        n = case["batch"] * case["n"] * case["hkv"]
        # new rows in, records out; the records read back, values out
        return {"bytes": n * 2 * (4 * case["d"] + case["d"] + 8), "flops": n * 2.0 * case["d"] * 6}
    # one row of the target for each sequence, and the draft's where a token is refused (about half of them)
    rows = case["batch"] * (1.5 if case["probs"] else 1.0)
    return {"bytes": rows * case["vocab"] * 4.0, "flops": rows * case["vocab"] * 2.0}
