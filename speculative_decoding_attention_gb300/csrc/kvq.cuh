// kvq.cuh -- the 4-bit KV cache: record layout, page lookup, and the schedule
// that splits a batch's key tiles over the grid.
//
// One record holds 64 positions of one KV head, K and V together, so the bytes
// an attention tile needs are contiguous and one bulk copy (no tensor map)
// brings them in:
//   K codes  [D / 32][64][16 bytes]   16 bytes = 32 channels of one position
//   V codes  [2][D][16 bytes]         16 bytes = 32 positions of one channel
//   K (scale, zero) [64] bf16 pairs,  V (scale, zero) [64] bf16 pairs
// 64 D + 512 bytes: 4 bits a value and 8 bytes per position and head.  Both code
// areas put the index that becomes the tensor-memory lane (position for K,
// channel for V) next to the 16-byte unit, so 32 lanes read 32 consecutive
// units: no bank conflict without any swizzle.  V is stored transposed because
// O^T = V^T P^T wants V's channels as lanes.
// In a 32-bit word, element e of 8 sits at bits 4 (e / 2 + 4 (e % 2)):
// (word >> 4 i) & 0x000f000f is then the pair (2 i, 2 i + 1) as two 16-bit
// integers, and a 16-bit integer c <= 15 read as fp16 is the subnormal c 2^-24
// exactly -- the tensor cores' operand, without a conversion.
#pragma once

#include <cstdint>

#include "wm_internal.h"
#include "../../include/wm_api.h"

namespace wm {

constexpr int kRecKeys = 64;
__host__ __device__ constexpr int rec_bytes(int d) { return 64 * d + 512; }
__host__ __device__ constexpr int rec_v_off(int d) { return 32 * d; }
__host__ __device__ constexpr int rec_ks_off(int d) { return 64 * d; }
__host__ __device__ constexpr int rec_vs_off(int d) { return 64 * d + 256; }

// Where the cache lives.  Contiguous: one "page" of n_cap positions per sequence.
struct KvqView {
    uint8_t *data;
    const int64_t *seq_lens;
    const int32_t *block_table;  // NULL: contiguous
    int64_t capacity;            // positions a sequence can hold
    int64_t n_pages;
    int32_t recs_per_page;       // page_size / 64, or n_cap / 64
    int32_t max_pages;
    int32_t batch;
    int32_t n_kv_heads;
    int32_t head_dim;
};

// Record `blk` (positions 64 blk .. 64 blk + 63) of sequence b, KV head h;
// NULL if the block table names a page outside the pool.
__device__ __forceinline__ uint8_t *kvq_record(const KvqView &c, int b, int h, int64_t blk) {
    int64_t page = b, within = blk;
    if (c.block_table) {
        const int64_t e = blk / c.recs_per_page;
        within = blk - e * c.recs_per_page;
        page = c.block_table[(int64_t)b * c.max_pages + e];
        if (page < 0 || page >= c.n_pages) return nullptr;
    }
    return c.data + ((page * c.n_kv_heads + h) * c.recs_per_page + within) * (int64_t)rec_bytes(c.head_dim);
}

__device__ __forceinline__ void kvq_report(int32_t *err, int32_t code) {
    if (err) atomicCAS(err, 0, code);
}

// Length of sequence b clamped to what the cache can hold.
__device__ __forceinline__ int64_t kvq_len(const KvqView &c, int b) {
    const int64_t len = c.seq_lens[b];
    return len < 0 ? 0 : len > c.capacity ? c.capacity : len;
}

// Parameters of the attention over the cache.
struct KvqAttnParams {
    KvqView c;
    const void *q;       // [B][n_q][Hq][D] bf16
    int32_t n_q, n_q_heads, group, rows;
    float scale_log2;    // scale * log2(e)
    int32_t *sched;      // [batch + 2]: tiles per CTA, then the tile prefix [batch + 1] (written by CTA 0)
    float *o_part;       // [n_cta + units - 1][rows][D]: each part normalised by its own sum
    float *lse_part;     // [n_cta + units - 1][rows], log2 units; -inf marks a part without a visible key
    void *out;
    float *lse;
    int32_t *err;
    uint32_t wait_limit; // polls before a pipeline wait is declared lost
    int32_t stall_tile;  // tests of the timeout path only, else -1
};

constexpr int kKvqTile = 256;  // positions per attention tile: two sub-tiles of two records
// Tiles whose products one accumulator takes up (attn_kvq.cuh has the drift of long chains).
// The error of an average over a million random positions, of which bf16's rounding of the
// output is 0.16%: 0.171% at 32 tiles, 0.189% at 48, 0.215% at 64 and 0.72% at 432 (head_dim
// 128); 64 are 2% faster than 32 where a CTA has 432.
constexpr int kKvqChain = 32;

__device__ __forceinline__ int kvq_tiles(const KvqView &c, int b) {
    return (int)((kvq_len(c, b) + kKvqTile - 1) / kKvqTile);
}

// The work of one CTA.  Unit u = b * n_kv_heads + h holds the tiles of sequence
// b's KV head h; the units' tiles laid end to end are cut into n_cta equal runs of
// `chunk` tiles, so every CTA streams the same number of bytes whatever the
// lengths.  The part of CTA c in unit u has index c + u: along the tiles each
// next part starts at a new CTA, a new unit or both, so the indexes rise and stay
// below n_cta + units - 1.  Every CTA works this out for itself from the
// lengths; a launch of its own would cost more.  CTA 0 also leaves the chunk and the
// prefix for the merge.  Tile counts fit 32 bits (at most 2^30 per call).
struct KvqRun {
    int b, h, t, n;  // sequence, KV head, first tile in the unit, tiles (0: no work)
    int len;         // positions of sequence b
};

// Run of `chunk` tiles at t0, found in sequences lo .. hi - 1 (acc tiles of one head before lo).
__device__ __forceinline__ KvqRun kvq_find(const KvqView &c, int lo, int hi, int acc, int t0, int n) {
    KvqRun r = {0, 0, 0, 0, 0};
    for (int b = lo; b < hi; ++b) {
        const int len = (int)kvq_len(c, b), nt = (len + kKvqTile - 1) / kKvqTile;
        if ((acc + nt) * c.n_kv_heads > t0) {
            const int within = t0 - acc * c.n_kv_heads;
            r.b = b;
            r.h = within / nt;
            r.t = within - r.h * nt;
            r.n = n;
            r.len = len;
            break;
        }
        acc += nt;
    }
    return r;
}

__device__ __forceinline__ int kvq_inclusive(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

constexpr int kKvqWarpBatch = 256;  // sequences up to which every warp finds the run by itself

// By one warp (batch <= kKvqWarpBatch), with no barrier; `leave`: this warp writes the schedule.
__device__ __forceinline__ KvqRun kvq_schedule_warp(const KvqAttnParams &p, bool leave) {
    const KvqView &c = p.c;
    const int lane = threadIdx.x & 31;
    const int per = (c.batch + 31) / 32;
    const int lo = min(c.batch, lane * per), hi = min(c.batch, lo + per);
    int mine = 0;
    for (int b = lo; b < hi; ++b) mine += kvq_tiles(c, b);
    const int incl = kvq_inclusive(mine, lane);
    const int all = __shfl_sync(0xffffffffu, incl, 31), total = all * c.n_kv_heads;
    const int chunk = total > 0 ? (total + (int)gridDim.x - 1) / (int)gridDim.x : 1;
    if (leave) {
        int acc = incl - mine;
        if (lane == 0) {
            p.sched[0] = chunk;
            p.sched[1 + c.batch] = all;
        }
        for (int b = lo; b < hi; ++b) {
            p.sched[1 + b] = acc;
            acc += kvq_tiles(c, b);
            if (c.seq_lens[b] != kvq_len(c, b)) kvq_report(p.err, WM_DEVERR_BAD_LENGTH);
        }
    }
    const int64_t t0 = (int64_t)blockIdx.x * chunk;
    KvqRun r = {0, 0, 0, 0, 0};
    if (t0 >= total) return r;
    const bool has = (incl - mine) * c.n_kv_heads <= t0 && t0 < incl * c.n_kv_heads;
    if (has) r = kvq_find(c, lo, hi, incl - mine, (int)t0, min(chunk, total - (int)t0));
    const int src = __ffs(__ballot_sync(0xffffffffu, has)) - 1;
    r.b = __shfl_sync(0xffffffffu, r.b, src);
    r.h = __shfl_sync(0xffffffffu, r.h, src);
    r.t = __shfl_sync(0xffffffffu, r.t, src);
    r.n = __shfl_sync(0xffffffffu, r.n, src);
    r.len = __shfl_sync(0xffffffffu, r.len, src);
    return r;
}

// By the whole block, for larger batches.
__device__ __forceinline__ KvqRun kvq_schedule_block(const KvqAttnParams &p, int *s_warp, KvqRun *s_run) {
    const KvqView &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_warps = blockDim.x >> 5;
    const int per = (c.batch + (int)blockDim.x - 1) / (int)blockDim.x;
    const int lo = min(c.batch, tid * per), hi = min(c.batch, lo + per);
    int mine = 0;
    for (int b = lo; b < hi; ++b) mine += kvq_tiles(c, b);
    const int incl = kvq_inclusive(mine, lane);
    if (lane == 31) s_warp[warp] = incl;
    if (tid == 0) *s_run = KvqRun{0, 0, 0, 0, 0};
    __syncthreads();
    const int w = kvq_inclusive(lane < n_warps ? s_warp[lane] : 0, lane);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0)), all = __shfl_sync(0xffffffffu, w, 31);
    int acc = (warp > 0 ? before : 0) + incl - mine;  // tiles of one head before sequence lo
    const int total = all * c.n_kv_heads;
    const int chunk = total > 0 ? (total + (int)gridDim.x - 1) / (int)gridDim.x : 1;
    const int64_t t0 = (int64_t)blockIdx.x * chunk;
    if (t0 < total && acc * c.n_kv_heads <= t0 && t0 < (acc + mine) * c.n_kv_heads)
        *s_run = kvq_find(c, lo, hi, acc, (int)t0, min(chunk, total - (int)t0));
    if (blockIdx.x == 0) {
        if (tid == 0) {
            p.sched[0] = chunk;
            p.sched[1 + c.batch] = all;
        }
        for (int b = lo; b < hi; ++b) {
            p.sched[1 + b] = acc;
            acc += kvq_tiles(c, b);
            if (c.seq_lens[b] != kvq_len(c, b)) kvq_report(p.err, WM_DEVERR_BAD_LENGTH);
        }
    }
    __syncthreads();
    return *s_run;
}

// Walks the parts of one CTA's run: tiles [t0, t0 + n) of unit (b, h), b of length len.
struct KvqPart {
    int b, h, t0, n, len;
};
struct KvqWalk {
    int b, h, t_off, left, len;
    __device__ __forceinline__ void init(const KvqRun &r) {
        b = r.b;
        h = r.h;
        t_off = r.t;
        left = r.n;
        len = r.len;
    }
    __device__ __forceinline__ bool next(const KvqView &c, KvqPart &q) {
        while (left > 0 && b < c.batch) {
            const int nt = (len + kKvqTile - 1) / kKvqTile;
            if (nt <= 0 || h == c.n_kv_heads) {  // no keys, or the sequence's last head is done
                if (++b < c.batch) len = (int)kvq_len(c, b);
                h = 0;
                t_off = 0;
                continue;
            }
            q.b = b;
            q.h = h;
            q.t0 = t_off;
            q.n = min(nt - t_off, left);
            q.len = len;
            left -= q.n;
            t_off = 0;
            ++h;
            return true;
        }
        return false;
    }
};

// The attention grid per head_dim (attn_kvq_d<D>.cu), and the merge of its parts.
cudaError_t launch_kvq_attn_d64(const KvqAttnParams &p, int n_cta, cudaStream_t stream);
cudaError_t launch_kvq_attn_d128(const KvqAttnParams &p, int n_cta, cudaStream_t stream);
cudaError_t launch_kvq_attn_d256(const KvqAttnParams &p, int n_cta, cudaStream_t stream);
cudaError_t launch_kvq_merge(const KvqAttnParams &p, int n_cta, cudaStream_t stream);

cudaError_t launch_kvq_append(const KvqView &c, const void *k_new, const void *v_new, int n_new, int32_t *err,
                              cudaStream_t stream);
cudaError_t launch_kvq_read(const KvqView &c, int n, void *k_out, void *v_out, int32_t *err, cudaStream_t stream);

struct AcceptParams {
    const float *target_probs;   // [batch][k + 1][vocab]
    const float *draft_probs;    // [batch][k][vocab] or NULL
    const int32_t *draft_tokens; // [batch][k]
    const int32_t *n_draft;      // [batch] or NULL
    const float *u_accept;       // [batch][k]
    const float *u_sample;       // [batch]
    const int64_t *seq_lens;     // [batch] or NULL
    int32_t *tokens;             // [batch][k + 1]
    int32_t *n_accepted;         // [batch]
    int64_t *new_len;            // [batch] or NULL
    int32_t batch, k, vocab;
    int32_t *err;
};
cudaError_t launch_spec_accept(const AcceptParams &p, int sms, cudaStream_t stream);

}  // namespace wm
