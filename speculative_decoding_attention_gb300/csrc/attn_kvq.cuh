// attn_kvq.cuh -- causal attention over the 4-bit KV cache on the 5th-generation
// tensor cores.
//
// With l_j = s_j (q . c_j) + z_j sum(q) the products run over the codes alone:
//   S^T[128 keys x NR] = C_K[128 x D] . Q^T        (A: codes in tensor memory, B: Q^T in shared memory)
//   O^T[D x NR]       += C_V^T[D x 128] . P'^T     (A: codes in tensor memory, B: P'^T in shared memory)
// in tiles of 256 keys, two sub-tiles of 128.
// A code c <= 15 in the low bits of 16 is the fp16 subnormal c 2^-24, exactly,
// and four bits higher c 2^-20: a word's eight codes are four masks and one
// shift.  The factor 16 of every other pair is taken out of the other operand
// (Q's channels and P's keys with bit 1 set), where it is exact.  The codes go to
// tensor memory rather than shared memory: as 16-bit operands in shared memory
// they would cost 2 bytes written and 2 read per code where HBM delivers half a
// byte, more than shared memory's 128 bytes per clock when HBM runs at full rate.
// Keys (for S) and channels (for O) are the MMA's M, so the few query rows are N.
//
// K's scale and zero enter the logit (log2 units, key j, row r):
//   t_jr = S_jr a_j + zq_r b_j + ls_j,  a = s_K 2^24 f,  b = z_K f,  f = scale log2(e)
//   zq_r = sum_d q_rd,  ls_j = log2(s_V).
// V's scale is folded into the weight: P'_jr = 2^(t_jr - m_r) = s_Vj p_jr, so that
//   o_r = [ 2^24 sum_j P'_jr (c_j - 8) + sum_j P'_jr (z_V / s_V + 8)_j ] / sum_j P'_jr (1 / s_V)_j
// with the running maximum m taken over t: the largest P' is near the top of fp16's
// range whatever the scales are.  P' is rounded to fp16 for the first sum only (at
// most 2^-11 of it; the others are fp32 sums of P' as it is).  That error is weighted
// by s_V (c - 8), about the value itself: with c in its place it would be weighted by the
// value's distance from the zero, which shows wherever values cancel.  The - 8 is
// a product with a constant operand, free on the tensor cores.  A row of constant
// values has s_V = 0 and codes 0; a stand-in scale |z| / 256 carries its zero.
//
// The tensor cores add to O by cutting off, not rounding, so a long chain of additions
// drifts: averages over a million random values were off by 0.7% after 432 tiles, where bf16
// rounds by 0.17%.  Every
// kKvqChain tiles the softmax warps therefore add O to fp32 sums of their own (rounded, in
// the part's slot of the workspace, which each thread alone touches) and the products start
// O anew.
//
// Each CTA takes one run of the batch's tiles (kvq_schedule), cut into parts at
// (sequence, KV head) borders; every role counts tiles across parts, so no
// buffer drains at a border.  Roles:
//   warp 0      bulk copies: the two 64-position records of a tile, K and V and scales, one stage
//   warp 1      one lane issues S, warp 2 P.V: each waits for its own operands only
//   ND warps    codes -> tensor memory, a thread per key (K) or channel (V); the K
//               warps also turn each key's scales and zeros into the softmax's constants
//   NSW warps   softmax: a thread per lane (two keys of the tile), HR rows each; the four
//               warps that share rows vote per tile whether the maxima have to be raised
// What bounds it: HBM, as long as the instructions per tile fit beside it.  8 ragged paged
// sequences, 12 rows of 128, 2.7 GB: 488 us, 5.5 TB/s; 1M positions, 32 rows of 256:
// 137 us, 4.0; 2 x 1M positions, 40 rows of 128: 674 us, 3.4 -- there 54% of the issue slots
// and 46% of the ALU are taken, the tensor pipe 35% (with the products of -8), and
// registers bar more softmax warps.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace wm {

constexpr float kKvqOff = 7.f;       // the running maximum sits at 2^7 in P': fp16 keeps 11 bits down to 2^-21 of it
constexpr float kKvqRaise = 8.f;     // raise the maximum only past 2^8 (P' <= 2^15, fp16 holds up to 65504)

// NR: the MMA's N, a multiple of 16; LIVE: rows that have softmax warps (nothing reads the
// columns of P', S and O past them).
template <int D_, int NR_, int LIVE_>
struct KvqCfg {
    static constexpr int D = D_, NR = NR_, LIVE = LIVE_;
    static constexpr int REC = rec_bytes(D);
    static constexpr int STAGE = 2 * REC;               // a sub-tile of 128 keys
    static constexpr int NC = D == 256 ? 2 : 1;         // 128-channel chunks
    static constexpr int KU = D == 64 ? 2 : 4;          // 16-byte units per key and chunk
    // Rows per softmax warp and converting warps.  More warps hide more latency, fewer leave
    // more registers to each and repeat less per-key work; measured in us, chosen form first:
    // up to 16 rows at head_dim 128 (ragged batch of 2.9 GB) 16 converting warps 515, 8 563, 4
    // 644; at 64 (64 short sequences) 8 warps 54, 4 55, 16 61; 24 rows at 128 (512K positions)
    // 8 warps 77, 4 82; at 256 (1M) 8 115, 4 124; 32 rows at 128 (512K) 8 86, 4 90, and
    // with 4 and 16 rows per softmax warp 88; at 256 (1M) 4 137 and 8 144 with peaked keys,
    // 134 and 125 without; 48 rows (2 x 1M) 16 rows per softmax warp and 4 converting 674,
    // 8 converting 907.
    static constexpr int HR = NR <= 32 ? 8 : 16;
    static constexpr int ND = NR == 16 ? (D == 128 ? 16 : 8) : NR == 32 && (D < 256 || LIVE == 24) ? 8 : 4;
    static constexpr int KG = ND == 16 ? 2 : 1, VG = KG;  // warp groups for K and V
    // Two groups take turns, each with slots of its own (a wait on a slot's barrier has to
    // follow every use of it).
    static_assert(KG == 1 || NC == 1, "a group owns its slots");
    static_assert(HR == 8 || HR == 16, "rows per softmax warp");
    static constexpr int NSW = 4 * (LIVE / HR);         // softmax warps
    static constexpr int W_D = 3, W_S = 3 + ND;         // first converting and first softmax warp
    static constexpr int THREADS = 32 * (W_S + NSW);
    // tensor memory: K and V code slots of 64 columns, the constant -8 (8 columns), S of two sub-tiles, O
    static constexpr int SLOTS = (512 - 8 - 2 * NR - NC * NR) / 64;
    static constexpr int KS = 2, VS = SLOTS >= 6 ? 4 : SLOTS >= 4 ? 2 : 1;
    static constexpr int V_COL = 64 * KS, S_COL = 64 * (KS + VS), O_COL = S_COL + 2 * NR, E_COL = O_COL + NC * NR;
    static_assert(VS >= 1 && E_COL + 8 <= 512, "tensor memory");
    // shared memory
    static constexpr int PT_ROW = NR <= 16 ? 32 : NR <= 32 ? 64 : 128;
    static constexpr uint32_t PT_SWIZZLE = NR <= 16 ? tc::SWIZZLE_32B : NR <= 32 ? tc::SWIZZLE_64B : tc::SWIZZLE_128B;
    static constexpr int PT_ATOM = 8 * PT_ROW, PT_BYTES = 128 * PT_ROW;  // one part of one sub-tile
    static constexpr int PB_BYTES = 2 * PT_BYTES;       // one P' buffer: two sub-tiles
    static constexpr int Q_REGION = NR * 128;           // 64 channels of every row
    static constexpr int Q_OFF = 0;
    static constexpr int PT_OFF = Q_OFF + (D / 64) * Q_REGION;
    // behind the stages: per-key constants, per-row scratch, barriers
    static constexpr int CONST_BYTES = 4 * 128 * 20;
    static constexpr int RED_BYTES = 8 * NR * 4, ROW_BYTES = 2 * NR * 4;
    static constexpr int TAIL = CONST_BYTES + RED_BYTES + 3 * ROW_BYTES + 256 + 512 + 32 * 8 + 64;
    static constexpr int ROOM = 227 * 1024 - 1024 - PT_OFF - TAIL;
    // A second P' buffer if four stages still fit (the softmax of a tile then need not
    // wait for the products of the last), then up to eight stages.
    static constexpr int NPB = (ROOM - 2 * PB_BYTES) / STAGE >= 4 ? 2 : 1;
    static constexpr int ST_OFF = PT_OFF + NPB * PB_BYTES;
    static constexpr int FIT = (ROOM - NPB * PB_BYTES) / STAGE;
    static constexpr int NST = FIT > 8 ? 8 : FIT;
    static_assert(NST >= 2, "stages");
    static constexpr int CONST_OFF = ST_OFF + NST * STAGE;        // float4 [4][128], float [4][128]
    static constexpr int RED_OFF = CONST_OFF + CONST_BYTES;       // float [2][NR][4]: per row and lane quadrant
    static constexpr int ZQ_OFF = RED_OFF + RED_BYTES;            // float [2][NR]: sums of a part's queries
    static constexpr int NM_OFF = ZQ_OFF + ROW_BYTES;             // float [2][NR]: minus (running maximum - kKvqOff)
    static constexpr int NP_OFF = NM_OFF + ROW_BYTES;             // float [2][NR]: the same when O was last taken over
    static constexpr int FLAG_OFF = NP_OFF + ROW_BYTES;           // int [64]: [0] abort, [8 + w] scratch
    static constexpr int BAR_OFF = FLAG_OFF + 256;
    static constexpr int NBAR = 2 * NST + 8 + 8 + 1 + 1 + 2 + 2 + 1 + 2;
    static_assert(NBAR * 8 <= 512, "barriers");
    static constexpr int WARP_OFF = BAR_OFF + 512;                // int [32] + KvqRun of the schedule
    static constexpr int TPTR_OFF = WARP_OFF + 32 * 8 + 16;
    static constexpr int TOTAL = ST_OFF + NST * STAGE + TAIL + 1024;
    static_assert(TPTR_OFF + 16 <= TOTAL - 1024 && TOTAL <= 227 * 1024, "shared memory");
    static_assert(PT_OFF % 1024 == 0 && ST_OFF % 128 == 0 && CONST_OFF % 16 == 0, "alignment");
};

// The 32 codes of one 16-byte unit as 16 fp16 pairs, in order, to 16 columns of
// this lane: c 2^-24 for elements 0, 1, 4, 5 of each 8 and c 2^-20 for 2, 3, 6, 7.
__device__ __forceinline__ void kvq_unit_to_tmem(uint32_t taddr, uint4 u) {
    constexpr uint32_t M0 = 0x000f000fu, M1 = 0x00f000f0u;
    const uint4 h = make_uint4(u.x >> 8, u.y >> 8, u.z >> 8, u.w >> 8);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(u.x & M0), "r"(u.x & M1), "r"(h.x & M0), "r"(h.x & M1), "r"(u.y & M0), "r"(u.y & M1), "r"(h.y & M0),
        "r"(h.y & M1), "r"(u.z & M0), "r"(u.z & M1), "r"(h.z & M0), "r"(h.z & M1), "r"(u.w & M0), "r"(u.w & M1),
        "r"(h.w & M0), "r"(h.w & M1)
        : "memory");
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Largest of one value per lane, NaN left out.
__device__ __forceinline__ float warp_max_f(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) { return __uint_as_float(ld_shared_u32(addr)); }
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    const uint4 v = ld_shared_v4(addr);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
// Two pairs of fp32.
__device__ __forceinline__ ulonglong2 ld_shared_pairs(uint32_t addr) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) { st_shared_u32(addr, __float_as_uint(v)); }

// D[tmem] (+)= A[tmem] * B[smem desc], fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: fp16 A (tensor memory, K-major) and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int n, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// One lane of a converged warp.  The compiler then knows the branch has one
// thread: MMAs issued behind a test of the lane number instead took 46 clocks
// each, behind this one 9 (N = 16, measured), their own rate of N / 2.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// Rest of a wait whose first poll failed.  Gives up after `limit` polls, or once another
// role has given up: records the timeout, raises the abort flag and returns false.
__device__ __forceinline__ bool kvq_wait_slow(uint32_t bar, uint32_t parity, uint32_t limit, volatile int *flags,
                                           int32_t *err) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (flags[0]) return false;
        if (i > 64) __nanosleep(64);
    }
    kvq_report(err, WM_DEVERR_TIMEOUT);
    flags[0] = 1;
    return false;
}

template <int D, int NR, int LIVE>
__global__ void __launch_bounds__(KvqCfg<D, NR, LIVE>::THREADS, 1) kvq_attn_kernel(const KvqAttnParams p) {
    using C = KvqCfg<D, NR, LIVE>;
    constexpr int TK = kKvqTile, NC = C::NC, HR = C::HR, NSW = C::NSW, ND = C::ND, NST = C::NST, NPB = C::NPB;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *gb = smem_raw + (sbase - raw);
    const uint32_t sQ = sbase + C::Q_OFF, sPT = sbase + C::PT_OFF, sST = sbase + C::ST_OFF;
    const uint32_t s_red = sbase + C::RED_OFF;              // float [2][NR][4]
    const uint32_t s_zq = sbase + C::ZQ_OFF;                // float [2][NR]
    const uint32_t s_nm = sbase + C::NM_OFF;                // float [2][NR]
    const uint32_t s_np = sbase + C::NP_OFF;                // float [2][NR]
    const uint32_t s_const = sbase + C::CONST_OFF;          // float4 [4][128]
    const uint32_t s_zr = s_const + 4 * 128 * 16;           // float [4][128]
    volatile int *flags = reinterpret_cast<volatile int *>(gb + C::FLAG_OFF);
    const uint32_t bars = sbase + C::BAR_OFF;
    const uint32_t bar_full = bars;                      // [NST] stage landed
    const uint32_t bar_empty = bar_full + 8 * NST;       // [NST] stage read by everyone
    const uint32_t bar_aready = bar_empty + 8 * NST;     // [KS + VS] code slot written
    const uint32_t bar_afree = bar_aready + 64;          // [KS + VS] code slot consumed
    const uint32_t bar_sfull = bar_afree + 64;           // S of tile t
    const uint32_t bar_sfree = bar_sfull + 8;
    const uint32_t bar_pfull = bar_sfree + 8;            // [2] P' of tile t, buffer t % NPB
    const uint32_t bar_odone = bar_pfull + 16;           // [2] its P.V
    const uint32_t bar_qfull = bar_odone + 16;           // phase k: queries of part k written
    const uint32_t bar_final = bar_qfull + 8;            // [2] the issuers' last commits
    uint32_t *tptr = reinterpret_cast<uint32_t *>(gb + C::TPTR_OFF);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // Set-up that touches only shared and tensor memory, while the previous kernel drains.
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 8);  // K and V conversion, four warps each
        }
        for (int i = 0; i < C::KS + C::VS; ++i) {
            mbar_init(bar_aready + 8 * i, 4);
            mbar_init(bar_afree + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_pfull + 8 * i, NSW);
            mbar_init(bar_odone + 8 * i, 1);
        }
        mbar_init(bar_sfull, 2);  // the issuer, and its products' completion
        mbar_init(bar_sfree, NSW);
        mbar_init(bar_qfull, NSW);
        mbar_init(bar_final, 1);
        mbar_init(bar_final + 8, 1);
        for (int i = 0; i < 64; ++i) flags[i] = 0;
        fence_mbar_init();
    }
    static_assert(C::KS + C::VS <= 8, "slot barriers");
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(tptr), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tptr;

    // The constant operand -8: for the 16 keys of one MMA, pairs of -8 2^-24 and -8 2^-20.
    if (warp >= C::W_D && warp < C::W_D + 4) {
        const uint32_t v0 = 0x80088008u, v1 = 0x80808080u;
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %1, %2, %1, %2, %1, %2};" ::"r"(
                         tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::E_COL),
                     "r"(v0), "r"(v1)
                     : "memory");
        tc::wait_st();
        tc::fence_before_sync();  // seen by the issuer through the first code slot's barrier
    }

    pdl_wait();
    pdl_launch_dependents();
    const KvqRun run = p.c.batch <= kKvqWarpBatch
                           ? kvq_schedule_warp(p, blockIdx.x == 0 && warp == 3)
                           : kvq_schedule_block(p, reinterpret_cast<int *>(gb + C::WARP_OFF),
                                                reinterpret_cast<KvqRun *>(gb + C::WARP_OFF + 32 * 4));
    const int n_all = run.n;
    if (n_all <= 0) {
        if (warp == 1) tc::tmem_dealloc(tmem, 512);
        return;
    }
    KvqWalk walk;
    walk.init(run);

    // Bounded wait for a barrier's phase; false once the pipeline is given up.
    const auto wait = [&](uint32_t bar, int phase) -> bool {
        return mbar_try_wait(bar, phase & 1) || kvq_wait_slow(bar, phase & 1, p.wait_limit, flags, p.err);
    };

    if (warp == 0) {
        // ============================================================ copies
        // Lane i finds the address of record i of every 32 (16 sub-tiles) and issues its
        // copy; the block-table entries of the next 32 are on their way meanwhile (one
        // lane looking up each page in turn held 64-position pages at a third of HBM's rate).
        const uint64_t policy = l2_policy_evict_first();
        const int rp = p.c.recs_per_page;
        int g = 0, issued = 0;
        bool stop = false;
        KvqPart q;
        while (!stop && walk.next(p.c, q)) {
            const int n = q.n;
            const int blk0 = (TK / kRecKeys) * q.t0;  // records of the part (capacity is below 2^31 positions)
            const int blk1 = min(blk0 + (TK / kRecKeys) * n, (q.len + kRecKeys - 1) / kRecKeys);
            const auto record = [&](int blk) -> const uint8_t * {
                if (blk >= blk1) return nullptr;
                int64_t page = q.b;
                int within = blk;
                if (p.c.block_table) {
                    const int e = blk / rp;
                    within = blk - e * rp;
                    page = p.c.block_table[(int64_t)q.b * p.c.max_pages + e];
                    if (page < 0 || page >= p.c.n_pages) {
                        kvq_report(p.err, WM_DEVERR_BAD_PAGE);
                        page = 0;
                    }
                }
                return p.c.data + ((page * p.c.n_kv_heads + q.h) * rp + within) * (int64_t)C::REC;
            };
            const uint8_t *cur = record(blk0 + lane);
            for (int i0 = 0; !stop && i0 < 2 * n; i0 += 16) {
                const uint8_t *next = record(blk0 + 2 * (i0 + 16) + lane);
                for (int i = i0; i < min(i0 + 16, 2 * n); ++i) {
                    const int u = 2 * g + i, s = u % NST;  // sub-tile of the run
                    bool ok = u != p.stall_tile;           // (the stall: tests of the timeout path only)
                    if (ok && u >= NST) ok = wait(bar_empty + 8 * s, u / NST - 1);
                    if (__any_sync(0xffffffffu, !ok)) {
                        stop = true;
                        break;
                    }
                    const int recs = min(2, max(0, blk1 - (blk0 + 2 * i)));
                    if (lane == 0) mbar_arrive_expect_tx(bar_full + 8 * s, recs * C::REC);
                    __syncwarp();
                    if (lane >> 1 == i - i0 && cur)
                        bulk_load(sST + s * C::STAGE + (lane & 1) * C::REC, cur, C::REC, bar_full + 8 * s, policy);
                    issued = u + 1;
                }
                cur = next;
            }
            g += n;
        }
        // never leave with copies still landing in this CTA's shared memory
        if (lane == 0)
            for (int u = max(0, issued - NST); u < issued; ++u)
                mbar_wait_bounded(bar_full + 8 * (u % NST), (u / NST) & 1, p.wait_limit);
    } else if (warp == 1) {
        // ============================================================ S = C_K . Q^T
        if (elect_one()) {
            constexpr uint32_t id_s = idesc_f16(NR, 0);
            const uint64_t q_desc = tc::smem_desc(sQ, 16, 1024, tc::SWIZZLE_128B);
            KvqPart q;
            int part = 0;
            bool ok = true;
            for (int g = 0; ok && walk.next(p.c, q); g += q.n, ++part) {
                ok = wait(bar_qfull, part);
                for (int t = 0; ok && t < q.n; ++t) {
                    const int gt = g + t;
                    if (gt >= 1) ok = wait(bar_sfree, gt - 1);
                    // with two P' buffers: S of a tile also says that its buffer is free
                    if (NPB == 2 && gt >= 2) ok = ok && wait(bar_odone + 8 * (gt & 1), (gt - 2) >> 1);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const int u = (2 * gt + j) * NC + c, slot = u % C::KS;
                            ok = ok && wait(bar_aready + 8 * slot, u / C::KS);
                            if (!ok) break;
                            tc::fence_after_sync();
                            const uint32_t a = tmem + 64 * slot, d = tmem + C::S_COL + j * NR;
#pragma unroll
                            for (int kk = 0; kk < 2 * C::KU; ++kk)  // 16 channels each
                                mma_f16_ts(d, a + 8 * kk,
                                           q_desc + (((2 * c + (kk >> 2)) * C::Q_REGION + (kk & 3) * 32) >> 4), id_s,
                                           c > 0 || kk > 0);
                            tc::commit(bar_afree + 8 * slot);
                        }
                    if (ok) {
                        tc::commit(bar_sfull);
                        // an arrival of this thread's own, which hands on what it has seen: the
                        // constants that the K warps wrote before their code slots
                        mbar_arrive(bar_sfull);
                    }
                }
            }
            tc::commit(bar_final);  // every MMA issued above has completed once this fires
            mbar_wait_bounded(bar_final, 0, p.wait_limit);
        }
    } else if (warp == 2) {
        // ============================================================ O += C_V^T . P'^T
        if (elect_one()) {
            constexpr uint32_t id_pv = idesc_f16(NR, 1);
            const uint64_t p_desc = tc::smem_desc(sPT, C::PT_BYTES, C::PT_ATOM, C::PT_SWIZZLE);
            KvqPart q;
            bool ok = true;
            for (int g = 0; ok && walk.next(p.c, q); g += q.n) {
                for (int t = 0; ok && t < q.n; ++t) {
                    const int gt = g + t, buf = gt % NPB;
                    ok = wait(bar_pfull + 8 * buf, gt / NPB);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint64_t pb = p_desc + ((buf * C::PB_BYTES + j * C::PT_BYTES) >> 4);
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const int u = (2 * gt + j) * NC + c, slot = u % C::VS;
                            ok = ok && wait(bar_aready + 8 * (C::KS + slot), u / C::VS);
                            if (!ok) break;
                            tc::fence_after_sync();
                            const uint32_t a = tmem + C::V_COL + 64 * slot, d = tmem + C::O_COL + c * NR;
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {  // 16 keys each
                                const uint64_t bp = pb + ((kk * 2 * C::PT_ATOM) >> 4);
                                mma_f16_ts(d, a + 8 * kk, bp, id_pv, t % kKvqChain > 0 || j > 0 || kk > 0);
                                mma_f16_ts(d, tmem + C::E_COL, bp, id_pv, 1u);
                            }
                            tc::commit(bar_afree + 8 * (C::KS + slot));
                        }
                    }
                    if (ok) tc::commit(bar_odone + 8 * buf);
                }
            }
            tc::commit(bar_final + 8);
            mbar_wait_bounded(bar_final + 8, 0, p.wait_limit);
        }
    } else if (warp < C::W_S) {
        // ============================================================ codes -> tensor memory
        const int dw = warp - C::W_D;
        const int q4 = warp & 3;
        const int L = 32 * q4 + lane;  // tensor-memory lane: key (K), channel of a chunk (V)
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;

        // A chunk's units of this lane are all loaded before the first is converted, so
        // that one latency of shared memory is paid.
        const auto convert = [&](const uint4 (&x)[4], int units, int slot, int use, bool live) {
            if (use > 0) wait(bar_afree + 8 * slot, use - 1);
            __syncwarp();
            tc::fence_after_sync();
            if (live) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < units) kvq_unit_to_tmem(tmem + lane_off + 64 * slot + 16 * j, x[j]);
            }
        };
        const auto ready = [&](int slot) {
            tc::wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_aready + 8 * slot);
        };
        const auto do_k = [&](int st) {
            wait(bar_full + 8 * (st % NST), st / NST);
            const uint32_t rec = sST + (st % NST) * C::STAGE + (L >> 6) * C::REC;
            const uint32_t unit = rec + (L & 63) * 16;
            const uint32_t ksz = ld_shared_u32(rec + rec_ks_off(D) + (L & 63) * 4);
            const uint32_t vsz = ld_shared_u32(rec + rec_vs_off(D) + (L & 63) * 4);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int u = st * NC + c;
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < C::KU; ++j) x[j] = ld_shared_v4(unit + (c * 4 + j) * 1024);
                convert(x, C::KU, u % C::KS, u / C::KS, true);
                if (c == 0) {
                    // Constants of this key.  Slot st % 4 is free once the code slot is: sub-tile
                    // st - 4's were read before S of the tile after it was issued, and the code
                    // slot waits for that S or a later one.
                    const float ks = __uint_as_float(ksz << 16), kz = __uint_as_float(ksz & 0xffff0000u);
                    const float vs = __uint_as_float(vsz << 16), vz = __uint_as_float(vsz & 0xffff0000u);
                    // Scale 0 (constant values, codes 0): a stand-in that keeps z / s in
                    // range.  At least 2^-86, which keeps the sums of P' / s below fp32's
                    // largest: values are off by 15 x 2^-86 where a scale is smaller.
                    const float se = fmaxf(vs > 0.f ? vs : fabsf(vz) * 0.00390625f, 1.2924697e-26f);
                    const bool by16 = L & 2;  // this key's V codes are 16 times too large: P' is divided by 16
                    const float up = by16 ? 16.f : 1.f;
                    float inv = rcp(se) * up, zr = fmaf(vz, inv, 8.f * up);
                    const bool bad = !(fabsf(ks) < CUDART_INF_F && fabsf(kz) < CUDART_INF_F && vs >= 0.f &&
                                       vs < CUDART_INF_F && fabsf(zr) < CUDART_INF_F);
                    // not finite: NaN in the logit reaches every row that sees this key, and only
                    // those (a weight of 0 times these is 0)
                    if (bad) inv = zr = 0.f;
                    const float ls = bad ? CUDART_NAN_F : lg2(se) - (by16 ? 4.f : 0.f);
                    st_shared_v4(s_const + ((st & 3) * 128 + L) * 16,
                                 make_uint4(__float_as_uint(ks * 16777216.f), __float_as_uint(kz), __float_as_uint(ls),
                                            __float_as_uint(inv)));
                    st_shared_f32(s_zr + ((st & 3) * 128 + L) * 4, zr);
                }
                ready(u % C::KS);
            }
            if (lane == 0) mbar_arrive(bar_empty + 8 * (st % NST));
        };
        const auto do_v = [&](int st) {
            // head_dim 64: lanes 64..127 have no channel; their rows of O are never read
            const bool live = D > 64 || q4 < 2;
            wait(bar_full + 8 * (st % NST), st / NST);
            const uint32_t unit = sST + (st % NST) * C::STAGE + rec_v_off(D) + L * 16;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int u = st * NC + c;
                uint4 x[4];
                if (live) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = ld_shared_v4(unit + c * 2048 + (j >> 1) * C::REC + (j & 1) * 16 * D);
                }
                convert(x, 4, C::KS + u % C::VS, u / C::VS, live);
                ready(C::KS + u % C::VS);
            }
            if (lane == 0) mbar_arrive(bar_empty + 8 * (st % NST));
        };
        // (Once the pipeline is given up every wait returns at once, and the loops run out.)
        const int n_sub = 2 * n_all;
        if constexpr (ND > 4) {
            const int grp = dw >> 2;
            if (grp < C::KG)
                for (int st = grp; st < n_sub; st += C::KG) do_k(st);
            else
                for (int st = grp - C::KG; st < n_sub; st += C::VG) do_v(st);
        } else {
            // one group: the next tile's K before this tile's V, so that S runs ahead
            do_k(0);
            do_k(1);
            for (int st = 0; st < n_sub; ++st) {
                if (st + 2 < n_sub) do_k(st + 2);
                do_v(st);
            }
        }
    } else {
        // ============================================================ softmax
        const int sw = warp - C::W_S;
        const int q4 = warp & 3;
        const int grp = sw >> 2;            // warps 4 grp .. 4 grp + 3 share rows r0 .. r0 + HR - 1
        const int r0 = grp * HR;
        const int kt = 32 * q4 + lane;      // tensor-memory lane: key of each sub-tile, channel of each O block
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const int ct = threadIdx.x - 32 * C::W_S;

        // Queries of unit (b, h), for part number `part`, as fp16: divided by one
        // power of two per unit so that the largest magnitude is in [2^14, 2^15) --
        // bf16's 8 bits survive down to 2^-27 of it even where a channel's 16 is
        // divided out -- and each row's sum.  Returns the power of two's inverse.
        const auto stage_q = [&](int b, int h, int part) -> float {
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
            constexpr int VPR = D / 8;  // 16-byte vectors per row: 8, 16 or 32 lanes
            constexpr int PER = (NR * VPR + 32 * NSW - 1) / (32 * NSW);  // vectors per thread
            static_assert(NR * VPR % 32 == 0, "whole warps");
            uint4 x[PER];
            uint32_t top = 0;  // largest magnitude's bits, infinities and NaN left out
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int idx = ct + 32 * NSW * k, r = idx / VPR, v = idx % VPR;
                x[k] = make_uint4(0u, 0u, 0u, 0u);
                if (r < p.rows) {
                    const int i = r / p.group, hh = r - i * p.group;
                    const int64_t row = ((int64_t)b * p.n_q + i) * p.n_q_heads + h * p.group + hh;
                    x[k] = __ldg(reinterpret_cast<const uint4 *>(q + row * D) + v);
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
                    if (lo < 0x7f80u) top = max(top, lo);
                    if (hi < 0x7f80u) top = max(top, hi);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) flags[8 + sw] = (int)top;
            named_bar_sync(1, 32 * NSW);
#pragma unroll
            for (int w = 0; w < NSW; ++w) top = max(top, (uint32_t)flags[8 + w]);
            const int ex = top == 0 ? 0 : min(100, max(-100, (int)(top >> 7) - 127 - 14));
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (ct < NR) st_shared_f32(s_nm + ((part & 1) * NR + ct) * 4, 0.f);
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int idx = ct + 32 * NSW * k, r = idx / VPR, v = idx % VPR;
                if (idx >= NR * VPR) break;  // whole warps
                const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
                uint32_t o[4];
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float fac = j & 1 ? down * 0.0625f : down;  // elements 2, 3, 6, 7 meet codes times 16
                    const __half2 hv = __floats2half2_rn(__uint_as_float(w[j] << 16) * fac,
                                                         __uint_as_float(w[j] & 0xffff0000u) * fac);
                    const float2 f2 = __half22float2(hv);
                    sum += (j & 1 ? 16.f : 1.f) * (f2.x + f2.y);
                    o[j] = *reinterpret_cast<const uint32_t *>(&hv);
                }
                st_shared_v4(sQ + (v >> 3) * C::Q_REGION + swz128(r, v & 7), make_uint4(o[0], o[1], o[2], o[3]));
#pragma unroll
                for (int o2 = VPR / 2; o2; o2 >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o2);
                if (v == 0) st_shared_f32(s_zq + ((part & 1) * NR + r) * 4, sum);
            }
            fence_proxy_async_smem();
            named_bar_sync(1, 32 * NSW);  // sums and maxima visible
            if (lane == 0) mbar_arrive(bar_qfull);
            return __uint_as_float((uint32_t)(127 + ex) << 23);
        };

        // This thread's addresses: its keys' constants, its row of P' (its first 16-byte unit,
        // swizzled; with 16 rows per warp the second is the neighbour in a pair).
        const uint32_t c_at = s_const + kt * 16, z_at = s_zr + kt * 4;
        const uint32_t swizzle = C::PT_ROW == 128 ? kt & 7 : C::PT_ROW == 64 ? (kt >> 1) & 3 : (kt >> 2) & 1;
        const uint32_t p_at = sPT + kt * C::PT_ROW + ((r0 / 8 ^ swizzle) << 4);

        KvqPart q;
        int g = 0, part = 0;
        bool have = walk.next(p.c, q);
        float f = have ? stage_q(q.b, q.h, 0) * p.scale_log2 : 0.f;
        while (have) {
            // positions fit 32 bits (the capacity does)
            const int n = q.n, key_first = q.t0 * TK;
            const int key_end = (int)min((int64_t)(q.t0 + n) * TK, (int64_t)q.len);
            const int qpos0 = q.len - p.n_q;
            const uint32_t zq = s_zq + ((part & 1) * NR + r0) * 4, nm = s_nm + ((part & 1) * NR + r0) * 4;

            uint64_t l2[HR / 2], z2[HR / 2];  // sums of P' / s_V and P' z_V / s_V, two rows each
#pragma unroll
            for (int i = 0; i < HR / 2; ++i) l2[i] = z2[i] = 0;
            const int64_t seg = (int64_t)blockIdx.x + (int64_t)q.b * p.c.n_kv_heads + q.h;
            // What was taken over of O before (n_over times, at least once), for 8 rows at the present
            // maxima, added to o8.
            const auto add_over = [&](int c, int j, int n_over, float (&o8)[8]) {
                const int d = c * 128 + kt;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + 8 * j + i;
                    if (r >= p.rows || (D == 64 && d >= 64)) continue;
                    const float np = ld_shared_f32(s_np + (((n_over - 1) & 1) * NR + r) * 4);
                    o8[i] = fmaf(p.o_part[(seg * p.rows + r) * D + d], ex2(ld_shared_f32(nm + 4 * (8 * j + i)) - np),
                                 o8[i]);
                }
            };
            for (int t = 0; t < n; ++t) {
                const int gt = g + t;
                const int key0 = key_first + t * TK;

                if (__builtin_expect(t > 0 && t % kKvqChain == 0, 0)) {
                    // take O over (it is at the maxima of the last tile, which are still the present ones)
                    wait(bar_odone + 8 * ((gt - 1) % NPB), (gt - 1) / NPB);
                    __syncwarp();
                    tc::fence_after_sync();
                    const int n_over = t / kKvqChain - 1;
#pragma unroll 1
                    for (int c = 0; c < NC; ++c)
#pragma unroll 1
                        for (int j = 0; j < HR / 8; ++j) {
                            float o8[8];
                            tc::ld_32x32b_x8(tmem + lane_off + C::O_COL + c * NR + r0 + 8 * j, o8);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o8[i] *= 16777216.f;
                            if (n_over > 0) add_over(c, j, n_over, o8);
                            const int d = c * 128 + kt;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = r0 + 8 * j + i;
                                if (r < p.rows && (D > 64 || d < 64)) p.o_part[(seg * p.rows + r) * D + d] = o8[i];
                            }
                        }
                    // (read by the next one, many barriers from here)
                    if (q4 == 0 && lane < HR)
                        st_shared_f32(s_np + ((n_over & 1) * NR + r0 + lane) * 4, ld_shared_f32(nm + 4 * lane));
                    tc::fence_before_sync();
                }

                wait(bar_sfull, gt);
                __syncwarp();
                tc::fence_after_sync();
                float s[2][HR];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t at = tmem + lane_off + C::S_COL + j * NR + r0;
                    if constexpr (HR == 16)
                        tc::ld_32x32b_x16(at, s[j]);
                    else
                        tc::ld_32x32b_x8(at, s[j]);
                }
                tc::wait_ld();
                tc::fence_before_sync();

                // t - m of every row
                const uint32_t held = 2 * gt & 3;
                uint64_t a2[2], b2[2], ls2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 kc = ld_shared_v4(c_at + (held + j) * 2048);
                    const float a = __uint_as_float(kc.x) * f, bz = __uint_as_float(kc.y) * f;
                    a2[j] = pack2(a, a);
                    b2[j] = pack2(bz, bz);
                    ls2[j] = pack2(__uint_as_float(kc.z), __uint_as_float(kc.z));
                }
#pragma unroll
                for (int i = 0; i < HR; i += 4) {
                    const ulonglong2 z4 = ld_shared_pairs(zq + 4 * i), m4 = ld_shared_pairs(nm + 4 * i);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float *x = s[j] + i;
                        unpack2(fma2(pack2(x[0], x[1]), a2[j], fma2(z4.x, b2[j], add2(ls2[j], m4.x))), x[0], x[1]);
                        unpack2(fma2(pack2(x[2], x[3]), a2[j], fma2(z4.y, b2[j], add2(ls2[j], m4.y))), x[2], x[3]);
                    }
                }
                float inv[2], zr[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    inv[j] = ld_shared_f32(c_at + (held + j) * 2048 + 12);
                    zr[j] = ld_shared_f32(z_at + (held + j) * 512);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sfree);  // S and the constants are read
                if (key0 + TK > key_end || key0 + TK - 1 > qpos0) {
                    // row r sees a key iff it is below key_end and at most qpos0 + r / group
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = key0 + 128 * j + kt;
                        // first row that sees it: query position key - qpos0, if that is not before the first
                        const int row = key >= key_end ? NR : min(max(key - qpos0, 0), NR) * p.group;
#pragma unroll
                        for (int i = 0; i < HR; ++i)
                            if (r0 + i < row) s[j][i] = -CUDART_INF_F;
                    }
                }
                float top = fmaxf(s[0][0], s[1][0]);
#pragma unroll
                for (int i = 1; i < HR; ++i) top = fmaxf(fmaxf(top, s[0][i]), s[1][i]);
                const bool raise = named_bar_sync_or(2 + grp, 128, top > kKvqOff + kKvqRaise);
                if (raise || t == 0) {
                    // Raise the maxima of this group's rows (at the part's first tile: set them).
#pragma unroll
                    for (int i = 0; i < HR; ++i) {
                        const float mx = warp_max_f(fmaxf(s[0][i], s[1][i]));
                        if (lane == 0) st_shared_f32(s_red + (4 * (r0 + i) + q4) * 4, mx);
                    }
                    named_bar_sync(2 + grp, 128);
                    // Lane i holds by how much the maximum of row i of HR goes up; the others ask it.
                    const float4 m4 = ld_shared_f4(s_red + 16 * (r0 + lane % HR));
                    const float mx = fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)) - kKvqOff;
                    const float up = t > 0 ? fmaxf(mx, 0.f) : mx == -CUDART_INF_F ? 0.f : mx, down = ex2(-up);
                    if (q4 == 0 && lane < HR) st_shared_f32(nm + 4 * lane, ld_shared_f32(nm + 4 * lane) - up);
#pragma unroll
                    for (int i = 0; i < HR; ++i) {
                        const float d = __shfl_sync(0xffffffffu, up, i);
                        s[0][i] -= d;
                        s[1][i] -= d;
                    }
                    if (t > 0) {
#pragma unroll
                        for (int j = 0; j < HR / 8; ++j) {
                            float al[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) al[i] = __shfl_sync(0xffffffffu, down, 8 * j + i);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint64_t al2 = pack2(al[2 * i], al[2 * i + 1]);
                                l2[4 * j + i] = mul2(l2[4 * j + i], al2);
                                z2[4 * j + i] = mul2(z2[4 * j + i], al2);
                            }
                        }
                    }
                    if (t % kKvqChain > 0) {
                        // O holds tiles at the old maxima
                        wait(bar_odone + 8 * ((gt - 1) % NPB), (gt - 1) / NPB);
                        __syncwarp();
                        tc::fence_after_sync();
                        // (unrolled, these loops cost the common path registers: 2 x 1M 696 us for 671)
#pragma unroll 1
                        for (int j = 0; j < HR / 8; ++j) {
                            float al[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) al[i] = __shfl_sync(0xffffffffu, down, 8 * j + i);
#pragma unroll 1
                            for (int c = 0; c < NC; ++c) {
                                const uint32_t at = tmem + lane_off + C::O_COL + c * NR + r0 + 8 * j;
                                float v8[8];
                                tc::ld_32x32b_x8(at, v8);
                                tc::wait_ld();
#pragma unroll
                                for (int i = 0; i < 8; ++i) v8[i] *= al[i];
                                tc::st_32x32b_x8(at, v8);
                            }
                        }
                        tc::wait_st();
                    }
                    named_bar_sync(2 + grp, 128);  // the new maxima are visible, red is free
                }

                // with one P' buffer: the last tile's products have read it
                if (NPB == 1 && gt >= 1) wait(bar_odone, gt - 1);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint64_t inv2 = pack2(inv[j], inv[j]), zr2 = pack2(zr[j], zr[j]);
                    const uint32_t pt = p_at + (gt % NPB) * C::PB_BYTES;
#pragma unroll
                    for (int i0 = 0; i0 < HR; i0 += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int i = i0 / 2 + k;
                            const float x = ex2(s[j][2 * i]), y = ex2(s[j][2 * i + 1]);
                            const uint64_t x2 = pack2(x, y);
                            l2[i] = fma2(x2, inv2, l2[i]);
                            z2[i] = fma2(x2, zr2, z2[i]);
                            const __half2 hv = __floats2half2_rn(x, y);
                            w[k] = *reinterpret_cast<const uint32_t *>(&hv);
                        }
                        st_shared_v4((pt ^ (2 * i0)) + j * C::PT_BYTES, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pfull + 8 * (gt % NPB));
            }

            have = walk.next(p.c, q);
            // The next part's queries, while the last P.V runs: the last S of this part
            // was read above, so every S that used the query buffer is complete.
            if (have) f = stage_q(q.b, q.h, part + 1) * p.scale_log2;

            // ---- the part's result: this thread owns tensor-memory lane kt of every O block
            const int g_last = g + n - 1;
            // Sums over the lanes: halve the values and the lanes that hold them at each step
            // (HR = 16: 31 shuffles for 32 sums), until lane i holds sum number i.
            float y[2 * HR];
#pragma unroll
            for (int i = 0; i < HR / 2; ++i) {
                unpack2(l2[i], y[2 * i], y[2 * i + 1]);
                unpack2(z2[i], y[HR + 2 * i], y[HR + 2 * i + 1]);
            }
#pragma unroll
            for (int o = HR; o >= 1; o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const float send = up ? y[i] : y[i + o], keep = up ? y[i + o] : y[i];
                    y[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
            if (HR == 8) y[0] += __shfl_xor_sync(0xffffffffu, y[0], 16);
            if (lane < 2 * HR)  // sums of l, then of z
                st_shared_f32(s_red + (lane / HR) * 16 * NR + (4 * (r0 + lane % HR) + q4) * 4, y[0]);
            named_bar_sync(2 + grp, 128);
            wait(bar_odone + 8 * (g_last % NPB), g_last / NPB);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll
            for (int j = 0; j < HR / 8; ++j) {
                float l8[8], z8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t at = s_red + 16 * (r0 + 8 * j + i);
                    const float4 x = ld_shared_f4(at), z = ld_shared_f4(at + 16 * NR);
                    l8[i] = (x.x + x.y) + (x.z + x.w);
                    z8[i] = (z.x + z.y) + (z.z + z.w);
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float o8[8];
                    tc::ld_32x32b_x8(tmem + lane_off + C::O_COL + c * NR + r0 + 8 * j, o8);
                    tc::wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) o8[i] = fmaf(o8[i], 16777216.f, z8[i]);
                    if (__builtin_expect(n > kKvqChain, 0)) add_over(c, j, (n - 1) / kKvqChain, o8);
                    const int d = c * 128 + kt;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + 8 * j + i;
                        if (r >= p.rows || (D == 64 && d >= 64)) continue;
                        p.o_part[(seg * p.rows + r) * D + d] = l8[i] == 0.f ? 0.f : o8[i] / l8[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + 8 * j + i;
                    if (r < p.rows && kt == r)
                        p.lse_part[seg * p.rows + r] = l8[i] == 0.f ? -CUDART_INF_F : lg2(l8[i]) - ld_shared_f32(nm + 4 * (8 * j + i));
                }
            }
            // O has been read (wait_ld) before this warp's next pfull arrival, which gates the next part's first P.V
            tc::fence_before_sync();
            g += n;
            ++part;
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, int NR, int LIVE = NR>
cudaError_t launch_kvq_attn_nr(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    constexpr int smem = KvqCfg<D, NR, LIVE>::TOTAL;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kvq_attn_kernel<D, NR, LIVE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_pdl(kvq_attn_kernel<D, NR, LIVE>, dim3(n_cta), dim3(KvqCfg<D, NR, LIVE>::THREADS), smem, stream, p);
}

template <int D>
cudaError_t launch_kvq_attn_d(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    // Rows past the last query's have no softmax warps where that frees a group of them: single
    // tokens of 16 sequences of 32K-64K, 8 rows of 128, 82 us (with warps for 16 rows 94); one
    // sequence of 512K, 24 rows of 128, 77 (with warps for 32 rows 86).
    if (p.rows <= 8) return launch_kvq_attn_nr<D, 16, 8>(p, n_cta, stream);
    switch ((p.rows + 15) / 16) {
        case 1: return launch_kvq_attn_nr<D, 16>(p, n_cta, stream);
        case 2:
            return p.rows <= 24 ? launch_kvq_attn_nr<D, 32, 24>(p, n_cta, stream)
                                : launch_kvq_attn_nr<D, 32>(p, n_cta, stream);
        case 3: return launch_kvq_attn_nr<D, 48>(p, n_cta, stream);
        case 4: return launch_kvq_attn_nr<D, 64>(p, n_cta, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace wm
