// attn_kvq.cuh -- causal attention over the 4-bit KV cache on the 5th-generation
// tensor cores.
//
// With l_j = s_j (q . c_j) + z_j sum(q) the products run over the codes alone:
//   S^T[128 keys x NR] = C_K[128 x D] . Q^T        (A: codes in tensor memory, B: Q^T in shared memory)
//   O^T[D x NR]       += C_V^T[D x 128] . P'^T     (A: codes in tensor memory, B: P'^T in shared memory)
// A code c <= 15 widened to 16 bits is the fp16 subnormal c 2^-24, exactly, so
// the conversion is one shift and one mask per two codes.  The codes go to
// tensor memory rather than shared memory: as 16-bit operands in shared memory
// they would cost 2 bytes written and 2 read per code where HBM delivers half a
// byte, more than shared memory's 128 bytes per clock when HBM runs at full rate.
// Keys (for S) and channels (for O) are the MMA's M, so the few query rows are N.
//
// K's scale and zero enter the logit (log2 units, key j, row r):
//   t_jr = S_jr a_j + zq_r b_j + ls_j,  a = s_K 2^24 f,  b = z_K f,  f = scale log2(e)
//   zq_r = sum_d q_rd,  ls_j = log2(s_V).
// V's scale is folded into the weight: P'_jr = 2^(t_jr - m_r) = s_Vj p_jr, so that
//   o_r = [ 2^24 sum_j P'_jr c_j  +  sum_j P'_jr (z_V / s_V)_j ] / sum_j P'_jr (1 / s_V)_j
// with the running maximum m taken over t: the largest P' is near the top of fp16's range
// whatever the scales are.  P' is rounded to fp16 (at most 2^-11 of it) for the
// tensor cores, and the two sums use the rounded P', in fp32: a common rounding
// of equal weights then cancels between the products, zeros and normaliser -- which
// matters because s c and z are large beside their sum.  A row of
// constant values has s_V = 0 and codes 0; a stand-in scale |z| / 256 carries its zero.
//
// Each CTA takes one run of the batch's tiles (kvq_schedule), cut into parts at
// (sequence, KV head) borders; every role counts tiles across parts, so no
// buffer drains at a border.  Roles:
//   warp 0      bulk copies: the two 64-position records of a tile, K and V and scales, one stage
//   warp 1      tensor memory; one lane issues the MMAs
//   ND warps    codes -> tensor memory: a thread per key (K) or channel (V)
//   NSW warps   softmax: a thread per key, HR rows each
// What bounds it: HBM, as long as the instructions per tile fit beside it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace wm {

constexpr int kKvqPageCache = 256;   // block-table entries of a part kept in shared memory
constexpr float kKvqOff = 7.f;       // the running maximum sits at 2^7 in P': fp16 keeps 11 bits down to 2^-21 of it
constexpr float kKvqRaise = 8.f;     // raise the maximum only past 2^8 (P' <= 2^15, fp16 holds up to 65504)
constexpr float kKvqFloor = -1e30f;  // running-maximum start, below any finite logit

template <int D_, int NR_>
struct KvqCfg {
    static constexpr int D = D_, NR = NR_;
    static constexpr int REC = rec_bytes(D);
    static constexpr int TILE = 2 * REC;
    static constexpr int NC = D == 256 ? 2 : 1;         // 128-channel chunks
    static constexpr int KU = D == 64 ? 2 : 4;          // 16-byte units per key and chunk
    static constexpr int ND = NR <= 32 ? 8 : 4;         // dequantising warps
    static constexpr int HR = NR <= 32 ? 8 : 16;        // rows per softmax warp
    static constexpr int NSW = 4 * (NR / HR);           // softmax warps
    static constexpr int THREADS = 32 * (2 + ND + NSW);
    // tensor memory: two K and two V code slots of 64 columns, S twice, O
    static constexpr int S_COL = 256, O_COL = 256 + 2 * NR;
    static_assert(O_COL + NC * NR <= 512, "tensor memory");
    // shared memory
    static constexpr int PT_ROW = NR <= 16 ? 32 : NR <= 32 ? 64 : 128;
    static constexpr uint32_t PT_SWIZZLE = NR <= 16 ? tc::SWIZZLE_32B : NR <= 32 ? tc::SWIZZLE_64B : tc::SWIZZLE_128B;
    static constexpr int PT_ATOM = 8 * PT_ROW, PT_BYTES = kKvqTile * PT_ROW;
    static constexpr int Q_REGION = NR * 128;           // 64 channels of every row
    static constexpr int Q_OFF = 0;
    static constexpr int PT_OFF = Q_OFF + (D / 64) * Q_REGION;
    static constexpr int ST_OFF = PT_OFF + 2 * PT_BYTES;
    static constexpr int FIXED = ST_OFF + 8 * NR * 4 + 2 * NR * 4 + 256 + 4 * kKvqPageCache + 64 * 8 + 512 + 1024;
    static constexpr int FIT = (227 * 1024 - FIXED) / TILE;
    static constexpr int NST = FIT > 8 ? 8 : FIT;       // 8 stages of 17 KB cover the latency of HBM
    static_assert(NST >= 2, "stages");
    static constexpr int RED_OFF = ST_OFF + NST * TILE;  // float [2][4][NR]
    static constexpr int ZQ_OFF = RED_OFF + 8 * NR * 4;  // float [NR] sums of the queries
    static constexpr int M_OFF = ZQ_OFF + NR * 4;        // float [NR] running maxima (less kKvqOff)
    static constexpr int FLAG_OFF = M_OFF + NR * 4;      // int [64]: [0] abort, [8 + 16 buf + w] votes, [40 + w] scratch
    static constexpr int BT_OFF = FLAG_OFF + 256;
    static constexpr int BAR_OFF = BT_OFF + 4 * kKvqPageCache;
    static constexpr int NBAR = 2 * NST + 4 + 4 + 8 + 2;
    static constexpr int WARP_OFF = (BAR_OFF + NBAR * 8 + 15) / 16 * 16;  // int64 [32] + int4 of the schedule
    static constexpr int TPTR_OFF = WARP_OFF + 32 * 8 + 16;
    static constexpr int TOTAL = TPTR_OFF + 16 + 1024;
    static_assert(TOTAL <= 227 * 1024, "shared memory");
    static_assert(PT_OFF % 1024 == 0 && ST_OFF % 128 == 0 && RED_OFF % 16 == 0, "alignment");
};

// 16 fp16 pairs of one 16-byte unit (32 codes), in order, to 16 columns of this lane.
__device__ __forceinline__ void kvq_unit_to_tmem(uint32_t taddr, uint4 u) {
    constexpr uint32_t M = 0x000f000fu;
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};" ::"r"(taddr),
        "r"(u.x & M), "r"((u.x >> 4) & M), "r"((u.x >> 8) & M), "r"((u.x >> 12) & M), "r"(u.y & M),
        "r"((u.y >> 4) & M), "r"((u.y >> 8) & M), "r"((u.y >> 12) & M), "r"(u.z & M), "r"((u.z >> 4) & M),
        "r"((u.z >> 8) & M), "r"((u.z >> 12) & M), "r"(u.w & M), "r"((u.w >> 4) & M), "r"((u.w >> 8) & M),
        "r"((u.w >> 12) & M)
        : "memory");
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

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
            "r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// The abort flag as lane 0 sees it: every lane takes the same branch around
// warp-collective tensor-memory accesses.
__device__ __forceinline__ bool kvq_aborted(volatile int *flags) {
    return __shfl_sync(0xffffffffu, flags[0], 0) != 0;
}

template <int D, int NR>
__global__ void __launch_bounds__(KvqCfg<D, NR>::THREADS, 1) kvq_attn_kernel(const KvqAttnParams p) {
    using C = KvqCfg<D, NR>;
    constexpr int TK = kKvqTile, NC = C::NC, HR = C::HR, NSW = C::NSW, ND = C::ND, NST = C::NST;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *gb = smem_raw + (sbase - raw);
    const uint32_t sQ = sbase + C::Q_OFF, sPT = sbase + C::PT_OFF, sST = sbase + C::ST_OFF;
    float *red = reinterpret_cast<float *>(gb + C::RED_OFF);  // [2][4][NR]
    float *s_zq = reinterpret_cast<float *>(gb + C::ZQ_OFF);
    float *s_m = reinterpret_cast<float *>(gb + C::M_OFF);
    volatile int *flags = reinterpret_cast<volatile int *>(gb + C::FLAG_OFF);
    const uint32_t bars = sbase + C::BAR_OFF;
    const uint32_t bar_full = bars;                      // [NST] stage landed
    const uint32_t bar_empty = bar_full + 8 * NST;       // [NST] stage read by everyone
    const uint32_t bar_aready = bar_empty + 8 * NST;     // [4] code slot written (K, K, V, V)
    const uint32_t bar_afree = bar_aready + 32;          // [4] code slot consumed
    const uint32_t bar_sfull = bar_afree + 32;           // [2]
    const uint32_t bar_sfree = bar_sfull + 16;           // [2]
    const uint32_t bar_pfull = bar_sfree + 16;           // [2]
    const uint32_t bar_odone = bar_pfull + 16;           // [2]
    const uint32_t bar_qfull = bar_odone + 16;           // phase k: queries of part k written
    const uint32_t bar_final = bar_qfull + 8;
    uint32_t *tptr = reinterpret_cast<uint32_t *>(gb + C::TPTR_OFF);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    // Set-up that touches only shared and tensor memory, while the previous kernel drains.
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 8 + NSW);  // K and V conversion (4 warps each), softmax
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar_aready + 8 * i, 4);
            mbar_init(bar_afree + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_sfull + 8 * i, 1);
            mbar_init(bar_sfree + 8 * i, NSW);
            mbar_init(bar_pfull + 8 * i, NSW);
            mbar_init(bar_odone + 8 * i, 1);
        }
        mbar_init(bar_qfull, NSW);
        mbar_init(bar_final, 1);
        for (int i = 0; i < 64; ++i) flags[i] = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(tptr), 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tptr;

    pdl_wait();
    pdl_launch_dependents();
    const int4 start = kvq_schedule(p, reinterpret_cast<int64_t *>(gb + C::WARP_OFF),
                                    reinterpret_cast<int4 *>(gb + C::WARP_OFF + 32 * 8));
    const int n_all = start.w;
    if (n_all <= 0) {
        if (warp == 1) tc::tmem_dealloc(tmem, 512);
        return;
    }
    KvqWalk walk;
    walk.init(start);

    // A wait that ran out: record it and make every role stop.
    const auto lost = [&]() {
        kvq_report(p.err, WM_DEVERR_TIMEOUT);
        flags[0] = 1;
    };

    if (warp == 0) {
        // ============================================================ copies
        int32_t *pages = reinterpret_cast<int32_t *>(gb + C::BT_OFF);
        const uint64_t policy = l2_policy_evict_first();
        const int rp = p.c.recs_per_page;
        int b = 0, h = 0, t0 = 0, n = 0, g = 0, issued = 0;
        bool stop = false;
        while (!stop && walk.next(p.c, b, h, t0, n)) {
            const int64_t len = kvq_len(p.c, b);
            const int64_t blk0 = 2 * (int64_t)t0;
            const int64_t blk1 = min(blk0 + 2 * (int64_t)n, (len + kRecKeys - 1) / kRecKeys);  // records of the part
            const int64_t page0 = p.c.block_table ? blk0 / rp : 0;
            const int32_t *bt = p.c.block_table ? p.c.block_table + (int64_t)b * p.c.max_pages + page0 : nullptr;
            if (bt) {
                __syncwarp();
                const int64_t n_pages = (blk1 - 1) / rp - page0 + 1;
                for (int i = lane; i < kKvqPageCache && i < n_pages; i += 32) pages[i] = bt[i];
                __syncwarp();
            }
            if (lane == 0) {
                int64_t local = 0;                             // page of the part
                int within = (int)(blk0 - page0 * rp);         // record of the page
                int64_t blk = blk0;
                for (int t = 0; t < n; ++t) {
                    const int gt = g + t, s = gt % NST;
                    if (gt == p.stall_tile) {  // tests of the timeout path only
                        stop = true;
                        break;
                    }
                    if (gt >= NST && !mbar_wait_bounded(bar_empty + 8 * s, ((gt / NST) & 1) ^ 1, p.wait_limit)) {
                        lost();
                        stop = true;
                        break;
                    }
                    if (flags[0]) {
                        stop = true;
                        break;
                    }
                    const int recs = (int)min((int64_t)2, blk1 - blk);
                    const uint32_t dst = sST + s * C::TILE;
                    mbar_arrive_expect_tx(bar_full + 8 * s, recs * C::REC);
                    for (int r = 0; r < recs;) {
                        int64_t page = b;
                        int run = recs - r;  // records copied together
                        if (bt) {
                            page = local < kKvqPageCache ? pages[local] : bt[local];
                            if (page < 0 || page >= p.c.n_pages) {
                                kvq_report(p.err, WM_DEVERR_BAD_PAGE);
                                page = 0;
                            }
                            run = min(run, rp - within);
                        }
                        bulk_load(dst + r * C::REC,
                                  p.c.data + ((page * p.c.n_kv_heads + h) * rp + within) * (int64_t)C::REC,
                                  run * C::REC, bar_full + 8 * s, policy);
                        r += run;
                        blk += run;
                        within += run;
                        if (bt && within == rp) {
                            within = 0;
                            ++local;
                        }
                    }
                    issued = gt + 1;
                }
            }
            stop = __shfl_sync(0xffffffffu, stop, 0);
            g += n;
        }
        // never leave with copies still landing in this CTA's shared memory
        if (lane == 0)
            for (int gt = max(0, issued - NST); gt < issued; ++gt)
                mbar_wait_bounded(bar_full + 8 * (gt % NST), (gt / NST) & 1, p.wait_limit);
    } else if (warp == 1) {
        // ============================================================ MMA issue
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_f16(NR, 0), id_pv = idesc_f16(NR, 1);
            KvqWalk walk_p = walk;  // one walker for S (tile ts), one for P.V (tile tp)
            int xb, xh, xt, xn;
            int ts_end = walk.next(p.c, xb, xh, xt, xn) ? xn : n_all;
            int tp_first = 0, tp_end = walk_p.next(p.c, xb, xh, xt, xn) ? xn : n_all;
            int part = 0;
            bool q_ready = false, ok = true;
            int ts = 0, cs = 0, tp = 0, cp = 0;
            uint32_t idle = 0;
            while (tp < n_all) {
                if (flags[0]) break;
                bool did = false;
                if (ts < n_all) {
                    if (ts == ts_end) {
                        ts_end = ts + (walk.next(p.c, xb, xh, xt, xn) ? xn : n_all);
                        ++part;
                        q_ready = false;
                    }
                    if (!q_ready) q_ready = mbar_test(bar_qfull, part & 1);
                    const int u = ts * NC + cs, slot = u & 1;
                    if (q_ready && mbar_test(bar_aready + 8 * slot, (u >> 1) & 1) &&
                        (cs > 0 || ts < 2 || mbar_test(bar_sfree + 8 * (ts & 1), ((ts - 2) >> 1) & 1))) {
                        tc::fence_after_sync();
                        const uint32_t d = tmem + C::S_COL + (ts & 1) * NR;
#pragma unroll
                        for (int kk = 0; kk < 2 * C::KU; ++kk) {
                            const int kg = cs * 8 + kk;
                            mma_f16_ts(d, tmem + 64 * slot + 8 * kk,
                                       tc::smem_desc(sQ + (kg >> 2) * C::Q_REGION + (kg & 3) * 32, 16, 1024,
                                                     tc::SWIZZLE_128B),
                                       id_s, kg != 0);
                        }
                        tc::commit(bar_afree + 8 * slot);
                        if (++cs == NC) {
                            tc::commit(bar_sfull + 8 * (ts & 1));
                            cs = 0;
                            ++ts;
                        }
                        did = true;
                    }
                }
                if (tp < ts) {
                    if (tp == tp_end) {
                        tp_first = tp;
                        tp_end = tp + (walk_p.next(p.c, xb, xh, xt, xn) ? xn : n_all);
                    }
                    const int u = tp * NC + cp, slot = 2 + (u & 1);
                    if (mbar_test(bar_aready + 8 * slot, (u >> 1) & 1) &&
                        (cp > 0 || mbar_test(bar_pfull + 8 * (tp & 1), (tp >> 1) & 1))) {
                        tc::fence_after_sync();
                        const uint32_t pt = sPT + (tp & 1) * C::PT_BYTES;
                        const uint32_t d = tmem + C::O_COL + cp * NR;
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            mma_f16_ts(d, tmem + 64 * slot + 8 * kk,
                                       tc::smem_desc(pt + kk * 2 * C::PT_ATOM, C::PT_BYTES, C::PT_ATOM, C::PT_SWIZZLE),
                                       id_pv, tp != tp_first || kk != 0);
                        tc::commit(bar_afree + 8 * slot);
                        if (++cp == NC) {
                            tc::commit(bar_odone + 8 * (tp & 1));
                            cp = 0;
                            ++tp;
                        }
                        did = true;
                    }
                }
                if (did) {
                    idle = 0;
                } else if (++idle > p.wait_limit) {
                    ok = false;
                    break;
                } else if (idle > 64) {
                    __nanosleep(32);
                }
            }
            if (!ok) lost();
            tc::commit(bar_final);  // every MMA issued above has completed once this fires
            mbar_wait_bounded(bar_final, 0, p.wait_limit);
        }
    } else if (warp < 2 + ND) {
        // ============================================================ codes -> tensor memory
        const int dw = warp - 2;
        const int q4 = warp & 3;
        const int L = 32 * q4 + lane;  // tensor-memory lane: key (K), channel of a chunk (V)
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;

        // One slot of 64 columns from the tile's stage; false once aborted.
        const auto fill = [&](int u, int slot, auto &&unit_addr, int units, bool live) {
            if (u >= 2 && !flags[0] &&
                !mbar_wait_bounded(bar_afree + 8 * slot, ((u >> 1) & 1) ^ 1, p.wait_limit))
                lost();
            tc::fence_after_sync();
            const bool go = !kvq_aborted(flags);
            if (go && live) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < units)
                        kvq_unit_to_tmem(tmem + lane_off + 64 * slot + 16 * j, ld_shared_v4(unit_addr(j)));
                tc::wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_aready + 8 * slot);
        };
        const auto landed = [&](int gt) {
            if (!flags[0] && !mbar_wait_bounded(bar_full + 8 * (gt % NST), (gt / NST) & 1, p.wait_limit)) lost();
        };
        const auto do_k = [&](int gt) {
            landed(gt);
            const uint32_t st = sST + (gt % NST) * C::TILE + (L >> 6) * C::REC + (L & 63) * 16;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int u = gt * NC + c;
                fill(u, u & 1, [&](int j) { return st + (c * 4 + j) * 1024; }, C::KU, true);
            }
            if (lane == 0) mbar_arrive(bar_empty + 8 * (gt % NST));
        };
        const auto do_v = [&](int gt) {
            landed(gt);
            const uint32_t st = sST + (gt % NST) * C::TILE + rec_v_off(D) + L * 16;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int u = gt * NC + c;
                // head_dim 64: lanes 64..127 have no channel; their rows of O are never read
                fill(u, 2 + (u & 1),
                     [&](int j) { return st + c * 2048 + (j >> 1) * C::REC + (j & 1) * 16 * D; }, 4, D > 64 || q4 < 2);
            }
            if (lane == 0) mbar_arrive(bar_empty + 8 * (gt % NST));
        };
        if constexpr (ND == 8) {
            for (int gt = 0; gt < n_all; ++gt) {
                if (kvq_aborted(flags)) break;
                if (dw < 4)
                    do_k(gt);
                else
                    do_v(gt);
            }
        } else {
            // one group: the next tile's K before this tile's V, so that S runs ahead
            do_k(0);
            for (int gt = 0; gt < n_all; ++gt) {
                if (kvq_aborted(flags)) break;
                if (gt + 1 < n_all) do_k(gt + 1);
                do_v(gt);
            }
        }
    } else {
        // ============================================================ softmax
        const int sw = warp - 2 - ND;
        const int q4 = warp & 3;
        const int r0 = (sw >> 2) * HR;      // first row of this warp
        const int kt = 32 * q4 + lane;      // key of the tile = tensor-memory lane
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const int ct = threadIdx.x - 32 * (2 + ND);

        // Queries of unit (b, h) as fp16, divided by one power of two per unit so
        // that the largest is in [1, 2) -- bf16's 8 bits survive down to 2^-17
        // of it, and below that the error is 2^-25 of it --, and each
        // row's sum of what was stored.  Returns the power of two.
        const auto stage_q = [&](int b, int h) -> float {
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q);
            constexpr int VPR = D / 8;  // 16-byte vectors per row: 8, 16 or 32 lanes
            const auto row_vec = [&](int r, int v) {
                const int i = r / p.group, hh = r - i * p.group;
                const int64_t row = ((int64_t)b * p.n_q + i) * p.n_q_heads + h * p.group + hh;
                return __ldg(reinterpret_cast<const uint4 *>(q + row * D) + v);
            };
            uint32_t top = 0;  // largest magnitude's bits, infinities and NaN left out
            for (int idx = ct; idx < p.rows * VPR; idx += 32 * NSW) {
                const uint4 x = row_vec(idx / VPR, idx % VPR);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
                    if (lo < 0x7f80u) top = max(top, lo);
                    if (hi < 0x7f80u) top = max(top, hi);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) flags[40 + sw] = (int)top;
            named_bar_sync(1, 32 * NSW);  // also: every warp is done with the previous part's rows
#pragma unroll
            for (int w = 0; w < NSW; ++w) top = max(top, (uint32_t)flags[40 + w]);
            if (ct < NR) s_m[ct] = kKvqFloor;
            const int ex = top == 0 ? 0 : min(120, max(-120, (int)(top >> 7) - 127));
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            for (int idx = ct; idx < NR * VPR; idx += 32 * NSW) {
                const int r = idx / VPR, v = idx % VPR;
                uint4 val = make_uint4(0u, 0u, 0u, 0u);
                float sum = 0.f;
                if (r < p.rows) {
                    const uint4 x = row_vec(r, v);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __half2 hv = __floats2half2_rn(__uint_as_float(w[k] << 16) * down,
                                                             __uint_as_float(w[k] & 0xffff0000u) * down);
                        const float2 f = __half22float2(hv);
                        sum += f.x + f.y;
                        o[k] = *reinterpret_cast<const uint32_t *>(&hv);
                    }
                    val = make_uint4(o[0], o[1], o[2], o[3]);
                }
                st_shared_v4(sQ + (v >> 3) * C::Q_REGION + swz128(r, v & 7), val);
#pragma unroll
                for (int o = VPR / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (v == 0) s_zq[r] = sum;
            }
            fence_proxy_async_smem();
            named_bar_sync(1, 32 * NSW);  // sums and maxima visible
            if (lane == 0) mbar_arrive(bar_qfull);
            return __uint_as_float((uint32_t)(127 + ex) << 23);
        };

        int b = 0, h = 0, t0 = 0, n = 0, g = 0;
        bool have = walk.next(p.c, b, h, t0, n);
        float f = have ? stage_q(b, h) * p.scale_log2 : 0.f;
        while (have) {
            const int64_t len = kvq_len(p.c, b);
            const int64_t k_begin = (int64_t)t0 * TK;
            const int64_t k_end = min(k_begin + (int64_t)n * TK, len);
            const int64_t qpos0 = len - p.n_q;
            int nb = 0, nh = 0, nt0 = 0, nn = 0;
            const bool have_next = walk.next(p.c, nb, nh, nt0, nn);

            float l_run[HR], z_run[HR];  // sums of P' / s_V and P' z_V / s_V
#pragma unroll
            for (int i = 0; i < HR; ++i) {
                l_run[i] = 0.f;
                z_run[i] = 0.f;
            }
            for (int t = 0; t < n; ++t) {
                const int gt = g + t, stage = gt % NST;
                const int64_t key0 = k_begin + (int64_t)t * TK;
                const int64_t kabs = key0 + kt;
                const bool key_ok = kabs < k_end;

                // this key's scales and zeros
                if (!flags[0] && !mbar_wait_bounded(bar_full + 8 * stage, (gt / NST) & 1, p.wait_limit)) lost();
                const uint32_t rec = sST + stage * C::TILE + (kt >> 6) * C::REC + (kt & 63) * 4;
                const uint32_t ksz = ld_shared_u32(rec + rec_ks_off(D)), vsz = ld_shared_u32(rec + rec_vs_off(D));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_empty + 8 * stage);
                const float ks = __uint_as_float(ksz << 16), kz = __uint_as_float(ksz & 0xffff0000u);
                const float vs = __uint_as_float(vsz << 16), vz = __uint_as_float(vsz & 0xffff0000u);
                // Scale 0 (constant values, codes 0): a stand-in that keeps z / s in
                // range.  At least 2^-90, which keeps the sums of P' / s below fp32's
                // largest: values are off by 15 x 2^-90 where a scale is smaller.
                const float se = fmaxf(vs > 0.f ? vs : fabsf(vz) * 0.00390625f, 8.0779357e-28f);
                float inv = 1.f / se, zr = vz * inv;
                const bool bad = !(fabsf(ks) < CUDART_INF_F && fabsf(kz) < CUDART_INF_F && vs >= 0.f &&
                                   vs < CUDART_INF_F && fabsf(zr) < CUDART_INF_F);
                // not finite: NaN in the logit reaches every row that sees this key, and only those
                const float ls = bad ? CUDART_NAN_F : lg2(se);
                const float a = ks * f * 16777216.f, bz = kz * f;
                if (bad || !key_ok) inv = zr = 0.f;  // a weight of 0 times these is 0

                if (!flags[0] && !mbar_wait_bounded(bar_sfull + 8 * (gt & 1), (gt >> 1) & 1, p.wait_limit)) lost();
                const bool live = !kvq_aborted(flags);
                tc::fence_after_sync();
                float s[HR];
#pragma unroll
                for (int i = 0; i < HR; ++i) s[i] = 0.f;
                if (live) {
#pragma unroll
                    for (int c = 0; c < HR / 8; ++c)
                        tc::ld_32x32b_x8(tmem + lane_off + C::S_COL + (gt & 1) * NR + r0 + 8 * c, s + 8 * c);
                    tc::wait_ld();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_sfree + 8 * (gt & 1));

                const bool masked = key0 + TK > k_end || key0 + TK - 1 > qpos0;
                const int64_t rel = qpos0 - kabs;  // row r sees the key iff rel + r / group >= 0
                bool need = false;
#pragma unroll
                for (int i = 0; i < HR; i += 4) {
                    const float4 zq = *reinterpret_cast<const float4 *>(s_zq + r0 + i);
                    s[i] = fmaf(s[i], a, fmaf(zq.x, bz, ls));
                    s[i + 1] = fmaf(s[i + 1], a, fmaf(zq.y, bz, ls));
                    s[i + 2] = fmaf(s[i + 2], a, fmaf(zq.z, bz, ls));
                    s[i + 3] = fmaf(s[i + 3], a, fmaf(zq.w, bz, ls));
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < HR; ++i)
                        if (!(key_ok && rel + (r0 + i) / p.group >= 0)) s[i] = -CUDART_INF_F;
                }
#pragma unroll
                for (int i = 0; i < HR; i += 4) {
                    const float4 m4 = *reinterpret_cast<const float4 *>(s_m + r0 + i);
                    need |= s[i] - m4.x > kKvqOff + kKvqRaise || s[i + 1] - m4.y > kKvqOff + kKvqRaise ||
                            s[i + 2] - m4.z > kKvqOff + kKvqRaise || s[i + 3] - m4.w > kKvqOff + kKvqRaise;
                }
                const unsigned any = __ballot_sync(0xffffffffu, need);
                if (lane == 0) flags[8 + 16 * (gt & 1) + sw] = any != 0u;
                named_bar_sync(1, 32 * NSW);
                int votes = 0;
#pragma unroll
                for (int w = 0; w < NSW; ++w) votes |= flags[8 + 16 * (gt & 1) + w];
                bool o_stable = t == 0;  // the previous part's epilogue waited for its last P.V
                if (votes) {
#pragma unroll
                    for (int i = 0; i < HR; ++i) {
                        float mx = s[i];
#pragma unroll
                        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        if (lane == 0) red[NR * q4 + r0 + i] = mx;
                    }
                    named_bar_sync(1, 32 * NSW);
                    float alpha[HR];
#pragma unroll
                    for (int i = 0; i < HR; ++i) {
                        const int r = r0 + i;
                        const float top = fmaxf(fmaxf(red[r], red[NR + r]), fmaxf(red[2 * NR + r], red[3 * NR + r]));
                        const float m_old = s_m[r], m_new = fmaxf(m_old, top - kKvqOff);
                        alpha[i] = ex2(m_old - m_new);
                        l_run[i] *= alpha[i];
                        z_run[i] *= alpha[i];
                    }
                    named_bar_sync(1, 32 * NSW);  // every warp has read the old maxima
                    if (ct < NR)
                        s_m[ct] = fmaxf(s_m[ct], fmaxf(fmaxf(red[ct], red[NR + ct]),
                                                       fmaxf(red[2 * NR + ct], red[3 * NR + ct])) - kKvqOff);
                    named_bar_sync(1, 32 * NSW);
                    if (t > 0) {
                        // O holds this part's tiles so far at the old maximum
                        if (!flags[0] &&
                            !mbar_wait_bounded(bar_odone + 8 * ((gt - 1) & 1), ((gt - 1) >> 1) & 1, p.wait_limit))
                            lost();
                        o_stable = true;
                        tc::fence_after_sync();
                        if (!kvq_aborted(flags)) {
#pragma unroll
                            for (int c = 0; c < NC; ++c)
#pragma unroll
                                for (int j = 0; j < HR / 8; ++j) {
                                    const uint32_t at = tmem + lane_off + C::O_COL + c * NR + r0 + 8 * j;
                                    float v8[8];
                                    tc::ld_32x32b_x8(at, v8);
                                    tc::wait_ld();
#pragma unroll
                                    for (int i = 0; i < 8; ++i) v8[i] *= alpha[8 * j + i];
                                    tc::st_32x32b_x8(at, v8);
                                }
                            tc::wait_st();
                        }
                    }
                }

                uint32_t pw[HR / 2];
#pragma unroll
                for (int i = 0; i < HR; i += 2) {
                    const float2 m2 = *reinterpret_cast<const float2 *>(s_m + r0 + i);
                    const __half2 hv = __floats2half2_rn(ex2(s[i] - m2.x), ex2(s[i + 1] - m2.y));
                    const float2 r = __half22float2(hv);
                    l_run[i] = fmaf(r.x, inv, l_run[i]);
                    l_run[i + 1] = fmaf(r.y, inv, l_run[i + 1]);
                    z_run[i] = fmaf(r.x, zr, z_run[i]);
                    z_run[i + 1] = fmaf(r.y, zr, z_run[i + 1]);
                    pw[i / 2] = *reinterpret_cast<const uint32_t *>(&hv);
                }
                // this P buffer was last read by P.V of tile gt - 2
                if (gt >= 2 && !o_stable && !flags[0] &&
                    !mbar_wait_bounded(bar_odone + 8 * (gt & 1), ((gt - 2) >> 1) & 1, p.wait_limit))
                    lost();
                const uint32_t pt = sPT + (gt & 1) * C::PT_BYTES;
#pragma unroll
                for (int j = 0; j < HR / 8; ++j) {
                    const int chunk = r0 / 8 + j;
                    const uint32_t phys = C::PT_ROW == 128 ? (uint32_t)(chunk ^ (kt & 7))
                                          : C::PT_ROW == 64 ? (uint32_t)(chunk ^ ((kt >> 1) & 3))
                                                            : (uint32_t)(chunk ^ ((kt >> 2) & 1));
                    st_shared_v4(pt + (uint32_t)kt * C::PT_ROW + (phys << 4),
                                 make_uint4(pw[4 * j], pw[4 * j + 1], pw[4 * j + 2], pw[4 * j + 3]));
                }
                fence_proxy_async_smem();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pfull + 8 * (gt & 1));
            }

            // ---- the part's result: this thread owns tensor-memory lane kt of every O block
            const int g_last = g + n - 1;
            if (!flags[0] && !mbar_wait_bounded(bar_odone + 8 * (g_last & 1), (g_last >> 1) & 1, p.wait_limit)) lost();
            tc::fence_after_sync();
            const bool have_o = !kvq_aborted(flags);
            named_bar_sync(1, 32 * NSW);
#pragma unroll
            for (int i = 0; i < HR; ++i) {
                float l = l_run[i], z = z_run[i];
#pragma unroll
                for (int o = 16; o; o >>= 1) {
                    l += __shfl_xor_sync(0xffffffffu, l, o);
                    z += __shfl_xor_sync(0xffffffffu, z, o);
                }
                if (lane == 0) {
                    red[NR * q4 + r0 + i] = l;
                    red[4 * NR + NR * q4 + r0 + i] = z;
                }
            }
            named_bar_sync(1, 32 * NSW);
            const int64_t part = (int64_t)blockIdx.x + (int64_t)b * p.c.n_kv_heads + h;
#pragma unroll
            for (int j = 0; j < HR / 8; ++j) {
                float l8[8], z8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *rl = red + r0 + 8 * j + i, *rz = rl + 4 * NR;
                    l8[i] = have_o ? (rl[0] + rl[NR]) + (rl[2 * NR] + rl[3 * NR]) : 0.f;
                    z8[i] = (rz[0] + rz[NR]) + (rz[2 * NR] + rz[3 * NR]);
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    float o8[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o8[i] = 0.f;
                    if (have_o) {
                        tc::ld_32x32b_x8(tmem + lane_off + C::O_COL + c * NR + r0 + 8 * j, o8);
                        tc::wait_ld();
                    }
                    const int d = c * 128 + kt;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = r0 + 8 * j + i;
                        if (r >= p.rows || (D == 64 && d >= 64)) continue;
                        p.o_part[(part * p.rows + r) * D + d] =
                            l8[i] == 0.f ? 0.f : fmaf(o8[i], 16777216.f, z8[i]) / l8[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + 8 * j + i;
                    if (r < p.rows && kt == r)
                        p.lse_part[part * p.rows + r] = l8[i] == 0.f ? -CUDART_INF_F : s_m[r] + lg2(l8[i]);
                }
            }
            // O has been read (wait_ld) before this warp's next pfull arrival, which gates the next part's first P.V
            tc::fence_before_sync();
            // The last S of the part was read above, so its queries are free: every S that used them is complete.
            if (have_next) f = stage_q(nb, nh) * p.scale_log2;
            g += n;
            have = have_next;
            b = nb;
            h = nh;
            t0 = nt0;
            n = nn;
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int D, int NR>
cudaError_t launch_kvq_attn_nr(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    constexpr int smem = KvqCfg<D, NR>::TOTAL;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kvq_attn_kernel<D, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_pdl(kvq_attn_kernel<D, NR>, dim3(n_cta), dim3(KvqCfg<D, NR>::THREADS), smem, stream, p);
}

template <int D>
cudaError_t launch_kvq_attn_d(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    switch ((p.rows + 15) / 16) {
        case 1: return launch_kvq_attn_nr<D, 16>(p, n_cta, stream);
        case 2: return launch_kvq_attn_nr<D, 32>(p, n_cta, stream);
        case 3: return launch_kvq_attn_nr<D, 48>(p, n_cta, stream);
        case 4: return launch_kvq_attn_nr<D, 64>(p, n_cta, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace wm
