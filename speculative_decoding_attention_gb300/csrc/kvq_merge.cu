// kvq_merge.cu -- merge of the parts of the attention over the 4-bit KV cache.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace wm {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Merge of the parts of one output row: out = sum_s 2^(lse_s - lse) o_s.  A thread holds 4
// columns of a row; PG threads share them, each folding every PG-th part in batches whose
// loads are in flight together.  A part without a visible key (-inf) is skipped; a NaN
// stays one.
constexpr int kMergeThreads = 128, kBatch = 4;

template <int PG>
__global__ void __launch_bounds__(kMergeThreads) kvq_merge_kernel(const KvqAttnParams p) {
    constexpr int CT = kMergeThreads / PG;
    __shared__ float m_s[PG][CT], z_s[PG][CT];
    __shared__ float4 acc_s[PG][CT];
    pdl_wait();
    pdl_launch_dependents();
    const int D = p.c.head_dim;
    const int ct = threadIdx.x % CT, pg = threadIdx.x / CT;
    // four columns of the D / 4 (a power of two) of a row; rows x D / 4 is below 2^29
    const int item = (int)blockIdx.x * CT + ct, quads = __ffs(D / 4) - 1;
    const int r = item >> quads, col = (item & (D / 4 - 1)) * 4;
    const bool live = r < p.c.batch * p.n_q * p.n_q_heads;
    const int per_b = p.n_q * p.n_q_heads;
    const int b = r / per_b, rem = r - b * per_b, qi = rem / p.n_q_heads, head = rem - qi * p.n_q_heads;
    const int h = head / p.group, ru = qi * p.group + head - h * p.group;
    const int chunk = p.sched[0], before = live ? p.sched[1 + b] : 0, nt = live ? p.sched[2 + b] - before : 0;
    int64_t s_first = 0;
    int n_parts = 0;
    if (live && nt > 0) {
        const int first = before * p.c.n_kv_heads + h * nt;
        const int c0 = first / chunk, c1 = (first + nt - 1) / chunk;
        n_parts = c1 - c0 + 1;
        s_first = c0 + (int64_t)b * p.c.n_kv_heads + h;
    }
    const float *ls = p.lse_part + s_first * p.rows + ru;
    const float *op = p.o_part + (s_first * p.rows + ru) * D + col;
    const int64_t o_stride = (int64_t)p.rows * D;
    float m = -CUDART_INF_F, z = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = pg; s0 < n_parts; s0 += kBatch * PG) {
        float l[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int s = s0 + j * PG;
            l[j] = -CUDART_INF_F;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s < n_parts) {
                l[j] = __ldg(ls + (int64_t)s * p.rows);
                v[j] = __ldg(reinterpret_cast<const float4 *>(op + s * o_stride));
            }
        }
        float mb = m;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mb = fmaxf(mb, l[j]);
        const float base = mb == -CUDART_INF_F ? 0.f : mb;
        const float keep = ex2(m - base);
        z *= keep;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (l[j] == -CUDART_INF_F) continue;
            const float w = ex2(l[j] - base);
            z += w;
            acc.x += w * v[j].x;
            acc.y += w * v[j].y;
            acc.z += w * v[j].z;
            acc.w += w * v[j].w;
        }
        m = mb;
    }
    m_s[pg][ct] = m;
    z_s[pg][ct] = z;
    acc_s[pg][ct] = acc;
    __syncthreads();
    if (pg != 0 || !live) return;
    float mt = -CUDART_INF_F;
#pragma unroll
    for (int g = 0; g < PG; ++g) mt = fmaxf(mt, m_s[g][ct]);
    const float base = mt == -CUDART_INF_F ? 0.f : mt;
    float zt = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < PG; ++g) {
        const float c = ex2(m_s[g][ct] - base);  // 0 for a group without a part
        const float4 u = acc_s[g][ct];
        zt += c * z_s[g][ct];
        t.x += c * u.x;
        t.y += c * u.y;
        t.z += c * u.z;
        t.w += c * u.w;
    }
    const float inv = zt == 0.f ? 0.f : 1.f / zt;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(t.x * inv, t.y * inv);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(t.z * inv, t.w * inv);
    uint2 pk;
    pk.x = *reinterpret_cast<const uint32_t *>(&lo);
    pk.y = *reinterpret_cast<const uint32_t *>(&hi);
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + (int64_t)r * D + col) = pk;
    if (col == 0 && p.lse) p.lse[r] = zt == 0.f ? -CUDART_INF_F : (mt + lg2(zt)) * kLn2;
}

}  // namespace

cudaError_t launch_kvq_merge(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    const int64_t items = (int64_t)p.c.batch * p.n_q * p.n_q_heads * (p.c.head_dim / 4);
    const auto grid = [&](int pg) { return dim3((unsigned)((items * pg + kMergeThreads - 1) / kMergeThreads)); };
    // Sixteen threads share a row's parts where there are many, four where a unit has few on
    // average.  Whole calls in us with four and with sixteen: 52 short sequences, 2496 rows of 256
    // from 208 units, 35.6 and 53.6; 2 x 1M, 640 rows of 128 from 16 units, 670 and 674; 128K, 128
    // rows from 4 units, 36.4 and 35.3.
    if ((int64_t)p.c.batch * p.c.n_kv_heads * 16 > n_cta)
        return launch_pdl(kvq_merge_kernel<4>, grid(4), dim3(kMergeThreads), 0, stream, p);
    return launch_pdl(kvq_merge_kernel<16>, grid(16), dim3(kMergeThreads), 0, stream, p);
}

}  // namespace wm
