// kvq_merge.cu -- merge of the parts of the attention over the 4-bit KV cache.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace wm {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Merge of the parts of one output row: out = sum_s 2^(lse_s - lse) o_s.  One CTA
// per (row, 32 columns): 8 column threads x 16 part groups, each group folding
// every 16th part in batches whose loads are in flight together.  A part
// without a visible key (-inf) is skipped; a NaN stays one.
constexpr int kColThreads = 8, kPartGroups = 16, kBatch = 4;

__global__ void __launch_bounds__(kColThreads *kPartGroups) kvq_merge_kernel(const KvqAttnParams p) {
    __shared__ float m_s[kPartGroups][kColThreads], z_s[kPartGroups][kColThreads];
    __shared__ float4 acc_s[kPartGroups][kColThreads];
    pdl_wait();
    pdl_launch_dependents();
    const int D = p.c.head_dim;
    const int r = blockIdx.x;
    const int ct = threadIdx.x % kColThreads, pg = threadIdx.x / kColThreads;
    const int col = ((int)blockIdx.y * kColThreads + ct) * 4;
    const int per_b = p.n_q * p.n_q_heads;
    const int b = r / per_b, rem = r - b * per_b, qi = rem / p.n_q_heads, head = rem - qi * p.n_q_heads;
    const int h = head / p.group, ru = qi * p.group + head - h * p.group;
    const int chunk = p.sched[0], before = p.sched[1 + b], nt = p.sched[2 + b] - before;
    int64_t s_first = 0;
    int n_parts = 0;
    if (nt > 0) {
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
    for (int s0 = pg; s0 < n_parts; s0 += kBatch * kPartGroups) {
        float l[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int s = s0 + j * kPartGroups;
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
    if (pg != 0) return;
    float mt = -CUDART_INF_F;
#pragma unroll
    for (int g = 0; g < kPartGroups; ++g) mt = fmaxf(mt, m_s[g][ct]);
    const float base = mt == -CUDART_INF_F ? 0.f : mt;
    float zt = 0.f;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kPartGroups; ++g) {
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
    if (blockIdx.y == 0 && ct == 0 && p.lse) p.lse[r] = zt == 0.f ? -CUDART_INF_F : (mt + lg2(zt)) * kLn2;
}

}  // namespace

cudaError_t launch_kvq_merge(const KvqAttnParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.c.batch * p.n_q * p.n_q_heads), (unsigned)(p.c.head_dim / (4 * kColThreads)));
    return launch_pdl(kvq_merge_kernel, grid, dim3(kColThreads * kPartGroups), 0, stream, p);
}

}  // namespace wm
