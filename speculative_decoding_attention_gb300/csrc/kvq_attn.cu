// kvq_attn.cu -- causal attention over the 4-bit KV cache: the attention grid
// and the merge of its parts.
//
// With l_j = q . (s_j c_j + z_j) = s_j (q . c_j) + z_j sum(q), the values of a key
// never have to be formed: the products run over the codes, and a key's scale and
// zero enter per (row, key).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace wm {

namespace {

constexpr float kLn2 = 0.6931471805599453f;

// One key per thread, rows one after the other.
template <int D>
__global__ void __launch_bounds__(128) kvq_attn_kernel(const KvqAttnParams p) {
    extern __shared__ float sm[];
    float *s_q = sm;                  // [rows][D]
    float *s_p = sm + p.rows * D;     // [rows][128]
    float *s_o = s_p + p.rows * 128;  // [rows][D]
    __shared__ int64_t s_warp[32];
    __shared__ int4 s_start;
    __shared__ float s_m[64], s_l[64], s_red[4];
    __shared__ float s_vs[128], s_vz[128];
    pdl_wait();
    pdl_launch_dependents();
    const int4 start = kvq_schedule(p, s_warp, &s_start);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    KvqWalk walk;
    walk.init(start);
    int b, h, t0, n;
    while (walk.next(p.c, b, h, t0, n)) {
        __syncthreads();
        const int64_t len = kvq_len(p.c, b);
        for (int i = tid; i < p.rows * D; i += 128) {
            const int r = i / D, d = i - r * D, qi = r / p.group, hh = r - qi * p.group;
            s_q[i] = __bfloat162float(static_cast<const __nv_bfloat16 *>(
                p.q)[(((int64_t)b * p.n_q + qi) * p.n_q_heads + h * p.group + hh) * D + d]);
            s_o[i] = 0.f;
        }
        for (int r = tid; r < p.rows; r += 128) {
            s_m[r] = -CUDART_INF_F;
            s_l[r] = 0.f;
        }
        for (int t = t0; t < t0 + n; ++t) {
            __syncthreads();
            const int64_t pos = (int64_t)t * kKvqTile + tid;
            const bool in = pos < len;
            const uint8_t *rec = in ? kvq_record(p.c, b, h, pos / kRecKeys) : nullptr;
            if (in && !rec) kvq_report(p.err, WM_DEVERR_BAD_PAGE);
            const int r64 = tid & 63;
            float ks = 0.f, kz = 0.f;
            if (rec) {
                const uint32_t a = reinterpret_cast<const uint32_t *>(rec + rec_ks_off(D))[r64];
                const uint32_t v = reinterpret_cast<const uint32_t *>(rec + rec_vs_off(D))[r64];
                ks = __uint_as_float(a << 16);
                kz = __uint_as_float(a & 0xffff0000u);
                s_vs[tid] = __uint_as_float(v << 16);
                s_vz[tid] = __uint_as_float(v & 0xffff0000u);
            }
            for (int r = 0; r < p.rows; ++r) {
                const bool ok = rec && pos <= len - p.n_q + r / p.group;
                float s = -CUDART_INF_F;
                if (ok) {
                    float dot = 0.f;
                    for (int w = 0; w < D / 8; ++w) {
                        const uint32_t x =
                            reinterpret_cast<const uint32_t *>(rec)[(w >> 2) * 256 + r64 * 4 + (w & 3)];
                        for (int e = 0; e < 8; ++e)
                            dot += s_q[r * D + 8 * w + e] *
                                   (ks * (float)((x >> (4 * (e / 2 + 4 * (e & 1)))) & 15u) + kz);
                    }
                    s = dot * p.scale_log2;
                }
                float mx = s;
                for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                __syncthreads();
                if (lane == 0) s_red[warp] = mx;
                __syncthreads();
                const float m_old = s_m[r];
                const float m = fmaxf(fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])), m_old);
                const float base = m == -CUDART_INF_F ? 0.f : m;
                const float e = ok ? ex2(s - base) : 0.f;
                float sum = e;
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                __syncthreads();
                if (lane == 0) s_red[warp] = sum;
                __syncthreads();
                s_p[r * 128 + tid] = e;
                const float keep = ex2(m_old - base);
                if (tid == 0) {
                    s_l[r] = s_l[r] * keep + s_red[0] + s_red[1] + s_red[2] + s_red[3];
                    s_m[r] = m;
                }
                for (int d = tid; d < D; d += 128) s_o[r * D + d] *= keep;
            }
            __syncthreads();
            for (int d = tid; d < D; d += 128)
                for (int j = 0; j < kKvqTile; ++j) {
                    const int64_t pj = (int64_t)t * kKvqTile + j;
                    if (pj >= len) break;
                    const uint8_t *rv = kvq_record(p.c, b, h, pj / kRecKeys);
                    if (!rv) continue;
                    const uint32_t x = reinterpret_cast<const uint32_t *>(
                        rv + rec_v_off(D))[((j & 63) / 32 * D + d) * 4 + (j & 31) / 8];
                    const float v = s_vs[j] * (float)((x >> (4 * ((j & 7) / 2 + 4 * (j & 1)))) & 15u) + s_vz[j];
                    for (int r = 0; r < p.rows; ++r) {
                        const float e = s_p[r * 128 + j];
                        if (e != 0.f) s_o[r * D + d] += e * v;
                    }
                }
        }
        __syncthreads();
        const int64_t part = (int64_t)blockIdx.x + (int64_t)b * p.c.n_kv_heads + h;
        for (int i = tid; i < p.rows * D; i += 128) {
            const float l = s_l[i / D];
            p.o_part[part * p.rows * D + i] = l == 0.f ? 0.f : s_o[i] / l;
        }
        for (int r = tid; r < p.rows; r += 128)
            p.lse_part[part * p.rows + r] = s_l[r] == 0.f ? -CUDART_INF_F : s_m[r] + lg2(s_l[r]);
    }
}

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
    const int64_t r = blockIdx.x;
    const int ct = threadIdx.x % kColThreads, pg = threadIdx.x / kColThreads;
    const int col = ((int)blockIdx.y * kColThreads + ct) * 4;
    const int64_t per_b = (int64_t)p.n_q * p.n_q_heads;
    const int b = (int)(r / per_b);
    const int rem = (int)(r - b * per_b), qi = rem / p.n_q_heads, head = rem - qi * p.n_q_heads;
    const int h = head / p.group, ru = qi * p.group + head - h * p.group;
    const int64_t chunk = p.sched[0], before = p.sched[1 + b], nt = p.sched[2 + b] - before;
    int64_t s_first = 0;
    int n_parts = 0;
    if (nt > 0) {
        const int64_t first = before * p.c.n_kv_heads + h * nt;
        const int64_t c0 = first / chunk, c1 = (first + nt - 1) / chunk;
        n_parts = (int)(c1 - c0 + 1);
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
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + r * D + col) = pk;
    if (blockIdx.y == 0 && ct == 0 && p.lse) p.lse[r] = zt == 0.f ? -CUDART_INF_F : (mt + lg2(zt)) * kLn2;
}

template <int D>
cudaError_t launch_d(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    const size_t smem = (size_t)p.rows * (2 * D + 128) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(kvq_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_attn_kernel<D>, dim3(n_cta), dim3(128), smem, stream, p);
}

}  // namespace

cudaError_t launch_kvq_attn(const KvqAttnParams &p, int n_cta, cudaStream_t stream) {
    switch (p.c.head_dim) {
        case 64: return launch_d<64>(p, n_cta, stream);
        case 128: return launch_d<128>(p, n_cta, stream);
        case 256: return launch_d<256>(p, n_cta, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kvq_merge(const KvqAttnParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)p.c.batch * p.n_q * p.n_q_heads), (unsigned)(p.c.head_dim / (4 * kColThreads)));
    return launch_pdl(kvq_merge_kernel, grid, dim3(kColThreads * kPartGroups), 0, stream, p);
}

}  // namespace wm
