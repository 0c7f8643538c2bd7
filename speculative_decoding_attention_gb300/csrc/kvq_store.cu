// kvq_store.cu -- writing to and reading from the 4-bit KV cache.
//
// Per token and KV head, K and V alike, over the D channels of a row x:
//   z = min x,  s = bf16((max x - z) / 15),  c = clamp(rint((x - z) / s), 0, 15),
// codes 0 if s = 0; the value held is s c + z.  z is a value of x, so bf16 holds
// it exactly.  s is rounded to bf16: it is off by at most 2^-9 of itself, so the
// held values move by at most 15 s 2^-9, a thirty-fourth of a code's step, and
// the range still fits (c is clamped).  A row with a NaN or an infinity gets
// s = z = NaN: whoever attends to it sees NaN, as with a bf16 cache.
//
// Codes and scales are those of the definition in 64 bits, bit for bit: both
// are computed in fp32, and where that lands next to a rounding border (where
// its error could choose the other side) the row or the element is recomputed
// in doubles.  At D = 128 that is 0.2% of the rows; doubles for every element would cost
// far more than the memory traffic (this GPU has 2 FP64 units per SM).
//
// One CTA handles one record (64 positions of one KV head).  A warp quantises a
// row; K's words go to a shared image of the record's K area, V's codes to a byte
// matrix that is read back by columns (the cache holds V transposed).  The
// image then leaves in 16-byte units; a V unit of which the append covers only
// some positions is read, merged and written back, so the other positions of
// the record keep their codes.  One CTA owns a record, so no two write one unit.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace wm {

namespace {

constexpr float kBorder = 1.f / 131072.f;  // 2^-17: over twice the fp32 error of (x - z) / s <= 15.1 (three roundings)

__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// bf16 of (hi - lo) / 15, the quotient as in 64 bits.  The fp32 quotient is
// within 1.5 of its last places; only one that close to the middle of two
// bf16 values (or too small for fp32's full precision) is taken again in doubles.
// The double is rounded to bf16 once: through fp32 rounded to odd.
__device__ float row_scale(float lo, float hi) {
    const float s = (hi - lo) / 15.f;
    const uint32_t low = __float_as_uint(s) & 0xffffu;
    if (isfinite(s) && s > 1e-30f && (low < 0x7ffcu || low > 0x8004u)) return __bfloat162float(__float2bfloat16_rn(s));
    const double d = ((double)hi - (double)lo) / 15.0;
    float t = __double2float_rz(d);
    if ((double)t != d) t = __uint_as_float(__float_as_uint(t) | 1u);
    return __bfloat162float(__float2bfloat16_rn(t));
}

// Codes of one warp's row, NE consecutive channels per lane; also its scale and zero.
template <int NE>
__device__ __forceinline__ void quantise_row(const float (&x)[NE], uint32_t (&c)[NE], float &s, float &z) {
    float lo = x[0], hi = x[0];
    bool odd = false;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        odd |= !isfinite(x[i]);
    }
    lo = warp_min(lo);
    hi = warp_max(hi);
    if (__any_sync(0xffffffffu, odd)) {
        s = z = CUDART_NAN_F;
#pragma unroll
        for (int i = 0; i < NE; ++i) c[i] = 0u;
        return;
    }
    z = lo;
    s = row_scale(lo, hi);
    if (!(s > 0.f)) {
#pragma unroll
        for (int i = 0; i < NE; ++i) c[i] = 0u;
        return;
    }
    const float rs = 1.f / s;
    bool near = !(s > 1e-30f && s < 1e30f);  // outside: quotients in doubles
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const float y = (x[i] - z) * rs;
        const float r = rintf(y);
        near |= fabsf(y - r) > 0.5f - kBorder;
        c[i] = (uint32_t)fminf(fmaxf(r, 0.f), 15.f);
    }
    if (near) {
#pragma unroll 1
        for (int i = 0; i < NE; ++i)
            c[i] = (uint32_t)fmin(fmax(rint(((double)x[i] - (double)z) / (double)s), 0.0), 15.0);
    }
}

template <int NE>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, int lane, float (&x)[NE]) {
    uint32_t w[NE / 2];
    if constexpr (NE == 2) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p) + lane);
    } else if constexpr (NE == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p) + lane);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + lane);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack_sz(float s, float z) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(s, z);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Bit position of element e in its word.
__host__ __device__ constexpr int nib_bit(int e) { return 4 * ((e & 7) / 2 + 4 * (e & 1)); }

template <int D>
__global__ void kvq_append_kernel(const KvqView c, const __nv_bfloat16 *__restrict__ kn,
                                  const __nv_bfloat16 *__restrict__ vn, int n_new, int32_t *__restrict__ err) {
    constexpr int NE = D / 32;
    __shared__ __align__(16) uint32_t s_k[8 * D];         // K area image: [D / 32][64][4 words]
    __shared__ __align__(16) uint8_t s_v[kRecKeys * D];   // V codes: [64][D]
    __shared__ uint32_t s_sz[2][kRecKeys];
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y / c.n_kv_heads, h = blockIdx.y - b * c.n_kv_heads;
    const int64_t len = c.seq_lens[b];
    if (len < 0 || len > c.capacity) {  // nothing is written for a length that cannot be
        if (threadIdx.x == 0 && blockIdx.x == 0) kvq_report(err, WM_DEVERR_BAD_LENGTH);
        return;
    }
    const int64_t pos0 = len - n_new;  // position of new token 0 (tokens before position 0 are padding)
    const int64_t first = pos0 > 0 ? pos0 : 0;
    const int64_t blk = first / kRecKeys + blockIdx.x;
    if (blk * kRecKeys >= len) return;
    const int r0 = (int)max(first - blk * kRecKeys, (int64_t)0);
    const int r1 = (int)min(len - blk * kRecKeys, (int64_t)kRecKeys);
    uint8_t *rec = kvq_record(c, b, h, blk);
    if (!rec) {
        if (threadIdx.x == 0) kvq_report(err, WM_DEVERR_BAD_PAGE);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
    for (int t = warp; t < 2 * (r1 - r0); t += n_warps) {
        const bool is_v = t & 1;
        const int r = r0 + (t >> 1);
        const int64_t tok = blk * kRecKeys + r - pos0;
        const __nv_bfloat16 *src =
            (is_v ? vn : kn) + (((int64_t)b * n_new + tok) * c.n_kv_heads + h) * D;
        float x[NE];
        load_row<NE>(src, lane, x);
        uint32_t code[NE];
        float s, z;
        quantise_row<NE>(x, code, s, z);
        if (lane == 0) s_sz[is_v][r] = pack_sz(s, z);
        if (is_v) {
            uint8_t *dst = s_v + r * D + lane * NE;
            if constexpr (NE == 2) {
                *reinterpret_cast<uint16_t *>(dst) = (uint16_t)(code[0] | (code[1] << 8));
            } else {
#pragma unroll
                for (int i = 0; i < NE; i += 4)
                    *reinterpret_cast<uint32_t *>(dst + i) =
                        code[i] | (code[i + 1] << 8) | (code[i + 2] << 16) | (code[i + 3] << 24);
            }
        } else {
            // this lane's part of a word, joined with the neighbours that share it
            uint32_t w = 0u;
#pragma unroll
            for (int i = 0; i < NE; ++i) w |= code[i] << nib_bit((lane * NE + i) & 7);
            if constexpr (NE == 2) w |= __shfl_xor_sync(0xffffffffu, w, 2);
            if constexpr (NE <= 4) w |= __shfl_xor_sync(0xffffffffu, w, 1);
            const int word = lane * NE / 8;  // of the row's D / 8
            if (lane * NE % 8 == 0) s_k[(word >> 2) * 256 + r * 4 + (word & 3)] = w;
        }
    }
    __syncthreads();
    // K units of the covered positions
    for (int i = threadIdx.x; i < (D / 32) * (r1 - r0); i += blockDim.x) {
        const int j = i / (r1 - r0), u = j * kRecKeys + r0 + (i - j * (r1 - r0));
        reinterpret_cast<uint4 *>(rec)[u] = reinterpret_cast<const uint4 *>(s_k)[u];
    }
    // V units: 32 positions of one channel
    for (int u = threadIdx.x; u < 2 * D; u += blockDim.x) {
        const int half = u / D, ch = u - half * D;
        const int a0 = max(r0 - 32 * half, 0), a1 = min(r1 - 32 * half, 32);
        if (a0 >= a1) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(rec + rec_v_off(D)) + u;
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (a0 > 0 || a1 < 32) {
            const uint4 old = *dst;
            w[0] = old.x;
            w[1] = old.y;
            w[2] = old.z;
            w[3] = old.w;
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e >= a0 && e < a1) {
                    const int bit = nib_bit(e);
                    w[e >> 3] = (w[e >> 3] & ~(15u << bit)) | ((uint32_t)s_v[(32 * half + e) * D + ch] << bit);
                }
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e >> 3] |= (uint32_t)s_v[(32 * half + e) * D + ch] << nib_bit(e);
        }
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
    }
    for (int i = threadIdx.x; i < 2 * kRecKeys; i += blockDim.x) {
        const int is_v = i / kRecKeys, r = i - is_v * kRecKeys;
        if (r >= r0 && r < r1)
            reinterpret_cast<uint32_t *>(rec + (is_v ? rec_vs_off(D) : rec_ks_off(D)))[r] = s_sz[is_v][r];
    }
}

// Two values s c + z as bf16 (one rounding: the fp32 product of an 8-bit and a
// 4-bit significand is exact, the sum is rounded to fp32 and then to bf16 -- off
// by at most half a bf16 step and 2^-24).
__device__ __forceinline__ uint32_t held_pair(uint32_t c0, float s0, float z0, uint32_t c1, float s1, float z1) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(fmaf((float)c0, s0, z0), fmaf((float)c1, s1, z1));
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void unpack_sz(uint32_t w, float &s, float &z) {
    s = __uint_as_float(w << 16);
    z = __uint_as_float(w & 0xffff0000u);
}

// The last n positions as bf16 [B][n][Hkv][D]; rows before position 0 are 0.
// One CTA per record; K: a thread turns one word into 8 channels of a row; V:
// a thread turns one unit pair (two channels, 32 positions) into 32 stores of a
// channel pair, so a warp's store covers 128 consecutive bytes of a row.
template <int D>
__global__ void __launch_bounds__(128)
    kvq_read_kernel(const KvqView c, int n, __nv_bfloat16 *__restrict__ ko, __nv_bfloat16 *__restrict__ vo,
                    int32_t *__restrict__ err) {
    __shared__ float s_s[2][kRecKeys], s_z[2][kRecKeys];
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y / c.n_kv_heads, h = blockIdx.y - b * c.n_kv_heads;
    const int64_t raw = c.seq_lens[b];
    const int64_t len = kvq_len(c, b);
    if (raw != len && threadIdx.x == 0 && blockIdx.x == 0) kvq_report(err, WM_DEVERR_BAD_LENGTH);
    const int64_t pos0 = len - n;  // may be negative: those rows are 0
    const int64_t first = pos0 >= 0 ? pos0 / kRecKeys : -((-pos0 + kRecKeys - 1) / kRecKeys);
    const int64_t blk = first + blockIdx.x;
    if (blk * kRecKeys >= len) return;
    const int r0 = (int)max(pos0 - blk * kRecKeys, (int64_t)0);
    const int r1 = (int)min(len - blk * kRecKeys, (int64_t)kRecKeys);
    const int64_t tok0 = blk * kRecKeys - pos0;  // output row of position 64 blk
    const auto out_row = [&](int r) { return (((int64_t)b * n + tok0 + r) * c.n_kv_heads + h) * D; };
    const uint8_t *rec = nullptr;
    if (blk >= 0) {
        rec = kvq_record(c, b, h, blk);
        if (!rec && threadIdx.x == 0) kvq_report(err, WM_DEVERR_BAD_PAGE);
    }
    if (!rec) {
        for (int i = threadIdx.x; i < (r1 - r0) * (D / 8); i += blockDim.x) {
            const int r = r0 + i / (D / 8), v = i - i / (D / 8) * (D / 8);
            reinterpret_cast<uint4 *>(ko + out_row(r))[v] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4 *>(vo + out_row(r))[v] = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    for (int i = threadIdx.x; i < 2 * kRecKeys; i += blockDim.x) {
        const int is_v = i / kRecKeys, r = i - is_v * kRecKeys;
        const uint32_t w = reinterpret_cast<const uint32_t *>(rec + (is_v ? rec_vs_off(D) : rec_ks_off(D)))[r];
        unpack_sz(w, s_s[is_v][r], s_z[is_v][r]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (r1 - r0) * (D / 8); i += blockDim.x) {
        const int r = r0 + i / (D / 8), wd = i - i / (D / 8) * (D / 8);
        const uint32_t w = reinterpret_cast<const uint32_t *>(rec)[(wd >> 2) * 256 + r * 4 + (wd & 3)];
        const float s = s_s[0][r], z = s_z[0][r];
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = held_pair((w >> nib_bit(2 * k)) & 15u, s, z, (w >> nib_bit(2 * k + 1)) & 15u, s, z);
        reinterpret_cast<uint4 *>(ko + out_row(r))[wd] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    const uint4 *vu = reinterpret_cast<const uint4 *>(rec + rec_v_off(D));
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
        const int half = i / (D / 2), ch = 2 * (i - half * (D / 2));
        if (32 * half >= r1 || 32 * half + 32 <= r0) continue;
        const uint4 ua = vu[half * D + ch], ub = vu[half * D + ch + 1];
        const uint32_t wa[4] = {ua.x, ua.y, ua.z, ua.w}, wb[4] = {ub.x, ub.y, ub.z, ub.w};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int r = 32 * half + e;
            if (r < r0 || r >= r1) continue;
            const float s = s_s[1][r], z = s_z[1][r];
            *reinterpret_cast<uint32_t *>(vo + out_row(r) + ch) = held_pair(
                (wa[e >> 3] >> nib_bit(e)) & 15u, s, z, (wb[e >> 3] >> nib_bit(e)) & 15u, s, z);
        }
    }
}

}  // namespace

cudaError_t launch_kvq_append(const KvqView &c, const void *k_new, const void *v_new, int n_new, int32_t *err,
                              cudaStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)n_new + kRecKeys - 2) / kRecKeys + 1), (unsigned)(c.batch * c.n_kv_heads));
    const int warps = n_new >= 8 ? 8 : n_new >= 2 ? 4 : 2;  // a warp per row, two rows per token, eight warps at most
    const auto *k = static_cast<const __nv_bfloat16 *>(k_new), *v = static_cast<const __nv_bfloat16 *>(v_new);
    const dim3 block(32 * warps);
    switch (c.head_dim) {
        case 64: return launch_pdl(kvq_append_kernel<64>, grid, block, 0, stream, c, k, v, n_new, err);
        case 128: return launch_pdl(kvq_append_kernel<128>, grid, block, 0, stream, c, k, v, n_new, err);
        case 256: return launch_pdl(kvq_append_kernel<256>, grid, block, 0, stream, c, k, v, n_new, err);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kvq_read(const KvqView &c, int n, void *k_out, void *v_out, int32_t *err, cudaStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)n + kRecKeys - 2) / kRecKeys + 1), (unsigned)(c.batch * c.n_kv_heads));
    auto *k = static_cast<__nv_bfloat16 *>(k_out), *v = static_cast<__nv_bfloat16 *>(v_out);
    switch (c.head_dim) {
        case 64: return launch_pdl(kvq_read_kernel<64>, grid, dim3(128), 0, stream, c, n, k, v, err);
        case 128: return launch_pdl(kvq_read_kernel<128>, grid, dim3(128), 0, stream, c, n, k, v, err);
        case 256: return launch_pdl(kvq_read_kernel<256>, grid, dim3(128), 0, stream, c, n, k, v, err);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace wm
