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
// Codes and scales are those of the definition, bit for bit.  With t = x - z
// (rounded to fp32; exact unless x is below 2^-16 of z) the quotient t / s is taken
// in fp32 with one Newton step, so an exact tie -- common in bf16 data, one or two per
// hundred elements -- comes out as k + 1/2 exactly and rounds to even.  The code r is then
// right if |t - r s| <= s / 2, which one FMA gives exactly; else it is one off.  The
// scale is taken again in doubles where fp32 lands next to the middle of two bf16
// values.  (This GPU has 2 FP64 units per SM: doubles for every tie took
// three quarters of the time.)
//
// One CTA handles one record (64 positions of one KV head).  A lane holds 8 channels (one
// 16-byte load), D / 8 lanes a row, so a warp takes the K and V rows of 256 / D tokens at a
// time and rows side by side share the instructions per row (range, scale, reciprocal);
// even lanes do them for K, odd ones for V, and exchange the results.  Least and greatest
// run as one packed bf16 pair (min, -max).  K's words go to a shared image of the record's
// K area, V's codes to a byte matrix from which a thread takes 4 channels x 8 positions and
// transposes them into 4 words (the cache holds V transposed).  A V word of which the append
// covers only some positions is read, merged and written back, so the other
// positions of the record keep their codes.  One CTA owns a record, so no two
// write one word.
// A prompt of 32K tokens with 8 heads of 128: 51 us, where HBM would take 25 for its 170 MB;
// instructions bound it (76% of the issue slots; 168 for 16 channels of a lane).  With the
// row's work done by every lane it was 62, with a row per warp and fp32 ranges 94; with 4
// CTAs per SM, which need not spill, 4 us more than with 6.  Reading it back as bf16: 26 us,
// HBM's rate (38 with fp32 arithmetic and stores of 4 bytes, 33 with loads behind the
// barrier).  For a step's few tokens the launch is the time.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvq.cuh"
#include "launch.h"
#include "ptx.cuh"

namespace wm {

namespace {

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_sz(float s, float z) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(s, z);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Least value of this lane's 8 channels of a row and minus the greatest (exact), as a bf16 pair.
__device__ __forceinline__ uint32_t lane_range(const uint4 &in) {
    const uint32_t lo = min2_nan(min2_nan(in.x, in.y), min2_nan(in.z, in.w));
    const uint32_t hi = 0x80008000u ^ max2_nan(max2_nan(in.x, in.y), max2_nan(in.z, in.w));
    return min2_nan(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
}

// Scale and zero of a row from its range, and 1 / s.  s is bf16 of the range over 15, the
// quotient as in 64 bits: the fp32 product with 1 / 15 is within 3 of its last places, and
// only one that close to the middle of two bf16 values (or too small or large for
// that) is taken again in doubles, and rounded to bf16 once: through fp32 rounded to odd.
// A scale that the fp32 quotients are not for gets NaN as 1 / s.
__device__ __forceinline__ void row_scale(uint32_t range, uint32_t &sz, float &rs) {
    const float z = __uint_as_float(range << 16), top = -__uint_as_float(range & 0xffff0000u);
    float s = (top - z) * (1.f / 15.f);
    const uint32_t low = __float_as_uint(s) & 0xffffu;
    if (!(s > 1e-28f && s < 1e30f) || (low >= 0x7ff8u && low <= 0x8008u)) {
        if (!(top - top == 0.f && z - z == 0.f)) {  // a NaN or an infinity
            sz = pack_sz(CUDART_NAN_F, CUDART_NAN_F);
            rs = CUDART_NAN_F;
            return;
        }
        const double d = ((double)top - (double)z) / 15.0;
        s = __double2float_rz(d);
        if ((double)s != d) s = __uint_as_float(__float_as_uint(s) | 1u);
    }
    sz = pack_sz(s, z);
    s = __uint_as_float(sz << 16);
    rs = s > 1e-28f && s < 1e30f ? rcp(s) : CUDART_NAN_F;
}

// 1.5 x 2^23: added to a y below 2^22 it leaves y, rounded to even, in the low bits.
constexpr float kMagic = 12582912.f;
constexpr uint32_t kMagicBits = 0x4b400000u;

// Codes of 8 channels of a row, each code i as m[i] = kMagicBits + code.
__device__ __forceinline__ void row_codes(const uint4 &in, uint32_t sz, float rs, uint32_t (&m)[8]) {
    const uint32_t w[4] = {in.x, in.y, in.z, in.w};
    const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xffff0000u);
    const uint64_t nz2 = pack2(-z, -z), rs2 = pack2(rs, rs), ns2 = pack2(-s, -s);
    const uint64_t magic2 = pack2(kMagic, kMagic), unmagic2 = pack2(-kMagic, -kMagic);
    const float half = 0.5f * s;
    float worst = 0.f;  // largest |t - r s|
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t t2 = add2(pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), nz2);
        uint64_t y2 = mul2(t2, rs2);
        y2 = fma2(fma2(y2, ns2, t2), rs2, y2);
        const uint64_t m2 = add2(y2, magic2);
        float a, b, d, e;
        unpack2(m2, a, b);
        m[2 * i] = __float_as_uint(a);
        m[2 * i + 1] = __float_as_uint(b);
        unpack2(fma2(add2(m2, unmagic2), ns2, t2), d, e);
        worst = fmaxf(worst, fmaxf(fabsf(d), fabsf(e)));
    }
    if (worst > half || !(rs == rs)) {  // a code that may be one off, or quotients that are not for fp32
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) - z;
            if (rs == rs) {
                const float d = fmaf((float)(int)(m[i] - kMagicBits), -s, t);
                m[i] += d > half ? 1u : d < -half ? ~0u : 0u;
            } else {  // no range (s = 0) or not finite: 0; else the quotient in doubles
                m[i] = kMagicBits + (s > 0.f ? (uint32_t)fmin(fmax(rint((double)t / (double)s), 0.0), 15.0) : 0u);
            }
        }
    }
}

// Bit position of element e in its word.
__host__ __device__ constexpr int nib_bit(int e) { return 4 * ((e & 7) / 2 + 4 * (e & 1)); }

// Sum of m[i] 2^bit(i) less the kMagicBits in it, modulo 2^32: the codes at their bits.
__device__ __forceinline__ uint32_t pack_nibbles(const uint32_t (&m)[8]) {
    uint32_t sub = 0u, w = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) sub += kMagicBits << nib_bit(i);
    w -= sub;
#pragma unroll
    for (int i = 0; i < 8; ++i) w += m[i] << nib_bit(i);
    return w;
}
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    constexpr uint32_t sub = kMagicBits + (kMagicBits << 8) + (kMagicBits << 16) + (kMagicBits << 24);
    return a + (b << 8) + (c << 16) + (d << 24) - sub;
}

// 4 channels (bytes) of 8 positions a[0..7] into 4 words of 8 codes.
__device__ __forceinline__ void transpose_codes(const uint32_t (&a)[8], uint32_t (&w)[4]) {
    const uint32_t u0 = a[0] | (a[2] << 4), v0 = a[4] | (a[6] << 4);
    const uint32_t u1 = a[1] | (a[3] << 4), v1 = a[5] | (a[7] << 4);
    const uint32_t l0 = __byte_perm(u0, v0, 0x5140), h0 = __byte_perm(u0, v0, 0x7362);  // channels 0 1, 2 3
    const uint32_t l1 = __byte_perm(u1, v1, 0x5140), h1 = __byte_perm(u1, v1, 0x7362);
    w[0] = __byte_perm(l0, l1, 0x5410);
    w[1] = __byte_perm(l0, l1, 0x7632);
    w[2] = __byte_perm(h0, h1, 0x5410);
    w[3] = __byte_perm(h0, h1, 0x7632);
}

constexpr int kAppendWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kAppendWarps, 6)
    kvq_append_kernel(const KvqView c, const __nv_bfloat16 *__restrict__ kn, const __nv_bfloat16 *__restrict__ vn,
                      int n_new, int32_t *__restrict__ err) {
    constexpr int LANES = D / 8, ROWS = 32 / LANES;  // lanes per row, rows per warp
    constexpr int VS = D + 4;  // bytes per row of V codes: 8 rows down is 8 banks on
    __shared__ __align__(16) uint32_t s_k[8 * D];               // K area image: [D / 32][64][4 words]
    __shared__ __align__(16) uint8_t s_v[kRecKeys * VS];        // V codes: [64][D]
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
    const int64_t row0 = ((int64_t)b * n_new + blk * kRecKeys - pos0) * c.n_kv_heads + h;  // input row of record row 0
    const int word = lane % LANES;  // of the row's D / 8
    for (int rb = r0 + warp * ROWS; rb < r1; rb += n_warps * ROWS) {
        const int r = rb + lane / LANES;
        const bool valid = r < r1;
        uint4 xk = make_uint4(0u, 0u, 0u, 0u), xv = xk;
        if (valid) {
            const int64_t at = (row0 + (int64_t)r * c.n_kv_heads) * D;
            xk = __ldg(reinterpret_cast<const uint4 *>(kn + at) + word);
            xv = __ldg(reinterpret_cast<const uint4 *>(vn + at) + word);
        }
        // Even lanes reduce K's range and find its scale, odd lanes V's.
        const uint32_t rk = lane_range(xk), rv = lane_range(xv);
        const bool odd = lane & 1;
        uint32_t range = min2_nan(odd ? rv : rk, __shfl_xor_sync(0xffffffffu, odd ? rk : rv, 1));
#pragma unroll
        for (int o = LANES / 2; o > 1; o >>= 1) range = min2_nan(range, __shfl_xor_sync(0xffffffffu, range, o));
        uint32_t sz;
        float rs;
        row_scale(range, sz, rs);
        const uint32_t sz2 = __shfl_xor_sync(0xffffffffu, sz, 1);
        const float rs2 = __shfl_xor_sync(0xffffffffu, rs, 1);
        uint32_t mk[8], mv[8];
        row_codes(xk, odd ? sz2 : sz, odd ? rs2 : rs, mk);
        row_codes(xv, odd ? sz : sz2, odd ? rs : rs2, mv);
        if (valid) {
            s_k[(word >> 2) * 256 + r * 4 + (word & 3)] = pack_nibbles(mk);
            uint32_t *dst = reinterpret_cast<uint32_t *>(s_v + r * VS + word * 8);
            dst[0] = pack_bytes(mv[0], mv[1], mv[2], mv[3]);
            dst[1] = pack_bytes(mv[4], mv[5], mv[6], mv[7]);
            if (word < 2) s_sz[word][r] = sz;
        }
    }
    __syncthreads();
    // K units of the covered positions
    for (int i = threadIdx.x; i < (D / 32) * kRecKeys; i += blockDim.x)
        if (i % kRecKeys >= r0 && i % kRecKeys < r1)
            reinterpret_cast<uint4 *>(rec)[i] = reinterpret_cast<const uint4 *>(s_k)[i];
    // V words: 8 positions of one channel; four channels at a time
    uint32_t *vw = reinterpret_cast<uint32_t *>(rec + rec_v_off(D));
    const int g0 = r0 >> 3, n_g = ((r1 + 7) >> 3) - g0;  // groups of 8 positions that the append touches
    for (int i = threadIdx.x; i < n_g * (D / 4); i += blockDim.x) {
        const int q = i / n_g, g = g0 + i - q * n_g;
        uint32_t a[8], w[4];
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = *reinterpret_cast<const uint32_t *>(s_v + (8 * g + e) * VS + 4 * q);
        const int e0 = max(r0 - 8 * g, 0), e1 = min(r1 - 8 * g, 8);
        const bool part = e0 > 0 || e1 < 8;
        uint32_t mask = 0xffffffffu;
        if (part) {  // rows of s_v that are not covered hold nothing
            mask = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e >= e0 && e < e1)
                    mask |= 15u << nib_bit(e);
                else
                    a[e] = 0u;
            }
        }
        transpose_codes(a, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t *dst = vw + ((g >> 2) * D + 4 * q + j) * 4 + (g & 3);
            *dst = part ? (*dst & ~mask) | w[j] : w[j];
        }
    }
    for (int i = threadIdx.x; i < 2 * kRecKeys; i += blockDim.x) {
        const int is_v = i / kRecKeys, r = i - is_v * kRecKeys;
        if (r >= r0 && r < r1)
            reinterpret_cast<uint32_t *>(rec + (is_v ? rec_vs_off(D) : rec_ks_off(D)))[r] = s_sz[is_v][r];
    }
}

// Elements 2 i and 2 i + 1 of a word as bf16 values s c + z, rounded once.  A code in the
// low bits of 128 (ulp 1) is 128 + c: one mask-and-or, and an exact subtraction.
__device__ __forceinline__ uint32_t held_pair(uint32_t w, int i, uint32_t s2, uint32_t z2) {
    uint32_t c2, y;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(c2) : "r"(((w >> (4 * i)) & 0x000f000fu) | 0x43004300u), "r"(0xc300c300u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(c2), "r"(s2), "r"(z2));
    return y;
}

// The last n positions as bf16 [B][n][Hkv][D]; rows before position 0 are 0.
// One CTA per record; K: a thread turns one word into 8 channels of a row; V: a thread turns
// 8 positions of 4 channels (a word each) into 8 stores of 8 bytes, four neighbouring
// threads take the words of one unit, so a warp's loads share units and its store covers
// 64 consecutive bytes of 4 rows.
constexpr int kReadThreads = 128;

template <int D>
__global__ void __launch_bounds__(kReadThreads)
    kvq_read_kernel(const KvqView c, int n, __nv_bfloat16 *__restrict__ ko, __nv_bfloat16 *__restrict__ vo,
                    int32_t *__restrict__ err) {
    // K: (s, z) of a row; V: s of two neighbouring rows, z of the same two
    __shared__ uint32_t s_k[kRecKeys];
    __shared__ uint2 s_v[kRecKeys / 2];
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
    // every load of the record before the first use
    constexpr int NK = kRecKeys * (D / 8) / kReadThreads, NV = 2 * D / kReadThreads;
    static_assert(NK * kReadThreads == kRecKeys * (D / 8) && NV * kReadThreads == 2 * D, "whole rounds");
    const auto k_row = [&](int j) { return (int)(threadIdx.x + j * kReadThreads) / (D / 8); };
    const auto v_group = [&](int j) { return (int)(threadIdx.x + j * kReadThreads) / D * 4 + (int)(threadIdx.x & 3); };
    const int wd = threadIdx.x % (D / 8);
    const uint32_t *words = reinterpret_cast<const uint32_t *>(rec), *vw = words + rec_v_off(D) / 4;
    uint32_t kw[NK], w[NV][4];
#pragma unroll
    for (int j = 0; j < NK; ++j)
        if (k_row(j) >= r0 && k_row(j) < r1) kw[j] = __ldg(words + (wd >> 2) * 256 + k_row(j) * 4 + (wd & 3));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int g = v_group(j), ch = (int)(threadIdx.x + j * kReadThreads) % D & ~3;
        if (8 * g < r1 && 8 * g + 8 > r0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[j][i] = __ldg(vw + ((g >> 2) * D + ch + i) * 4 + (g & 3));
        }
    }
    if (threadIdx.x < kRecKeys) {
        s_k[threadIdx.x] = __ldg(words + rec_ks_off(D) / 4 + threadIdx.x);
    } else if (threadIdx.x < 3 * kRecKeys / 2) {
        const int i = threadIdx.x - kRecKeys;
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(rec + rec_vs_off(D)) + i);
        s_v[i] = make_uint2(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632));
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NK; ++j) {
        const int r = k_row(j);
        if (r < r0 || r >= r1) continue;
        const uint32_t sz = s_k[r], s2 = __byte_perm(sz, sz, 0x1010), z2 = __byte_perm(sz, sz, 0x3232);
        reinterpret_cast<uint4 *>(ko + out_row(r))[wd] = make_uint4(
            held_pair(kw[j], 0, s2, z2), held_pair(kw[j], 1, s2, z2), held_pair(kw[j], 2, s2, z2), held_pair(kw[j], 3, s2, z2));
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {  // D / 4 channel quads x 8 groups of positions
        const int g = v_group(j), ch = (int)(threadIdx.x + j * kReadThreads) % D & ~3;
        if (8 * g >= r1 || 8 * g + 8 <= r0) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint2 sz = s_v[4 * g + k];  // rows 8 g + 2 k and the next
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = held_pair(w[j][i], k, sz.x, sz.y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * g + 2 * k + e;
                if (r < r0 || r >= r1) continue;
                const unsigned sel = e ? 0x7632 : 0x5410;
                *reinterpret_cast<uint2 *>(vo + out_row(r) + ch) =
                    make_uint2(__byte_perm(y[0], y[1], sel), __byte_perm(y[2], y[3], sel));
            }
        }
    }
}

}  // namespace

cudaError_t launch_kvq_append(const KvqView &c, const void *k_new, const void *v_new, int n_new, int32_t *err,
                              cudaStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)n_new + kRecKeys - 2) / kRecKeys + 1), (unsigned)(c.batch * c.n_kv_heads));
    const int warps = n_new >= 8 ? kAppendWarps : 4;  // four also share out a single token's V words
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
        case 64: return launch_pdl(kvq_read_kernel<64>, grid, dim3(kReadThreads), 0, stream, c, n, k, v, err);
        case 128: return launch_pdl(kvq_read_kernel<128>, grid, dim3(kReadThreads), 0, stream, c, n, k, v, err);
        case 256: return launch_pdl(kvq_read_kernel<256>, grid, dim3(kReadThreads), 0, stream, c, n, k, v, err);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace wm
