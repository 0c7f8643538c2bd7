// accept.cu -- verification of drafted tokens against the target's
// probabilities (speculative sampling), random numbers given by the caller.
//
// Sequence b, drafts x_0 .. x_{n-1}: x_j is accepted while u_j q_j(x_j) < p_j(x_j);
// a = the accepted count.  One more token comes from r = max(p_a - q_a, 0) if
// a < n, else r = p_n, by inversion: the least i with r_0 + .. + r_i > w sum(r).
//
// Exactness: the products u q are exact in 64 bits, and a difference p - q
// with p > q is exact as a pair of floats (d = fl(p - q), e = (p - d) - q).
// Sums run in such pairs (two-sum, about 48 bits) per lane and in doubles
// above; the 64-bit units of this GPU are too few (about 2 FMA per SM and
// clock) to add every entry in doubles: 128K entries on one SM would take 35 us.
//
// One cluster of CTAs per sequence: each CTA sums a run of the row, the totals
// meet through distributed shared memory, and the CTA that holds the threshold
// looks for the token in its run -- warp by warp, then lane by lane, then entry
// by entry, re-reading only one warp's run (from L2).  One launch, no workspace, no
// atomics, so the same inputs give the same token in any launch.
#include <cooperative_groups.h>

#include "kvq.cuh"
#include "ptx.cuh"

namespace wm {

namespace {

namespace cg = cooperative_groups;

constexpr int kAcceptThreads = 512;
constexpr int kAcceptWarps = kAcceptThreads / 32;
constexpr int kLoads = 8;  // entries per lane whose loads are in flight together

struct Pair {
    float hi = 0.f, lo = 0.f;
    // + (d + e), d exact
    __device__ __forceinline__ void add(float d, float e) {
        const float s = hi + d;
        const float bb = s - hi;
        lo += ((hi - (s - bb)) + (d - bb)) + e;
        hi = s;
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// Weight of entry i: max(p - q, 0) as an exact pair, or p; NaN and negative
// entries count as 0, entries above 1 as 1.
struct Row {
    const float *p, *q;
    int skip;  // entry taken as 0 (one-hot draft), -1 for none
    __device__ __forceinline__ void weight(float pv, float qv, int i, float &d, float &e) const {
        pv = __saturatef(pv);
        e = 0.f;
        d = i == skip ? 0.f : pv;
        if (q) {
            qv = __saturatef(qv);
            d = pv - qv;
            e = (pv - d) - qv;
            if (!(d > 0.f)) d = e = 0.f;
        }
    }
    __device__ __forceinline__ void load(int i, float &pv, float &qv) const {
        pv = __ldg(p + i);
        qv = q ? __ldg(q + i) : 0.f;
    }
};

// Inclusive sum over the lanes of one warp.
__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The lane whose share of [0, total) holds t: the first with v > 0 and
// base + (sum of lanes up to it) > t, else the last with v > 0; -1 if none.
// Adds the shares before it to base.
__device__ __forceinline__ int pick(double v, double t, double &base, int lane) {
    const double incl = base + warp_scan(v, lane);
    const unsigned some = __ballot_sync(0xffffffffu, v > 0.0);
    const unsigned past = __ballot_sync(0xffffffffu, v > 0.0 && incl > t);
    if (!some) return -1;
    const int l = past ? __ffs(past) - 1 : 31 - __clz(some);
    base = __shfl_sync(0xffffffffu, incl - v, l);
    return l;
}

__global__ void __launch_bounds__(kAcceptThreads) spec_accept_kernel(const AcceptParams P) {
    __shared__ int s_a, s_n, s_x;
    __shared__ double s_warp[2][kAcceptWarps];
    __shared__ double s_total[2];
    pdl_wait();
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.y, rank = (int)cluster.block_rank(), n_cta = (int)cluster.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t V = P.vocab;

    if (warp == 0) {
        int n = P.k;
        if (P.n_draft) {
            n = P.n_draft[b];
            if (n < 0 || n > P.k) {
                if (lane == 0 && rank == 0) kvq_report(P.err, WM_DEVERR_BAD_LENGTH);
                n = n < 0 ? 0 : P.k;
            }
        }
        int a = n;
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int j = j0 + lane;
            bool ok = true;
            if (j < n) {
                const int x = P.draft_tokens[(int64_t)b * P.k + j];
                ok = x >= 0 && x < P.vocab;
                if (ok) {
                    const float pv = __saturatef(P.target_probs[((int64_t)b * (P.k + 1) + j) * V + x]);
                    const float qv = P.draft_probs ? __saturatef(P.draft_probs[((int64_t)b * P.k + j) * V + x]) : 1.f;
                    const float u = __saturatef(P.u_accept[(int64_t)b * P.k + j]);
                    ok = (double)u * (double)qv < (double)pv;
                }
            }
            const unsigned bad = __ballot_sync(0xffffffffu, !ok);
            if (bad) {
                a = j0 + __ffs(bad) - 1;
                break;
            }
        }
        if (lane == 0) {
            s_a = a;
            s_n = n;
            s_x = -1;
            if (a < n) {
                const int x = P.draft_tokens[(int64_t)b * P.k + a];
                if (x >= 0 && x < P.vocab)
                    s_x = x;
                else if (rank == 0)
                    kvq_report(P.err, WM_DEVERR_BAD_TOKEN);
            }
        }
    }
    __syncthreads();
    const int a = s_a, n = s_n;
    Row row;
    row.p = P.target_probs + ((int64_t)b * (P.k + 1) + a) * V;
    row.q = a < n && P.draft_probs ? P.draft_probs + ((int64_t)b * P.k + a) * V : nullptr;
    row.skip = a < n && !P.draft_probs ? s_x : -1;

    // this CTA's run of the row, and this warp's run of it (multiples of 32 entries)
    const int per_cta = (int)(((V + n_cta - 1) / n_cta + 31) / 32 * 32);
    const int c0 = (int)min(V, (int64_t)rank * per_cta), c1 = (int)min(V, (int64_t)c0 + per_cta);
    const int per_warp = ((c1 - c0 + kAcceptWarps - 1) / kAcceptWarps + 31) / 32 * 32;
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);

    int token = -1;
    bool mine = false;
    for (int pass = 0; pass < 2; ++pass) {
        Pair acc;
        for (int i0 = w0; i0 < w1; i0 += 32 * kLoads) {
            float pv[kLoads], qv[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int i = i0 + 32 * j + lane;
                pv[j] = qv[j] = 0.f;
                if (i < w1) row.load(i, pv[j], qv[j]);
            }
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                float d, e;
                row.weight(pv[j], qv[j], i0 + 32 * j + lane, d, e);
                acc.add(d, e);
            }
        }
        double v = acc.value();
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_warp[pass][warp] = v;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = 0.0;
            for (int w = 0; w < kAcceptWarps; ++w) t += s_warp[pass][w];
            s_total[pass] = t;
        }
        cluster.sync();
        if (warp == 0) {
            const double share = lane < n_cta ? *cluster.map_shared_rank(&s_total[pass], lane) : 0.0;
            const double total = __shfl_sync(0xffffffffu, warp_scan(share, lane), 31);
            if (total > 0.0) {
                const double t = (double)__saturatef(P.u_sample[b]) * total;
                double base = 0.0;
                mine = pick(share, t, base, lane) == rank;
                if (mine) {
                    // the warp, then the lane (contiguous shares this time), then the entry
                    const int w = pick(lane < kAcceptWarps ? s_warp[pass][lane] : 0.0, t, base, lane);
                    const int x0 = c0 + w * per_warp, x1 = min(c1, x0 + per_warp);
                    const int each = (x1 - x0 + 31) / 32;
                    Pair part;
                    for (int j = 0; j < each; ++j) {
                        const int i = x0 + lane * each + j;
                        if (i < x1) {
                            float pv, qv, d, e;
                            row.load(i, pv, qv);
                            row.weight(pv, qv, i, d, e);
                            part.add(d, e);
                        }
                    }
                    const int l = pick(part.value(), t, base, lane);
                    const int y0 = x0 + l * each, y1 = min(x1, y0 + each);
                    for (int i0 = y0; i0 < y1; i0 += 32) {
                        const int i = i0 + lane;
                        double r = 0.0;
                        if (i < y1) {
                            float pv, qv, d, e;
                            row.load(i, pv, qv);
                            row.weight(pv, qv, i, d, e);
                            r = (double)d + (double)e;
                        }
                        const double incl = base + warp_scan(r, lane);
                        const unsigned some = __ballot_sync(0xffffffffu, r > 0.0);
                        const unsigned past = __ballot_sync(0xffffffffu, r > 0.0 && incl > t);
                        if (past) {
                            token = i0 + __ffs(past) - 1;
                            break;
                        }
                        if (some) token = i0 + 31 - __clz(some);  // kept if rounding leaves none past t
                        base = __shfl_sync(0xffffffffu, incl, 31);
                    }
                }
            }
            if (lane == 0) s_x = total > 0.0;
        }
        __syncthreads();
        if (s_x || (!row.q && row.skip < 0)) break;
        // nothing left where the target exceeds the draft: the target's own row
        row.q = nullptr;
        row.skip = -1;
        __syncthreads();
    }
    if (warp == 0) {
        const bool none = !s_x;  // the target's row holds no weight at all
        if (rank == 0) {
            for (int j = lane; j <= P.k; j += 32)
                if (j != a)
                    P.tokens[(int64_t)b * (P.k + 1) + j] = j < a ? P.draft_tokens[(int64_t)b * P.k + j] : -1;
            if (lane == 0) {
                P.n_accepted[b] = a;
                if (P.new_len) P.new_len[b] = P.seq_lens[b] - P.k + a;
                if (none) kvq_report(P.err, WM_DEVERR_BAD_PROB);
            }
        }
        if (lane == 0 && (mine || (none && rank == 0))) P.tokens[(int64_t)b * (P.k + 1) + a] = mine ? token : -1;
    }
    cluster.sync();  // no CTA leaves while another may still read its totals
}

}  // namespace

cudaError_t launch_spec_accept(const AcceptParams &p, int sms, cudaStream_t stream) {
    (void)sms;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kAcceptThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 8;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(8, (unsigned)p.batch);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, spec_accept_kernel, p);
}

}  // namespace wm
