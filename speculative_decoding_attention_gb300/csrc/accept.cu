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
// looks for the token in its run -- the warp's run, then its sixteenth (every warp sums
// one, from L2), then the entry.  The other CTAs leave as soon as every total has
// been read.  One launch, no workspace, no atomics, so the same inputs give the
// same token in any launch.
// What bounds it: HBM for a large batch; for one sequence the chain of dependent
// loads (draft, its probabilities, the row, the search).
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

// Sum over the lanes of a warp, on every lane.
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float d = __shfl_xor_sync(0xffffffffu, x.hi, o), e = __shfl_xor_sync(0xffffffffu, x.lo, o);
        // the same operation on both sides, so that all lanes end with the same bits
        const Pair a = x.hi >= d ? x : Pair{d, e}, b = x.hi >= d ? Pair{d, e} : x;
        x = a;
        x.add(b.hi, b.lo);
    }
    return x;
}

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

// Sum of entries [i0, i1) of the row over one warp, on every lane.
__device__ __forceinline__ double run_sum(const Row &row, int i0, int i1, int lane) {
    Pair acc;
    for (; i0 < i1; i0 += 32 * kLoads) {
        float pv[kLoads], qv[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = i0 + 32 * j + lane;
            pv[j] = qv[j] = 0.f;
            if (i < i1) row.load(i, pv[j], qv[j]);
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            float d, e;
            row.weight(pv[j], qv[j], i0 + 32 * j + lane, d, e);
            acc.add(d, e);
        }
    }
    return warp_sum(acc).value();
}

__global__ void __launch_bounds__(kAcceptThreads, 4) spec_accept_kernel(const AcceptParams P) {
    __shared__ int s_a, s_n, s_x, s_owner;
    __shared__ double s_warp[kAcceptWarps], s_sub[kAcceptWarps], s_total[2], s_base, s_t;
    pdl_wait();
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.y, rank = (int)cluster.block_rank(), n_cta = (int)cluster.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t V = P.vocab;

    if (warp == 0) {
        int n = P.n_draft ? P.n_draft[b] : P.k;
        if (n < 0 || n > P.k) {
            if (lane == 0 && rank == 0) kvq_report(P.err, WM_DEVERR_BAD_LENGTH);
            n = n < 0 ? 0 : P.k;
        }
        int a = n, xa = -1;
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int j = j0 + lane;
            bool ok = true;
            int x = -1;
            if (j < n) {
                x = P.draft_tokens[(int64_t)b * P.k + j];
                const float u = __saturatef(P.u_accept[(int64_t)b * P.k + j]);
                ok = x >= 0 && x < P.vocab;
                if (ok) {
                    const float pv = __saturatef(P.target_probs[((int64_t)b * (P.k + 1) + j) * V + x]);
                    const float qv = P.draft_probs ? __saturatef(P.draft_probs[((int64_t)b * P.k + j) * V + x]) : 1.f;
                    ok = (double)u * (double)qv < (double)pv;
                }
            }
            const unsigned bad = __ballot_sync(0xffffffffu, !ok);
            if (bad) {
                a = j0 + __ffs(bad) - 1;
                xa = __shfl_sync(0xffffffffu, x, a - j0);
                if ((xa < 0 || xa >= P.vocab) && lane == 0 && rank == 0) kvq_report(P.err, WM_DEVERR_BAD_TOKEN);
                break;
            }
        }
        if (lane == 0) {
            s_a = a;
            s_n = n;
            s_x = xa;
        }
    }
    __syncthreads();
    const int a = s_a;
    const bool refused = a < s_n;
    Row row;
    row.p = P.target_probs + ((int64_t)b * (P.k + 1) + a) * V;
    row.q = refused && P.draft_probs ? P.draft_probs + ((int64_t)b * P.k + a) * V : nullptr;
    row.skip = refused && !P.draft_probs ? s_x : -1;

    // this CTA's run of the row, and this warp's run of it (multiples of 32 entries)
    const int per_cta = (int)(((V + n_cta - 1) / n_cta + 31) / 32 * 32);
    const int c0 = (int)min(V, (int64_t)rank * per_cta), c1 = (int)min(V, (int64_t)c0 + per_cta);
    const int per_warp = ((c1 - c0 + kAcceptWarps - 1) / kAcceptWarps + 31) / 32 * 32;
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);

    for (int pass = 0;; ++pass) {
        const double v = run_sum(row, w0, w1, lane);
        if (lane == 0) s_warp[warp] = v;
        __syncthreads();
        if (warp == 0) {
            const double t = __shfl_sync(0xffffffffu, warp_scan(lane < kAcceptWarps ? s_warp[lane] : 0.0, lane), 31);
            if (lane == 0) s_total[pass] = t;
        }
        cluster.sync();
        if (warp == 0) {
            const double share = lane < n_cta ? *cluster.map_shared_rank(&s_total[pass], lane) : 0.0;
            const double total = __shfl_sync(0xffffffffu, warp_scan(share, lane), 31);
            const double t = (double)__saturatef(P.u_sample[b]) * total;
            double base = 0.0;
            const int owner = pick(share, t, base, lane);  // -1: no weight at all
            if (lane == 0) {
                s_owner = owner;
                s_base = base;
                s_t = t;
            }
        }
        __syncthreads();
        cluster.barrier_arrive();  // this CTA has read the others' totals
        if (s_owner >= 0 || (!row.q && row.skip < 0)) break;
        // nothing left where the target exceeds the draft: the target's own row
        row.q = nullptr;
        row.skip = -1;
        cluster.barrier_wait();
    }
    const int owner = s_owner;
    int32_t *tokens = P.tokens + (int64_t)b * (P.k + 1);
    if (rank == 0 && warp == 0) {
        for (int j = lane; j <= P.k; j += 32)
            if (j != a) tokens[j] = j < a ? P.draft_tokens[(int64_t)b * P.k + j] : -1;
        if (lane == 0) {
            P.n_accepted[b] = a;
            if (P.new_len) P.new_len[b] = P.seq_lens[b] - P.k + a;
            if (owner < 0) {
                tokens[a] = -1;
                kvq_report(P.err, WM_DEVERR_BAD_PROB);
            }
        }
    }
    if (owner == rank) {
        const double t = s_t;
        double base = s_base;
        // the warp's run that holds t, its sixteenth, then the entry
        const int w = pick(lane < kAcceptWarps ? s_warp[lane] : 0.0, t, base, lane);
        const int x0 = c0 + w * per_warp, x1 = min(c1, x0 + per_warp);
        const int per_sub = ((x1 - x0 + kAcceptWarps - 1) / kAcceptWarps + 31) / 32 * 32;
        const int y0 = min(x1, x0 + warp * per_sub);
        const double v = run_sum(row, y0, min(x1, y0 + per_sub), lane);
        if (lane == 0) s_sub[warp] = v;
        __syncthreads();
        if (warp == 0) {
            const int s = pick(lane < kAcceptWarps ? s_sub[lane] : 0.0, t, base, lane);
            const int z0 = x0 + s * per_sub, z1 = min(x1, z0 + per_sub);
            int token = -1;
            for (int i0 = z0; i0 < z1; i0 += 32) {
                const int i = i0 + lane;
                double r = 0.0;
                if (i < z1) {
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
            if (lane == 0) tokens[a] = token;
        }
    }
    cluster.barrier_wait();  // no CTA leaves while another may still read its total
}

}  // namespace

cudaError_t launch_spec_accept(const AcceptParams &p, int sms, cudaStream_t stream) {
    // CTAs per sequence: as many as leave every CTA resident at once (four per SM), so
    // that one sequence is spread as wide as a portable cluster goes and a large
    // batch pays the fixed cost of a CTA (about as long as 128 KB take) rarely.
    unsigned n = 8;
    while (n > 1 && (int64_t)p.batch * n > 4ll * sms) n >>= 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kAcceptThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(n, (unsigned)p.batch);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, spec_accept_kernel, p);
}

}  // namespace wm
