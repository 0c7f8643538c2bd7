// accept.cu -- verification of drafted tokens against the target's
// probabilities (speculative sampling), random numbers given by the caller.
//
// Sequence b, drafts x_0 .. x_{n-1}: x_j is accepted while u_j q_j(x_j) < p_j(x_j);
// a = the accepted count.  One more token comes from r = max(p_a - q_a, 0) if
// a < n, else r = p_n, by inversion: the least i with r_0 + .. + r_i > w sum(r).
//
// Exactness: a product u q is compared as the pair (fl(u q), its error), and a
// difference p - q with p > q is exact as a pair of floats (d = fl(p - q), e = (p - d) - q).
// Every sum is such a pair (two-sum, about 48 bits), at every level: this GPU has 2 FP64
// units per SM, on which one scan of a warp took 1000 clocks where a scan of
// pairs takes 300.
//
// One cluster of CTAs per sequence: each CTA sums a run of the row, the totals
// meet through distributed shared memory, and the CTA that holds the threshold
// looks for the token in its run -- the warp's run, then its sixteenth (every warp sums
// one, from L2), then the entry.  The other CTAs leave as soon as every total has
// been read.  One launch, no workspace, no atomics, so the same inputs give the
// same token in any launch.
// A row is summed in one pass, two entries per instruction (6 instructions an entry without
// a draft row; one at a time, with checks in the loop, 31 took 50 us where this takes 32).
// What bounds it: HBM for a large batch (256 rows of 131072 entries, 134 MB: 32 us, of
// which the stream is 20 at HBM's rate); for one sequence the chain of dependent loads
// (draft, its probabilities, the row, the search), 9 us.
#include <cooperative_groups.h>

#include "kvq.cuh"
#include "ptx.cuh"

namespace wm {

namespace {

namespace cg = cooperative_groups;

constexpr int kAcceptThreads = 512;
constexpr int kAcceptWarps = kAcceptThreads / 32;
// Loads per lane in flight together, and CTAs per SM, which bound the registers: 256 rows of
// 131072 entries take 32 us; with 8 loads 34.7, with 32 35.5; with 4 CTAs and 8 loads 37, with
// 3 38.8.
constexpr int kLoads = 16, kAcceptPerSm = 2;

// hi + lo, hi the nearest float.
struct Pair {
    float hi = 0.f, lo = 0.f;
    // + (d + e), d exact; lo is left to grow
    __device__ __forceinline__ void add(float d, float e) {
        const float s = hi + d;
        const float bb = s - hi;
        lo += ((hi - (s - bb)) + (d - bb)) + e;
        hi = s;
    }
    __device__ __forceinline__ bool positive() const { return hi > 0.f; }
};

// The same bits whichever operand comes first.
__device__ __forceinline__ Pair operator+(const Pair &a, const Pair &b) {
    const float s = a.hi + b.hi, bb = s - a.hi;
    const float e = ((a.hi - (s - bb)) + (b.hi - bb)) + (a.lo + b.lo);
    Pair r;
    r.hi = s + e;
    r.lo = e - (r.hi - s);
    return r;
}

__device__ __forceinline__ bool operator>(const Pair &a, const Pair &b) {
    return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}

// u x, u a float
__device__ __forceinline__ Pair times(float u, const Pair &x) {
    const float h = u * x.hi, l = fmaf(u, x.hi, -h) + u * x.lo;
    Pair r;
    r.hi = h + l;
    r.lo = l - (r.hi - h);
    return r;
}

__device__ __forceinline__ Pair shfl(const Pair &x, int lane) {
    return Pair{__shfl_sync(0xffffffffu, x.hi, lane), __shfl_sync(0xffffffffu, x.lo, lane)};
}

// Sum over the lanes of a warp, on every lane.
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = x + Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
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
__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
        if (lane >= o) x = y + x;
    }
    return x;
}

// The lane whose share holds t: the first with v > 0 and base + (sum of the lanes up to
// it) > t, else (past = false) the last with v > 0; -1 if none.  Adds the shares
// before it to base.  With u >= 0 the threshold is set first: u times the sum of all shares.
__device__ __forceinline__ int pick(const Pair &v, float u, Pair &t, Pair &base, int lane, bool &past) {
    const Pair incl = base + warp_scan(v, lane);
    if (u >= 0.f) t = times(u, shfl(incl, 31));
    const unsigned some = __ballot_sync(0xffffffffu, v.positive());
    const unsigned beyond = __ballot_sync(0xffffffffu, v.positive() && incl > t);
    past = beyond != 0u;
    if (!some) return -1;
    const int l = beyond ? __ffs(beyond) - 1 : 31 - __clz(some);
    const Pair before = shfl(incl, max(l - 1, 0));
    if (l > 0) base = before;
    return l;
}

// Lane's entry of n sums in shared memory.
__device__ __forceinline__ Pair from(const float2 *x, int lane, int n) {
    return lane < n ? Pair{x[lane].x, x[lane].y} : Pair{};
}

// Sums of two entries' lanes side by side, each as a Pair.
struct Pairs {
    uint64_t hi = 0, lo = 0;
    // a - b in both, rounded once
    static __device__ __forceinline__ uint64_t minus(uint64_t a, uint64_t b) {
        return fma2(b, pack2(-1.f, -1.f), a);
    }
    __device__ __forceinline__ uint64_t add(uint64_t d) {  // returns the errors
        const uint64_t s = add2(hi, d), bb = minus(s, hi);
        const uint64_t e = add2(minus(hi, minus(s, bb)), minus(d, bb));
        hi = s;
        return e;
    }
    __device__ __forceinline__ Pair sum() const {
        float h0, h1, l0, l1;
        unpack2(hi, h0, h1);
        unpack2(lo, l0, l1);
        return (Pair{} + Pair{h0, l0}) + (Pair{} + Pair{h1, l1});
    }
};

// Adds entries i, i + 32, .. of a lane (L of them, those below i1 if TAIL); p and q point at i.
template <bool Q, bool TAIL, int L>
__device__ __forceinline__ void add_block(Pairs &acc, const float *p, const float *q, int i, int i1, int skip) {
    float pv[L], qv[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        pv[j] = qv[j] = 0.f;
        if (!TAIL || i + 32 * j < i1) {
            pv[j] = __ldg(p + 32 * j);
            if (Q) qv[j] = __ldg(q + 32 * j);
        }
    }
    if (!Q && (unsigned)(skip - i) < 32u * L) {
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (i + 32 * j == skip) pv[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < L; j += 2) {
        const uint64_t p2 = pack2(__saturatef(pv[j]), __saturatef(pv[j + 1]));
        if (Q) {
            const uint64_t q2 = pack2(__saturatef(qv[j]), __saturatef(qv[j + 1]));
            const uint64_t d2 = Pairs::minus(p2, q2);
            float d0, d1, e0, e1;
            unpack2(d2, d0, d1);
            unpack2(Pairs::minus(Pairs::minus(p2, d2), q2), e0, e1);  // exact where d > 0
            if (!(d0 > 0.f)) d0 = e0 = 0.f;
            if (!(d1 > 0.f)) d1 = e1 = 0.f;
            acc.lo = add2(acc.lo, add2(acc.add(pack2(d0, d1)), pack2(e0, e1)));
        } else {
            acc.lo = add2(acc.lo, acc.add(p2));
        }
    }
}

// Sum of entries [i0, i1) of the row over one warp, on every lane.
template <bool Q>
__device__ __forceinline__ Pair run_sum(const Row &row, int i0, int i1, int lane) {
    constexpr int L = Q ? kLoads / 2 : kLoads;
    Pairs acc;
    int i = i0 + lane;
    const float *p = row.p + i, *q = Q ? row.q + i : nullptr;
    for (; i - lane + 32 * L <= i1; i += 32 * L, p += 32 * L) {
        add_block<Q, false, L>(acc, p, q, i, i1, row.skip);
        if (Q) q += 32 * L;
    }
    if (i - lane < i1) add_block<Q, true, L>(acc, p, q, i, i1, row.skip);
    return warp_sum(acc.sum());
}

__device__ __forceinline__ Pair run_sum(const Row &row, int i0, int i1, int lane) {
    return row.q ? run_sum<true>(row, i0, i1, lane) : run_sum<false>(row, i0, i1, lane);
}

__global__ void __launch_bounds__(kAcceptThreads, kAcceptPerSm) spec_accept_kernel(const AcceptParams P) {
    __shared__ int s_a, s_n, s_x, s_owner;
    __shared__ float2 s_warp[kAcceptWarps], s_sub[kAcceptWarps], s_total[2], s_base, s_t;
    pdl_wait();
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int b = blockIdx.y, rank = (int)cluster.block_rank(), n_cta = (int)cluster.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t V = P.vocab;

    float u_sample = 0.f;
    if (warp == 0) {
        u_sample = __saturatef(P.u_sample[b]);
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
                    // u q < p exactly: scaled so that the product's error cannot underflow where it matters
                    const float us = u * 0x1p60f, qs = qv * 0x1p60f, ps = pv * 0x1p120f, h = us * qs;
                    ok = h < ps || (h == ps && fmaf(us, qs, -h) < 0.f);
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
        const Pair v = run_sum(row, w0, w1, lane);
        if (lane == 0) s_warp[warp] = make_float2(v.hi, v.lo);
        __syncthreads();
        if (warp == 0) {
            const Pair t = warp_sum(from(s_warp, lane, kAcceptWarps));
            if (lane == 0) s_total[pass] = make_float2(t.hi, t.lo);
        }
        cluster.sync();
        if (warp == 0) {
            Pair share;
            if (lane < n_cta) {
                const float2 x = *cluster.map_shared_rank(&s_total[pass], lane);
                share = Pair{x.x, x.y};
            }
            Pair t, base;
            bool past;
            const int owner = pick(share, u_sample, t, base, lane, past);  // -1: no weight at all
            if (lane == 0) {
                s_owner = owner;
                s_base = make_float2(base.hi, base.lo);
                s_t = make_float2(t.hi, t.lo);
            }
        }
        __syncthreads();
        // this CTA has read the others' totals (nothing else is handed over: no release)
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
        if (s_owner >= 0 || (!row.q && row.skip < 0)) break;
        // nothing left where the target exceeds the draft: the target's own row
        row.q = nullptr;
        row.skip = -1;
        asm volatile("barrier.cluster.wait;" ::: "memory");
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
        Pair t{s_t.x, s_t.y}, base{s_base.x, s_base.y};
        // the warp's run that holds t, its part, the lane's eight entries, the entry
        bool past;
        const int w = pick(from(s_warp, lane, kAcceptWarps), -1.f, t, base, lane, past);
        const int x0 = c0 + w * per_warp, x1 = min(c1, x0 + per_warp);
        const int per_sub = ((x1 - x0 + kAcceptWarps - 1) / kAcceptWarps + 31) / 32 * 32;
        const int y0 = min(x1, x0 + warp * per_sub);
        const Pair v = run_sum(row, y0, min(x1, y0 + per_sub), lane);
        if (lane == 0) s_sub[warp] = make_float2(v.hi, v.lo);
        __syncthreads();
        if (warp == 0) {
            const int s = pick(from(s_sub, lane, kAcceptWarps), -1.f, t, base, lane, past);
            const int z0 = x0 + s * per_sub, z1 = min(x1, z0 + per_sub);
            int token = -1;
            for (int z = z0; z < z1; z += 256) {
                float pv[8], qv[8];
                Pair e[8], part;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = z + 8 * lane + j;
                    pv[j] = qv[j] = 0.f;
                    if (i < z1) row.load(i, pv[j], qv[j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    row.weight(pv[j], qv[j], z + 8 * lane + j, e[j].hi, e[j].lo);
                    part.add(e[j].hi, e[j].lo);
                }
                part = Pair{} + part;
                const Pair end = base + warp_sum(part);
                const int l = pick(part, -1.f, t, base, lane, past);
                if (l < 0) continue;
                Pair r;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const Pair x = shfl(e[j], l);
                    if (lane == j) r = x;
                }
                const bool found = past;
                token = z + 8 * l + pick(r, -1.f, t, base, lane, past);
                if (found) break;
                base = end;  // the last entry with weight is kept if rounding leaves none past t
            }
            if (lane == 0) tokens[a] = token;
        }
    }
    asm volatile("barrier.cluster.wait;" ::: "memory");  // no CTA leaves while another may still read its total
}

}  // namespace

cudaError_t launch_spec_accept(const AcceptParams &p, int sms, cudaStream_t stream) {
    // CTAs per sequence: as many as leave every CTA resident at once, so that one sequence is
    // spread as wide as a portable cluster goes and a large batch pays the fixed cost of a
    // CTA (about as long as 128 KB take) rarely.
    unsigned n = 8;
    while (n > 1 && (int64_t)p.batch * n > (int64_t)kAcceptPerSm * sms) n >>= 1;
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
