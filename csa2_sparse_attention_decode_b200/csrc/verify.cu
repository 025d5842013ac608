// Verification of drafted tokens against the target's probabilities, and the
// token that follows the accepted ones, from given random numbers.
//
// Draft i is kept while u_i q_i(x_i) < p_i(x_i) (the product is exact in
// fp64).  At the first refused draft the next token is drawn from
// max(p_i - q_i, 0), after all drafts from p_n; the index drawn is the first
// whose cumulative weight exceeds u times the total.
//
// Bound: one row of `vocab` probabilities per request, two after a refusal,
// read once.  A cluster of CTAs shares a request's row: every warp sums a
// contiguous piece, the sums meet over distributed shared memory, and only
// the warp whose piece holds the drawn index reads it again, from L2.  Sums
// are fp64 (of fp32 differences that are exact there): over 10^5 terms fp32
// sums would move the borders between tokens by more than a token's weight.
#include "common.cuh"
#include "serve.cuh"

#include <cooperative_groups.h>
namespace cg = cooperative_groups;

namespace csa2 {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int UNROLL = 8;

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// Weight of token v: the target's probability, or what the drafter's leaves of it.
struct Weights {
    const float *p, *q;                        // q null: the drafter named token x for certain
    int x;
    bool residual;
    __device__ __forceinline__ double of(float pv, float qv) const
    {
        if (!residual) return pv > 0.0f ? (double)pv : 0.0;
        return pv > qv ? (double)pv - (double)qv : 0.0;
    }
    __device__ __forceinline__ float draft(int v) const { return q ? q[v] : (v == x ? 1.0f : 0.0f); }
    __device__ __forceinline__ double operator()(int v) const { return of(p[v], residual ? draft(v) : 0.0f); }
};

__global__ void __launch_bounds__(THREADS) verify_kernel(VerifyArgs a)
{
    __shared__ double part[WARPS];
    __shared__ double cta_sum;
    __shared__ int accepted_s;
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / nc, K = a.max_draft, V = a.vocab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependents();

    int nd = a.n_draft[b];
    if (nd < 0 || nd > K) {
        if (rank == 0 && threadIdx.x == 0) set_error(a.error, CSA2_DEV_BAD_REQUEST);
        nd = max(0, min(nd, K));
    }
    if (warp == 0) {                                                   // one lane a draft: K <= 31
        bool refused = lane >= nd;
        if (lane < nd) {
            const int x = a.draft[(size_t)b * K + lane];
            if (x < 0 || x >= V) {
                if (rank == 0) set_error(a.error, CSA2_DEV_BAD_INDEX);
                refused = true;
            } else {
                const double p = a.target[((size_t)b * (K + 1) + lane) * V + x];
                const double q = a.probs ? a.probs[((size_t)b * K + lane) * V + x] : 1.0f;
                refused = !((double)a.u[(size_t)b * (K + 1) + lane] * q < p);
            }
        }
        const int n = __ffs(__ballot_sync(~0u, refused)) - 1;          // lane 31 always refuses
        if (lane == 0) accepted_s = n;
    }
    __syncthreads();
    const int n = accepted_s;
    Weights w;
    w.p = a.target + ((size_t)b * (K + 1) + n) * V;
    w.residual = n < nd;
    w.q = w.residual && a.probs ? a.probs + ((size_t)b * K + n) * V : nullptr;
    w.x = w.residual ? a.draft[(size_t)b * K + n] : -1;

    // piece of this warp: contiguous, a multiple of 32 so that rows stay aligned with one another
    const int per = ((V + nc * WARPS - 1) / (nc * WARPS) + 31) & ~31;
    const int v0 = min(V, (rank * WARPS + warp) * per), v1 = min(V, v0 + per);
    double before = 0.0, total = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        double s = 0.0;
        for (int v = v0 + lane; v < v1; v += 32 * UNROLL) {
            float pv[UNROLL], qv[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int j = v + 32 * i;
                pv[i] = j < v1 ? w.p[j] : 0.0f;
                qv[i] = w.residual && j < v1 ? w.draft(j) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) s += w.of(pv[i], qv[i]);
        }
        s = warp_sum(s);
        if (lane == 0) part[warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            double t = 0.0;
            for (int i = 0; i < WARPS; ++i) t += part[i];
            cta_sum = t;
        }
        cluster.sync();
        before = total = 0.0;
        for (int r = 0; r < nc; ++r) {
            const double t = *cluster.map_shared_rank(&cta_sum, r);
            if (r < rank) before += t;
            total += t;
        }
        cluster.sync();                                                // the sums are read: they may change, or the CTA end
        if (total > 0.0 || !w.residual) break;
        w.residual = false;                                            // p <= q everywhere: what is left is p itself
    }
    // The CTA whose sums straddle the mark holds the drawn index; in it, the
    // first warp whose running end passes the mark, or, where the warps' sums
    // round a last bit below the CTA's, the last warp with any weight.
    // Without a finite positive total (rows of zeros, NaN) it is the last token.
    const double mark = fmin(fmax((double)a.u[(size_t)b * (K + 1) + K], 0.0), 1.0 - 0x1p-24) * total;
    int *tokens = a.tokens + (size_t)b * (K + 1);
    if (total > 0.0 && total < INFINITY) {
        int chosen = -1, any = -1;
        double at = before, c = before;
        for (int i = 0; i < WARPS; ++i) {
            if (chosen < 0 && part[i] > 0.0) {
                any = i;
                c = at;
                if (at + part[i] > mark) chosen = i;
            }
            at += part[i];
        }
        if (chosen < 0) chosen = any;
        if (before <= mark && mark < before + cta_sum && warp == chosen) {
            int hit = -1, last = v0;
            for (int v = v0; v < v1 && hit < 0; v += 32) {
                const double x = v + lane < v1 ? w(v + lane) : 0.0;
                double s = x;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const double y = __shfl_up_sync(~0u, s, d);
                    if (lane >= d) s += y;
                }
                const unsigned over = __ballot_sync(~0u, c + s > mark && x > 0.0), some = __ballot_sync(~0u, x > 0.0);
                if (over) hit = v + __ffs(over) - 1;
                if (some) last = v + 31 - __clz(some);
                c += __shfl_sync(~0u, s, 31);
            }
            if (lane == 0) tokens[n] = hit >= 0 ? hit : last;          // likewise a last bit short
        }
    } else if (rank == 0 && threadIdx.x == 0) {
        set_error(a.error, CSA2_DEV_BAD_REQUEST);
        tokens[n] = V - 1;
    }
    if (rank == 0 && threadIdx.x <= K && (int)threadIdx.x != n)
        tokens[threadIdx.x] = (int)threadIdx.x < n ? a.draft[(size_t)b * K + threadIdx.x] : -1;
    if (rank == 0 && threadIdx.x == 0) a.n_accepted[b] = n;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st)
{
    LaunchScope scope(-1, st);
    const int nc = a.vocab >= 16384 ? MAX_CLUSTER : 1;
    return launch_pdl_cluster(verify_kernel, dim3((unsigned)a.batch * nc), dim3(THREADS), 0, st, nc, a);
}

}  // namespace csa2
