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
// the warp whose piece holds the drawn index reads it again, from L2.  A
// lane adds 16 weights at a time as a tree of fp32 sums that keeps what each
// addition rounds off, in fp32 too: off by at most 2^-42 of the 16 (low parts
// of 5 x 2^-24, 8 roundings).  All further sums are fp64.  With every weight
// converted to fp64 instead 64 requests x 131072 tokens take 19.0 us: a warp
// converts 32 values in 16 cycles.  As it is 17.3 us, 51 MB in 2.9 TB/s; what
// is left is latency: the drafts' probabilities, then the row, then the sums,
// then the index, each waits for the one before.
#include "common.cuh"
#include "serve.cuh"

#include <cooperative_groups.h>
namespace cg = cooperative_groups;

namespace csa2 {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int BLOCK = 16;                      // loads of each row in flight, a lane; a block is 16 x 32 weights

__device__ __forceinline__ double warp_sum(double v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// What t = a + b, rounded, leaves of the exact sum (Knuth's two-sum).
__device__ __forceinline__ float lost(float a, float b, float t)
{
    const float z = t - a;
    return (a - (t - z)) + (b - z);
}

// Weight of token v: the target's probability, or what the drafter's leaves of it.
struct Weights {
    const float *p, *q;                        // q null: the drafter named token x for certain
    int x;
    bool residual;
    __device__ __forceinline__ double of(float pv, float qv) const     // exact
    {
        if (!residual) return pv > 0.0f ? (double)pv : 0.0;
        return pv > qv ? (double)pv - (double)qv : 0.0;
    }
    __device__ __forceinline__ float draft(int v) const { return q ? q[v] : (v == x ? 1.0f : 0.0f); }
    __device__ __forceinline__ double operator()(int v) const { return of(p[v], residual ? draft(v) : 0.0f); }
};

__device__ __forceinline__ double inclusive(double v)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += y;
    }
    return v;
}

// First index in [v0, v1) whose cumulative weight, from `c` on, passes the
// mark; where rounding leaves it a last bit short, the last with any weight.
// 512 weights at a time: read side by side, then through shared memory to
// lanes of 16 consecutive ones each: the lane that holds the index has it in
// registers.
struct Turn {
    double w[BLOCK * (32 + 2)];                // 16 weights and a gap
};
__device__ __forceinline__ int search(const Weights &w, Turn &turn, int v0, int v1, double c, double mark)
{
    const int lane = threadIdx.x & 31;
    int last = v0;
    for (int v = v0; v < v1; v += 32 * BLOCK) {
        float p[BLOCK], q[BLOCK];                                      // all on their way before the first store
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) {
            const int j = v + 32 * i + lane;
            p[i] = j < v1 ? w.p[j] : 0.0f;
            q[i] = w.residual && j < v1 ? w.draft(j) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) {
            const int j = 32 * i + lane;
            turn.w[j + j / BLOCK] = w.of(p[i], q[i]);
        }
        __syncwarp();
        double x[BLOCK], sum = 0.0;
#pragma unroll
        for (int i = 0; i < BLOCK; ++i) {
            x[i] = turn.w[(BLOCK + 1) * lane + i];
            sum += x[i];
        }
        __syncwarp();
        const double upto = inclusive(sum);
        const unsigned over = __ballot_sync(~0u, c + upto > mark && sum > 0.0), some = __ballot_sync(~0u, sum > 0.0);
        if (some) {                                                    // the lane that holds the index, or the last with any weight
            const int holder = over ? __ffs(over) - 1 : 31 - __clz(some);
            int at = -1, any = 0;
            if (lane == holder) {
                double run = c + (upto - sum);
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    run += x[i];
                    if (x[i] > 0.0) any = i;
                    if (x[i] > 0.0 && at < 0 && run > mark) at = i;
                }
            }
            last = v + BLOCK * holder + __shfl_sync(~0u, over && at >= 0 ? at : any, holder);
            if (over) return last;
        }
        c += __shfl_sync(~0u, upto, 31);
    }
    return last;
}

__global__ void __launch_bounds__(THREADS, 2) verify_kernel(VerifyArgs a)
{
    __shared__ double part[WARPS];
    __shared__ double cta_sum[2];
    __shared__ int accepted_s;
    __shared__ Turn turn;
    cg::cluster_group cluster = cg::this_cluster();
    const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / nc, K = a.max_draft, V = a.vocab;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependents();

    int nd = a.n_draft[b];
    const float u_last = a.u[(size_t)b * (K + 1) + K];
    if (warp == 0) {                                                   // one lane a draft: K <= 31
        int x = -1;
        float u = 0.0f, p = 0.0f, q = 1.0f;
        if (lane < K) {
            x = a.draft[(size_t)b * K + lane];
            u = a.u[(size_t)b * (K + 1) + lane];
            if (x >= 0 && x < V) {
                p = a.target[((size_t)b * (K + 1) + lane) * V + x];
                if (a.probs) q = a.probs[((size_t)b * K + lane) * V + x];
            }
        }
        if (rank == 0 && lane < min(nd, K) && (x < 0 || x >= V)) set_error(a.error, CSA2_DEV_BAD_INDEX);
        const bool kept = lane < min(nd, K) && x >= 0 && x < V && (double)u * (double)q < (double)p;
        const int n = __ffs(__ballot_sync(~0u, !kept)) - 1;            // lane 31 keeps nothing
        if (lane == 0) accepted_s = n;
    }
    if (nd < 0 || nd > K) {
        if (rank == 0 && threadIdx.x == 0) set_error(a.error, CSA2_DEV_BAD_REQUEST);
        nd = max(0, min(nd, K));
    }
    __syncthreads();
    const int n = accepted_s;
    Weights w;
    w.p = a.target + ((size_t)b * (K + 1) + n) * V;
    w.residual = n < nd;
    w.q = w.residual && a.probs ? a.probs + ((size_t)b * K + n) * V : nullptr;
    w.x = w.residual ? a.draft[(size_t)b * K + n] : -1;

    // piece of this warp: contiguous, whole blocks of 512; lane i keeps the sum of its i-th run of blocks
    const int blocks = (V + nc * WARPS * BLOCK * 32 - 1) / (nc * WARPS * BLOCK * 32), run = (blocks + 31) / 32 * BLOCK * 32;
    const int per = blocks * BLOCK * 32;
    const int64_t begin = (int64_t)(rank * WARPS + warp) * per;
    const int v0 = (int)min((int64_t)V, begin), v1 = (int)min((int64_t)V, begin + per);
    double before = 0.0, after = 0.0, total = 0.0, upto = 0.0, sums = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        sums = 0.0;
        for (int r = 0; v0 + (int64_t)r * run < v1; ++r) {
            double s = 0.0;
            const int e = min(v1, v0 + (r + 1) * run);
            for (int v = v0 + r * run + lane; v < e; v += 32 * BLOCK) {
                float pv[BLOCK], qv[BLOCK];
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    const int j = v + 32 * i;
                    pv[i] = j < e ? w.p[j] : 0.0f;
                    qv[i] = w.residual && j < e ? w.draft(j) : 0.0f;
                }
                // the weights, then their sums; low: what each subtraction and addition rounded off
                float low[BLOCK];
#pragma unroll
                for (int i = 0; i < BLOCK; ++i) {
                    low[i] = 0.0f;
                    if (w.residual) {
                        const float d = pv[i] - qv[i];
                        const bool some = pv[i] > qv[i];
                        low[i] = some ? (pv[i] - d) - qv[i] : 0.0f;    // exact for p > q >= 0 (Dekker)
                        pv[i] = some ? d : 0.0f;
                    } else {
                        pv[i] = fmaxf(pv[i], 0.0f);                    // a NaN too
                    }
                }
#pragma unroll
                for (int i = BLOCK / 2; i > 0; i >>= 1)
#pragma unroll
                    for (int j = 0; j < i; ++j) {
                        const float t = pv[j] + pv[j + i];
                        low[j] += low[j + i] + lost(pv[j], pv[j + i], t);
                        pv[j] = t;
                    }
                s += (double)pv[0] + (double)low[0];
            }
            if (!(s < INFINITY)) {                                     // an infinite weight, or sums past fp32's range
                s = 0.0;
                for (int v = v0 + r * run + lane; v < e; v += 32) s += w(v);
            }
            s = warp_sum(s);
            if (lane == r) sums = s;
        }
        upto = inclusive(sums);
        if (lane == 31) part[warp] = upto;
        __syncthreads();
        if (warp == 0) {
            const double t = inclusive(lane < WARPS ? part[lane] : 0.0);
            if (lane == 31) cta_sum[pass] = t;
        }
        cluster.sync();
        const double theirs = lane < nc ? *cluster.map_shared_rank(&cta_sum[pass], lane) : 0.0;
        total = 0.0;
        for (int r = 0; r < nc; ++r) {                                 // one after another: CTAs meet without a gap
            if (r == rank) before = total;
            total += __shfl_sync(~0u, theirs, r);
            if (r == rank) after = total;
        }
        if (total > 0.0 || !w.residual) break;
        w.residual = false;                                            // p <= q everywhere: what is left is p itself
        __syncthreads();                                               // part is read
    }
    // The others may still be reading this CTA's sum: it stays until all have arrived here.
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // The CTA whose sums straddle the mark holds the drawn index; in it, the
    // first warp whose running end passes the mark, or, where the warps' sums
    // round a last bit below the CTA's, the last warp with any weight; in that
    // the run of blocks, likewise.  Without a finite positive total (rows of
    // zeros, NaN) it is the last token.
    const double mark = fmin(fmax((double)u_last, 0.0), 1.0 - 0x1p-24) * total;
    int *tokens = a.tokens + (size_t)b * (K + 1);
    if (total > 0.0 && total < INFINITY) {
        if (before <= mark && mark < after) {
            const double here = lane < WARPS ? part[lane] : 0.0, end = before + inclusive(here);
            const unsigned over = __ballot_sync(~0u, end > mark && here > 0.0), any = __ballot_sync(~0u, here > 0.0);
            const int chosen = over ? __ffs(over) - 1 : 31 - __clz(any);
            if (warp == chosen) {
                const double start = __shfl_sync(~0u, end - here, chosen);
                const unsigned o = __ballot_sync(~0u, start + upto > mark && sums > 0.0), s = __ballot_sync(~0u, sums > 0.0);
                const int r = o ? __ffs(o) - 1 : 31 - __clz(s);
                const double c = start + __shfl_sync(~0u, upto - sums, r);
                const int x = search(w, turn, v0 + r * run, min(v1, v0 + (r + 1) * run), c, mark);
                if (lane == 0) tokens[n] = x;
            }
        }
    } else if (rank == 0 && threadIdx.x == 0) {
        set_error(a.error, CSA2_DEV_BAD_REQUEST);
        tokens[n] = V - 1;
    }
    if (rank == 0 && threadIdx.x <= K && (int)threadIdx.x != n)
        tokens[threadIdx.x] = (int)threadIdx.x < n ? a.draft[(size_t)b * K + threadIdx.x] : -1;
    if (rank == 0 && threadIdx.x == 0) a.n_accepted[b] = n;
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st)
{
    // As many CTAs to a request as can all be at work (two on each of 148
    // SMs), and no more than its row has blocks for.  64 rows of 131072: 17.3
    // us with 4, 18.3 with 2, 21.9 with 8; 8 of 100003: 8.6 with 8, 11.6 with
    // 4; 2 of 16384: 6.4 with 2, 6.6 with 4 or 8, 7.8 with 1.
    int nc = MAX_CLUSTER;
    while (nc > 1 && ((int64_t)a.batch * nc > 2 * 148 || a.vocab < nc * WARPS * 32 * BLOCK / 2)) nc /= 2;
    LaunchScope scope(-1, st);
    return launch_pdl_cluster(verify_kernel, dim3((unsigned)a.batch * nc), dim3(THREADS), 0, st, nc, a);
}

}  // namespace csa2
