// Pages and slots for a batch's new tokens: the page tables, the free-page
// stack and the per-token maps of one step, from the requests' lengths.
//
// Request b holds past = n_tokens[b] tokens and gains (or, negative, drops)
// n_new[b].  With pages(t) = ceil(floor(t / m) / 64) it owns pages(past) and
// needs pages(past + n_new).  Released pages go on the stack in request
// order, then the new pages come off its top, so three prefix sums over the
// batch (released pages, taken pages, granted tokens) place everything.
//
// Bound: 12 bytes written per new token (request, position, slot); a decode
// step's 64 tokens are pure latency (4.8 us, of them 2.5 the launch).  So one
// launch does it all, and no CTA waits for another: each repeats the prefix sums (two loads' latency and
// three block scans) and then takes its share of the tokens.  That works
// because nothing a CTA reads is written in the same launch: a taken page is
// looked up in the old stack, or, above n_free, in the tables of the requests
// that release; the stack grows only above n_free; tables change only past
// the pages owned before; the new n_free goes to another word.
#include "common.cuh"
#include "serve.cuh"

namespace csa2 {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int TOK_PER_THREAD = 4;

// Exclusive prefix sums of two values over the CTA's threads; total gets their
// sums.  `red` is reused by the next call: two barriers keep the calls apart.
struct Pair {
    int64_t a, b;
};
__device__ __forceinline__ Pair block_exclusive(Pair v, Pair *red, Pair &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t a = __shfl_up_sync(~0u, x.a, d), b = __shfl_up_sync(~0u, x.b, d);
        if (lane >= d) {
            x.a += a;
            x.b += b;
        }
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    Pair before = {0, 0}, sum = {0, 0};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) {
            before.a += red[w].a;
            before.b += red[w].b;
        }
        sum.a += red[w].a;
        sum.b += red[w].b;
    }
    total = sum;
    return {before.a + x.a - v.a, before.b + x.b - v.b};
}

// Last index i of a[0 .. n] with a[i] <= x; a is non-decreasing, a[0] <= x < a[n].
__device__ __forceinline__ int segment_of(const int *a, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int m)
{
    return ((tokens >> (m - 1)) + CSA2_PAGE_ENTRIES - 1) / CSA2_PAGE_ENTRIES;
}

__global__ void __launch_bounds__(THREADS) plan_kernel(PlanArgs a)
{
    extern __shared__ int sh[];
    const int B = a.batch;
    int *cu = sh, *taken = cu + B + 1, *rel = taken + B + 1;           // prefix sums
    int *past = rel + B + 1, *owned = past + B, *ratio = owned + B;
    __shared__ Pair red[WARPS];
    grid_dependency_wait();
    allow_dependents();
    const bool first = blockIdx.x == 0;                                // reports and writes what is there once
    const int n_free_in = *a.n_free, n_free = max(0, min(n_free_in, a.n_pages));

    // Each thread owns `per` consecutive requests, so one block scan of the
    // threads' sums gives every request its offset.  Until the last scan cu
    // holds the request's new tokens and taken its new pages; a request with
    // bad data, or one the token rows or the stack cannot serve, has neither.
    const int per = (B + THREADS - 1) / THREADS;
    const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    int64_t s_tok = 0, s_rel = 0;
    Pair total;
    for (int b = b0; b < b1; ++b) {
        const int t = a.n_tokens[b], m = a.m[b];
        int64_t nw = a.n_new[b];
        int code = 0;
        const int64_t cap = (int64_t)a.max_pages * CSA2_PAGE_ENTRIES * m;
        if ((m != 1 && m != 2) || t < 0 || t > cap || t + nw < 0) code = CSA2_DEV_BAD_REQUEST;
        else if (t + nw > cap || t + nw > INT32_MAX) code = CSA2_DEV_CAPACITY;
        if (code && first) set_error(a.error, code);
        const bool bad_past = code == CSA2_DEV_BAD_REQUEST;
        if (code) nw = 0;
        ratio[b] = m == 2 ? 2 : 1;
        past[b] = bad_past ? 0 : t;
        owned[b] = bad_past ? 0 : pages_of(t, m);
        const int need = bad_past ? 0 : pages_of((int)(t + nw), m);
        cu[b] = (int)max((int64_t)0, nw);
        taken[b] = max(0, need - owned[b]);
        rel[b] = max(0, owned[b] - need);
        s_tok += cu[b];
        s_rel += rel[b];
    }
    if (n_free != n_free_in && first && threadIdx.x == 0) set_error(a.error, CSA2_DEV_BAD_REQUEST);
    const Pair start = block_exclusive({s_rel, s_tok}, red, total);
    const int64_t released = total.a;
    int64_t top = n_free + released;
    if (top > a.n_pages) {                                             // more pages than exist: a corrupt table
        if (first && threadIdx.x == 0) set_error(a.error, CSA2_DEV_CAPACITY);
        top = a.n_pages;
    }
    int64_t at = start.b, s_get = 0;
    for (int b = b0; b < b1; ++b) {                                    // token rows: served in order while they last
        at += cu[b];
        if (cu[b] > 0 && at > a.max_new) {
            if (first) set_error(a.error, CSA2_DEV_CAPACITY);
            cu[b] = taken[b] = 0;
        }
        s_get += taken[b];
    }
    at = block_exclusive({s_get, 0}, red, total).a;
    s_tok = s_get = 0;
    for (int b = b0; b < b1; ++b) {                                    // pages: likewise
        at += taken[b];
        if (taken[b] > 0 && at > top) {
            if (first) set_error(a.error, CSA2_DEV_CAPACITY);
            cu[b] = taken[b] = 0;
        }
        s_tok += cu[b];
        s_get += taken[b];
    }
    const Pair granted = block_exclusive({s_tok, s_get}, red, total);
    const int64_t n_tok = total.a, n_get = total.b;
    int64_t at_tok = granted.a, at_get = granted.b, at_rel = start.a;
    for (int b = b0; b < b1; ++b) {
        const int x = cu[b], y = taken[b], z = rel[b];
        cu[b] = (int)at_tok;
        taken[b] = (int)at_get;
        rel[b] = (int)min(at_rel, (int64_t)INT32_MAX);
        at_tok += x;
        at_get += y;
        at_rel += z;
    }
    if (threadIdx.x == 0) {
        cu[B] = (int)n_tok;
        taken[B] = (int)n_get;
        rel[B] = (int)min(released, (int64_t)INT32_MAX);
    }
    __syncthreads();

    // page at stack position p < top, the released ones included
    auto stack_page = [&](int p) {
        int pid;
        if (p < n_free) {
            pid = a.free_pages[p];
        } else {
            const int r = segment_of(rel, B, p - n_free);
            const int need = owned[r] - (rel[r + 1] - rel[r]);
            pid = a.page_table[(size_t)r * a.max_pages + need + (p - n_free - rel[r])];
        }
        if (pid < 0 || pid >= a.n_pages) {
            set_error(a.error, CSA2_DEV_BAD_PAGE);
            pid = -1;
        }
        return pid;
    };

    // Pages from the last thread down, tokens from the first up: in a small
    // step their loads do not wait for one another.
    const int gt = blockIdx.x * THREADS + threadIdx.x, threads = gridDim.x * THREADS, down = threads - 1 - gt;
    for (int k = down; k < (int)top - n_free; k += threads) {          // released pages onto the stack, as many as it has room for
        const int r = segment_of(rel, B, k);
        const int need = owned[r] - (rel[r + 1] - rel[r]);
        a.free_pages[n_free + k] = a.page_table[(size_t)r * a.max_pages + need + (k - rel[r])];
    }
    for (int k = down; k < taken[B]; k += threads) {                   // new pages into the tables
        const int r = segment_of(taken, B, k);
        a.page_table[(size_t)r * a.max_pages + owned[r] + (k - taken[r])] = stack_page((int)top - 1 - k);
    }
    if (first) {
        for (int b = threadIdx.x; b <= B; b += THREADS) a.cu_new[b] = cu[b];
        if (threadIdx.x == 0) *a.n_free_out = (int)(top - n_get);
    }

    // Four consecutive tokens a thread: one search, 16-byte stores.
    const bool wide = ((uintptr_t)a.token_req | (uintptr_t)a.token_pos | (uintptr_t)a.token_slot) % 16 == 0;
    for (int64_t i0 = (int64_t)gt * TOK_PER_THREAD; i0 < n_tok; i0 += (int64_t)threads * TOK_PER_THREAD) {
        const int n = (int)min((int64_t)TOK_PER_THREAD, n_tok - i0);
        int r = segment_of(cu, B, (int)i0);
        int req[TOK_PER_THREAD], pos[TOK_PER_THREAD], slot[TOK_PER_THREAD];
        int page = -1, pid = -1, page_r = -1;
#pragma unroll
        for (int j = 0; j < TOK_PER_THREAD; ++j) {
            if (j >= n) break;
            const int i = (int)i0 + j;
            while (i >= cu[r + 1]) ++r;
            const int p = past[r] + (i - cu[r]);
            const int e = p >> (ratio[r] - 1);
            req[j] = r;
            pos[j] = p;
            if (ratio[r] == 2 && !(p & 1)) {                           // waits for the second token of its pair
                slot[j] = -1;
                continue;
            }
            if (page != e >> 6 || page_r != r) {
                page = e >> 6;
                page_r = r;
                if (page < owned[r]) {
                    pid = a.page_table[(size_t)r * a.max_pages + page];
                    if (pid < 0 || pid >= a.n_pages) {
                        set_error(a.error, CSA2_DEV_BAD_PAGE);
                        pid = -1;
                    }
                } else {
                    pid = stack_page((int)top - 1 - (taken[r] + page - owned[r]));
                }
            }
            slot[j] = pid < 0 ? -1 : pid * CSA2_PAGE_ENTRIES + (e & (CSA2_PAGE_ENTRIES - 1));
        }
        if (n == TOK_PER_THREAD && wide) {
            *reinterpret_cast<int4 *>(a.token_req + i0) = make_int4(req[0], req[1], req[2], req[3]);
            *reinterpret_cast<int4 *>(a.token_pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(a.token_slot + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int j = 0; j < TOK_PER_THREAD; ++j) {
                if (j >= n) break;
                a.token_req[i0 + j] = req[j];
                a.token_pos[i0 + j] = pos[j];
                a.token_slot[i0 + j] = slot[j];
            }
        }
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t st)
{
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const size_t smem_max = sizeof(int) * (6 * CSA2_PLAN_MAX_BATCH + 3);
    if (e == cudaSuccess)
        e = once.run(dev, [=] {
            return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_max);
        });
    if (e != cudaSuccess) return e;
    // 1024 tokens a CTA; and, since releases can be many pages whatever the
    // tokens (300 requests, a quarter of them dropping tokens: 8.3 us with two
    // CTAs, 7.2 with 8 or more), 16 requests a CTA.  More than two CTAs an SM
    // only repeat the prefix sums (295000 tokens: 5.6 us with 296, 7.4 with
    // 592, 13 with 37).
    const int64_t want = std::max(((int64_t)a.max_new + THREADS * TOK_PER_THREAD - 1) / (THREADS * TOK_PER_THREAD),
                                  ((int64_t)a.batch + 15) / 16);
    const int grid = (int)std::min<int64_t>(want, 2 * 148);
    LaunchScope scope(-1, st);
    return launch_pdl(plan_kernel, dim3(grid), dim3(THREADS), sizeof(int) * (6 * (size_t)a.batch + 3), st, a);
}

}  // namespace csa2
