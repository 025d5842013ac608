// Attention of packed prompts over the raw latents, on the 5th-generation
// tensor cores.  Every head shares the token's 512-dim latent, as key and as
// value:  o = sum_j softmax_j(scale q . k_j) k_j  over the keys the row sees,
// a causal range cut to a window.
//
// The rows (token, head) of the packed queries form one matrix; a tile is 64
// consecutive rows, of one token or of several, also of several requests:
// each row carries its own key range [lo, hi), and the tile walks the union,
// 128 keys at a time.  Per key tile, with the latents [128 keys x 512] in
// shared memory once for both products:
//   S^T[128 keys x 64 rows]  = K . Q^T        32 MMAs, fp32 in tensor memory
//   P  = exp2(S * scale * log2 e - m)         one key per thread pair
//   O^T[512 dims x 64 rows] += K^T . P^T      4 chunks of 128 dims, 8 MMAs each
// The transposed products put the 512 output channels on the tensor-memory
// lanes: O takes 256 of its 512 columns and S 64, where 128 rows upright
// would fill all of it with O alone.
//
// Running softmax.  m is a reference, not the maximum: it moves only when a
// score passes it by a factor 2^32, so the usual tile has no reduction over
// keys; the weights stay below 2^32, and l and O are fp32.  The sums l stay in registers
// per key slot and are reduced once per tile of rows.
//
// P is rounded to bf16 for the second product (off by at most 2^-8 of itself,
// as the bf16 output is); for an fp32 output it is split into two bf16 parts
// (2^-16) and the product taken twice.  Doing that for bf16 outputs too would
// take their error from 0.0022 to 0.0017 (windows of 128; 0.0019 to 0.0017
// for 6000 causal tokens) and cost 42 % there, 18 % for ragged decode tokens.
//
// The tensor cores round every sum toward zero: O loses 2^-22 of itself, on
// average, with each key tile, 2^-12 over 131072 latents.  An fp32 output is
// therefore collected in memory, with ordinary additions, every 16 key tiles.
// A bf16 output is not: the loss reaches half a step of it, 2^-8, where one
// CTA takes a row over some 2 million latents.
//
// Roles: eight warps do the softmax and the output, one warp plans the row
// tiles and issues the TMA loads, one issues the MMAs.  A 128-dim chunk of
// the latents is refilled as soon as its second product is done, and the next
// S starts on the chunks that have arrived.
//
// Few rows, many keys: the (row tile, key tile) units are dealt out evenly to
// the SMs, a row tile may be shared by several, and a second kernel joins the
// parts.  Many rows: whole row tiles, dealt round robin.  A window of at most
// one key tile: runs of tokens that slide over a ring of latents.
//
// What bounds it (64 heads, sustained clocks vary from 1.6 to 1.9 GHz):
//   - long causal prompts: shared memory.  An M = 128, N = 64 product reads 6
//     KB of operands, 49 cycles where the arithmetic takes 32, and only 64
//     rows of O fit beside S; then the softmax (about 1200 of 4800 cycles a
//     key tile), during which no latents can be loaded either, for all of
//     shared memory holds the tile in use.  6000 tokens: 2.65 ms, 890 TFLOP/s,
//     0.53 of the measured bf16 rate; 2.76 ms in a loop that lasts.
//   - windows: the chain S, softmax, second product of one token, under the
//     power limit; 16384 tokens x 128 keys: 415 us in short runs, 5.2 TB/s of q
//     and output, 0.81 of the measured copy rate; 490 to 510 us, 4.4 TB/s,
//     0.68, in a loop that lasts.
//   - few rows: memory; one token over 131072 latents 45 us (3.0 TB/s), of
//     which 8 plan and join; 32 tokens over 353600 latents 89 us (4.1 TB/s),
//     94 over inputs that change.
#include "common.cuh"
#include "serve.cuh"
#include "umma.cuh"

namespace csa2 {
using namespace umma;

namespace {

constexpr int D = CSA2_LATENT;
constexpr int KT = 128;                        // keys per tile
constexpr int RT = 64;                         // rows per tile
constexpr int SOFT_WARPS = 8, STORE_WARPS = 4;   // then the producer's warp and the MMAs'
constexpr int LOAD_WARP = SOFT_WARPS + STORE_WARPS, MMA_WARP = LOAD_WARP + 1;
constexpr int THREADS = (MMA_WARP + 1) * 32;
constexpr int K_SLAB = KT * 128;               // 64 channels of the keys: 16 KB
constexpr int Q_SLAB = RT * 128;               // 8 KB
constexpr int P_BYTES = KT * 128;              // [key][row] bf16, 16 KB; twice, for P's low parts or the output's staging
constexpr int CHUNKS = 4;                      // of 128 channels
constexpr int K_OFF = 0, Q_OFF = 8 * K_SLAB, P_OFF = Q_OFF + 8 * Q_SLAB;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 256, O_COL = 0;
constexpr uint32_t IDESC_S = idesc_f16(KT, RT, true, false, false);
constexpr uint32_t IDESC_O = idesc_f16(128, RT, true, true, true);
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float RISE = 32.0f;                  // how far (in log2) a score may pass the reference
constexpr float FRESH = -3.0e38f;              // reference of a row that has seen no key: every score passes it
constexpr int CTAS = 148;                      // one per SM
// Key tiles whose products one O takes for an fp32 output.  1000 tokens over
// 131072 latents are off by 4.6e-6 (7.4e-6 over latents of one sign, which
// pass 1e-5 with 24), uncut by 2.5e-4; 6000 causal tokens take 4.2 ms, 3.7.
constexpr int CUT = 16;
// A share of the units ends at a row tile's border if one is this near: a part
// costs its way through memory and the join (8 ragged tokens 30 us with 2,
// 24 with 0 or 1; 400 tokens after 1000 latents 98 with 1, 101 with 0 or 2).
constexpr int SNAP = 1;
constexpr int MAX_SPLIT_TILES = 2 * THREADS;   // row tiles that the split path plans in every CTA

// How row tiles meet the CTAs.
enum Deal {
    WHOLE,                                     // round robin
    SHARED,                                    // (row tile, key tile) units evenly: a row tile may have several CTAs
    SLIDING                                    // runs of single-token row tiles whose keys fit one key tile
};

// Whether a run of key tiles is cut: a sliding window's is one.
template <bool SPLIT_P, Deal DEAL>
constexpr bool CUTS = SPLIT_P && DEAL != SLIDING;

struct Segment {                               // n consecutive key tiles of one row tile
    int tile, n, key0;                         // key0: first key of the first of them; key key0 + i lies in row
                                               // (i + turn) % 128 of the tile
    int max_lo, min_hi;                        // keys in [max_lo, min_hi) are seen by every live row
    int slot;                                  // partial result's slot, -1: the segment is the whole row tile
    bool uniform : 1;                          // every row sees [max_lo, min_hi), which is not empty
    bool boxed : 1;                            // every row that exists belongs to a request
    bool again : 1, more : 1;                  // an earlier, a later segment has other key tiles of the same run
    uint8_t turn;
};

struct Misc {
    uint64_t q_full, q_empty, k_full[CHUNKS], k_empty[CHUNKS], s_full, p_full, o_full, o_empty, fac_full[2], seg_full[2], seg_empty[2], drain;
    Segment seg[2];
    int lo[2][RT], hi[2][RT];
    alignas(16) float muse[RT], red[4][RT], fac[2][RT];
    uint32_t tmem;
    int abort;
    uint32_t cleared[KT / 32];                 // SLIDING: latents that were not finite and lie in the tile as zeros
};
constexpr size_t SMEM_BYTES = P_OFF + 2 * P_BYTES + sizeof(Misc);
static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");

struct Share {                                 // SHARED: what deal_units() leaves for the producer, in Misc::red
    int units, tile, at;
};

struct Args {
    const int32_t *cu_q, *cu_k;
    int batch, n_q, n_k, heads, window, tiles;
    const uint16_t *lat;
    int64_t lat_stride;
    float scale;
    void *out;
    float *lse;
    int32_t *error;
    float *part_o;                             // [slots][RT][D]
    float2 *part_ml;                           // [slots][RT]
    int4 *shared;                              // [CTAS] row tiles that several CTAs share: tile, first CTA, CTAs (0: none), slot
};

// Tokens of the packed batch that belong to a request; the rows behind them are left alone.
__device__ __forceinline__ int live_tokens(const Args &a) { return max(0, min(a.n_q, __ldg(a.cu_q + a.batch))); }

// Last request with cu_q[b] <= t.
__device__ __forceinline__ int request_of(const Args &a, int t)
{
    int b = 0, e = a.batch;
    while (e - b > 1) {
        const int mid = (b + e) >> 1;
        if (__ldg(a.cu_q + mid) <= t) b = mid; else e = mid;
    }
    return b;
}

// A request: its tokens end before q1, its keys are [k0, k1), all clamped to
// what exists.
struct Request {
    int q1, k0, k1;
};
__device__ __forceinline__ Request request(const Args &a, int b)
{
    return {min(a.n_q, __ldg(a.cu_q + b + 1)), max(0, min(a.n_k, __ldg(a.cu_k + b))), max(0, min(a.n_k, __ldg(a.cu_k + b + 1)))};
}

// Keys [lo, hi) of its token t: within [0, n_k] and hi >= lo however the
// prefix sums look, non-decreasing in t where they are sound.
__device__ __forceinline__ void key_range(const Args &a, const Request &q, int t, int &lo, int &hi)
{
    const int back = max(1, q.q1 - t);                                 // this token and those behind it
    hi = max(q.k0, q.k1 - back + 1);
    lo = a.window > 0 ? max(q.k0, hi - a.window) : q.k0;
}

// Key tiles of a row tile, 0 if it has no live row; key0 gets the first key
// of tile `which`.  The ranges of one request's tokens join without gaps, so
// the walk goes request by request and skips what lies between.
__device__ __forceinline__ int key_tiles(const Args &a, int live, int tile, int which, int &key0)
{
    int t = tile * RT / a.heads;
    key0 = 0;
    if (t >= live) return 0;
    const int t1 = min(live - 1, (tile * RT + RT - 1) / a.heads);
    int n = 0, p = 0;
    for (int b = request_of(a, t); t <= t1; ++b) {
        if (b < a.batch - 1 && __ldg(a.cu_q + b + 1) <= t) continue;   // an empty request
        const int e = b < a.batch - 1 ? max(t, min(t1, __ldg(a.cu_q + b + 1) - 1)) : t1;
        const Request q = request(a, b);
        int lo, hi, lo1;
        key_range(a, q, t, lo, hi);
        if (e > t) key_range(a, q, e, lo1, hi);
        p = max(p, lo);
        if (hi > p && hi > lo) {
            const int c = (hi - p + KT - 1) / KT;
            if (which >= n && which < n + c) key0 = p + (which - n) * KT;
            n += c;
            p += c * KT;
        }
        t = e + 1;
    }
    return max(1, n);                                                  // rows without keys are written too
}

// The next key tile: behind this one, or where the first row with keys left
// begins.  A whole warp calls it; lo and hi are non-decreasing over the rows.
__device__ __forceinline__ int next_tile(const Segment &g, const int *lo, const int *hi, int key0)
{
    key0 += KT;
    if (g.uniform || key0 < g.min_hi) return key0;
    const int lane = threadIdx.x & 31;
    const uint32_t a = __ballot_sync(~0u, hi[lane] > key0), b = __ballot_sync(~0u, hi[32 + lane] > key0);
    const int row = a ? __ffs(a) - 1 : b ? 31 + __ffs(b) : -1;
    return row < 0 ? key0 : max(key0, lo[row]);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait that gives up after 2^28 polls or four seconds (a row tile over a
// million keys takes 20 ms), or as soon as another role has.
__device__ __forceinline__ uint64_t nanoseconds()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool wait(Misc *m, uint64_t *bar, uint32_t parity)
{
    uint64_t start = 0;
    for (uint32_t i = 0; i < (1u << 28); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 1023) == 1023) {
            if (*reinterpret_cast<volatile int *>(&m->abort)) return false;
            const uint64_t now = nanoseconds();
            if (start == 0) start = now;
            if (now - start > 4000000000ull) break;
        }
    }
    *reinterpret_cast<volatile int *>(&m->abort) = 1;
    return false;
}
__device__ __forceinline__ bool warp_wait(Misc *m, uint64_t *bar, uint32_t parity)
{
    return __all_sync(~0u, wait(m, bar, parity));
}

// True in one lane of a converged warp, the same each time.  Loads, stores and
// MMAs issue from uniform registers: behind a test of the lane number the
// compiler cannot see that one lane is left, and each issue costs hundreds of
// cycles more.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.b32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(SOFT_WARPS * 32) : "memory"); }
__device__ __forceinline__ bool soft_any(bool v)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, 1, %2, p;\nselp.b32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v), "n"(SOFT_WARPS * 32)
                 : "memory");
    return r != 0;
}

// The two warps that fill a box of the output.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 64;" ::"r"(2 + group) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool v)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %1, 0;\nbar.red.or.pred q, %2, 64, p;\nselp.b32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(2 + group)
                 : "memory");
    return r != 0;
}

// Brings a box to L2 only.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z)
{
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"((uint64_t)map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}
// All but the thread's N newest bulk stores have read their boxes.
template <int N>
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Column sums or maxima of a warp's 32 x 32 values (one row per lane): lane c gets column c's.
template <bool MAX>
__device__ __forceinline__ float columns(float (&v)[32])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const float keep = up ? v[i + d] : v[i], send = up ? v[i] : v[i + d];
            const float got = __shfl_xor_sync(~0u, send, d);
            v[i] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
    return v[0];
}

// ------------------------------------------------------------------ roles
// Plans the CTA's segments and loads their queries and latents.
//
// SLIDING: a token's keys are the last token's, one in and one out.  The tile
// is a ring then: key k lies in row (k - base) % 128, the new latent goes
// over the one that left, and 1 KB comes in a token instead of 128 KB.
template <bool SPLIT_P, Deal DEAL>
__device__ void producer(const Args &a, Misc *m, uint8_t *sm, const CUtensorMap *map_q, const CUtensorMap *map_k)
{
    const int lane = threadIdx.x & 31;
    const int live = live_tokens(a);
    const Share share = *reinterpret_cast<const Share *>(m->red);
    int tile = blockIdx.x, at = 0, last = a.tiles;
    if (DEAL == WHOLE) tile = a.tiles - 1 - tile;                      // later tokens see more: heavy row tiles first
    if (DEAL == SHARED) tile = share.tile, at = share.at;
    if (DEAL == SLIDING) {
        const int64_t tiles = ((int64_t)live * a.heads + RT - 1) / RT;  // not a padded batch's empty end
        tile = (int)(tiles * blockIdx.x / gridDim.x);
        last = (int)(tiles * (blockIdx.x + 1) / gridDim.x);
    }
    int left = DEAL == SHARED ? share.units : 0;
    int runs = 0, rest = 0, resume = 0;                                // CUTS: key tiles of the run behind this segment, its next key
    constexpr Segment NOTHING = {-1, 0, 0, 0, 0, -1, false, false, false, false, 0};
    Segment g = NOTHING;
    uint32_t queries = 0;                                              // loads of them
    Request req = {-1, 0, 0};
    int base = 0, top = -1;                                            // SLIDING: the ring holds keys [top - 128, top)
    uint32_t unit = 0;
    for (uint32_t s = 0;; ++s) {
        const bool again = CUTS<SPLIT_P, DEAL> && rest > 0;
        if (!again) g = NOTHING;
        g.again = again;
        if (again) {                                                   // the run goes on
            g.key0 = resume;
            g.n = rest;
        } else if (DEAL == SHARED) {
            for (; left > 0 && tile < last; ++tile, at = 0) {
                const int total = key_tiles(a, live, tile, at, g.key0);
                if (total - at <= 0) continue;
                g.tile = tile;
                g.n = min(left, total - at);
                if (g.n < total) g.slot = 2 * blockIdx.x + (runs == 0 ? 0 : 1);
                ++runs;
                left -= g.n;
                ++tile;
                at = 0;
                break;
            }
        } else if (DEAL == WHOLE) {
            for (; tile >= 0; tile -= gridDim.x) {
                const int total = key_tiles(a, live, tile, 0, g.key0);
                if (total == 0) continue;
                g.tile = tile;
                g.n = total;
                tile -= gridDim.x;
                break;
            }
        } else if (tile < last) {
            g.tile = tile++;
            g.n = 1;
        }
        if (CUTS<SPLIT_P, DEAL>) {
            rest = max(0, g.n - CUT);
            g.more = rest > 0;
            g.n -= rest;
        }
        int lo[2] = {0, 0}, hi[2] = {-1, -1};                          // hi < 0: no such row
        if (DEAL == SLIDING && g.tile >= 0) {                          // rows of one token
            const int t = g.tile * RT / a.heads;
            if (t >= req.q1) req = request(a, request_of(a, t));       // loads, one after another: once a request
            key_range(a, req, t, lo[0], hi[0]);
            if (hi[0] <= lo[0]) lo[0] = hi[0] = 0;                     // no keys
            lo[1] = g.max_lo = lo[0];
            hi[1] = g.min_hi = hi[0];
            g.uniform = hi[0] > 0;
            g.boxed = true;
        } else if (g.tile >= 0) {
            int max_lo = 0, min_hi = INT32_MAX, min_lo = INT32_MAX, max_hi = -1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = (g.tile * RT + 32 * i + lane) / a.heads;
                if (t < live) {
                    key_range(a, request(a, request_of(a, t)), t, lo[i], hi[i]);
                    if (hi[i] <= lo[i]) lo[i] = hi[i] = 0;             // no keys
                    max_lo = max(max_lo, lo[i]);
                    min_hi = min(min_hi, hi[i]);
                    min_lo = min(min_lo, lo[i]);
                    max_hi = max(max_hi, hi[i]);
                }
            }
            g.max_lo = __reduce_max_sync(~0u, max_lo);
            g.min_hi = __reduce_min_sync(~0u, min_hi);
            g.uniform = __reduce_min_sync(~0u, min_lo) == g.max_lo && __reduce_max_sync(~0u, max_hi) == g.min_hi && g.min_hi > 0;
            g.boxed = (int64_t)live * a.heads >= min((int64_t)(g.tile + 1) * RT, (int64_t)a.n_q * a.heads);
        }
        // SLIDING: what the ring lacks: nothing, the latent that follows, or all
        bool refill = true;
        int fresh = -1;                                                // ring row of the one latent
        uint4 latent[2];
        if (DEAL == SLIDING && g.tile >= 0) {
            refill = top < 0 || g.max_lo < top - KT || g.min_hi > top + 1 || (g.min_hi > top && g.max_lo == top - KT);
            if (refill) {
                base = g.max_lo;
                top = base + KT;
            } else if (g.min_hi > top) {
                // lanes 0-15 hold 16 bytes each of chunks 0 and 2, the others of chunks 1 and 3
                const uint4 *src = reinterpret_cast<const uint4 *>(a.lat + (size_t)top * a.lat_stride) + lane;
                latent[0] = __ldg(src);
                latent[1] = __ldg(src + 32);
                fresh = (top - base) & (KT - 1);
                ++top;
            }
            g.key0 = top - KT;
            g.turn = (uint8_t)((g.key0 - base) & (KT - 1));
        }
        const uint32_t r = s & 1;
        bool ok = warp_wait(m, &m->seg_empty[r], ((s >> 1) & 1) ^ 1);
        if (ok) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m->lo[r][32 * i + lane] = lo[i];
                m->hi[r][32 * i + lane] = hi[i];
            }
        }
        if (ok && lane == 0) m->seg[r] = g;
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&m->seg_full[r]);
        if (ok && g.tile < 0) return;

        if (!again) ok = ok && warp_wait(m, &m->q_empty, (queries++ & 1) ^ 1);
        if (ok && !again && elect_one()) {
            mbar_arrive_expect_tx(&m->q_full, 8 * Q_SLAB);
            tma_load_3d(sm + Q_OFF, map_q, 0, g.tile * RT, 0, &m->q_full);
            // the rows after these come to L2 meanwhile: from memory they would arrive after the last product
            if (DEAL == SLIDING) tma_prefetch_3d(map_q, 0, (g.tile + 1) * RT, 0);
        }
        int key0 = DEAL == SLIDING ? base : g.key0;
        for (int k = 0; ok && k < g.n; ++k, ++unit) {
            const int next = next_tile(g, m->lo[r], m->hi[r], key0);   // before its last load: then lo may be written
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                ok = warp_wait(m, &m->k_empty[c], (unit & 1) ^ 1);
                if (!ok) break;
                if (DEAL == SLIDING && c == 0 && lane < KT / 32) {     // read before the products that are done now
                    if (refill) m->cleared[lane] = 0;
                    else if (fresh >= 0 && lane == fresh >> 5) m->cleared[lane] &= ~(1u << (fresh & 31));
                }
                __syncwarp();
                if (!refill) {
                    if (fresh >= 0 && lane >> 4 == (c & 1)) {
                        const int piece = lane & 15;
                        *reinterpret_cast<uint4 *>(sm + K_OFF + (2 * c + (piece >> 3)) * K_SLAB + fresh * 128 +
                                                   (((piece & 7) ^ (fresh & 7)) << 4)) = latent[c >> 1];
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m->k_full[c]);
                } else if (elect_one()) {
                    mbar_arrive_expect_tx(&m->k_full[c], 2 * K_SLAB);
                    tma_load_3d(sm + K_OFF + 2 * c * K_SLAB, map_k, 0, key0, 2 * c, &m->k_full[c]);
                }
            }
            key0 = next;
        }
        resume = key0;
        if (!ok) {                                                     // gave up: no copy may be in flight at exit
            for (int parity = 0; parity < 2; ++parity) {
                mbar_wait(&m->q_full, parity, 1u << 16);
                for (int c = 0; c < CHUNKS; ++c) mbar_wait(&m->k_full[c], parity, 1u << 16);
            }
            return;
        }
    }
}

// Issues every product.
template <bool SPLIT_P, Deal DEAL>
__device__ void mma_issuer(Misc *m, uint8_t *sm)
{
    // Descriptors of the operands' first steps; a step on adds its bytes / 16.
    const uint64_t k_keys = smem_desc(smem_addr(sm + K_OFF), 16, 1024), q_rows = smem_desc(smem_addr(sm + Q_OFF), 16, 1024);
    const uint64_t k_chans = smem_desc(smem_addr(sm + K_OFF), K_SLAB, 1024), p_rows = smem_desc(smem_addr(sm + P_OFF), 8192, 1024);
    const uint32_t tb = m->tmem;
    uint32_t unit = 0;
    // The next segment is looked up before the last product of this one, so
    // that nothing stands between that product and the next S.
    bool again = false, more = false;                                  // of the segment looked up last
    auto length = [&](uint32_t s) {
        if (!wait(m, &m->seg_full[s & 1], (s >> 1) & 1)) return 0;
        const int n = m->seg[s & 1].n;
        again = CUTS<SPLIT_P, DEAL> && m->seg[s & 1].again;
        more = CUTS<SPLIT_P, DEAL> && m->seg[s & 1].more;
        mbar_arrive(&m->seg_empty[s & 1]);
        return n;
    };
    int n = length(0);
    uint32_t queries = 0;
    for (uint32_t s = 0; n > 0; ++s) {
        if (!again && !wait(m, &m->q_full, queries++ & 1)) return;
        int next = 0;
        for (int k = 0; k < n; ++k, ++unit) {
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
                if (!wait(m, &m->k_full[c], unit & 1)) return;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    mma_ss(tb + S_COL, k_keys + ((2 * c + (i >> 2)) * K_SLAB + (i & 3) * 32) / 16,
                           q_rows + ((2 * c + (i >> 2)) * Q_SLAB + (i & 3) * 32) / 16, IDESC_S, (c > 0 || i > 0) ? 1u : 0u);
            }
            mma_commit(&m->s_full);
            if (k == n - 1) {
                if (!more) mma_commit(&m->q_empty);
                next = length(s + 1);
            }
            if (k == 0 && !wait(m, &m->o_empty, (s & 1) ^ 1)) return;  // the last row tile's output is out of O
            if (!wait(m, &m->p_full, unit & 1)) return;
            fence_after_sync();
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c) {
#pragma unroll
                for (int i = 0; i < (SPLIT_P ? 16 : 8); ++i)
                    mma_ss(tb + O_COL + RT * c, k_chans + (2 * c * K_SLAB + (i & 7) * 2048) / 16,
                           p_rows + ((i >> 3) * P_BYTES + (i & 7) * 2048) / 16, IDESC_O, (k > 0 || i > 0) ? 1u : 0u);
                mma_commit(&m->k_empty[c]);
            }
            if (k == n - 1) mma_commit(&m->o_full);
        }
        n = next;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Channel d, row q of a part lies at part_at(q, d): four rows side by side, so
// that a warp (32 channels) stores 512 bytes at once.
__device__ __forceinline__ size_t part_at(int q, int d)
{
    return ((size_t)((d >> 7) * (RT / 4) + (q >> 2)) * 128 + (d & 127)) * 4 + (q & 3);
}

// 16 lanes x 32 columns: lane t gets, of each 8 columns, columns 2 (t % 4) and
// the next, in rows t / 4 (two registers) and t / 4 + 8 (two more).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : CSA2_R8(0), CSA2_R8(8)
                 : "r"(taddr));
}

// One warp has all of O that it stores in registers, and the factors it
// scales them with: the softmax of the segment after next, which writes the
// factors' other use, starts behind this.
__device__ __forceinline__ void o_read(Misc *m)
{
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&m->o_empty);
}

// The output of a row tile, by four warps of their own: warp w takes channels
// 32 w .. 32 w + 31 of every chunk while the others are at the next row tile.
//
// bf16: O is turned round with stmatrix into boxes of 64 channels x 64 rows,
// which two warps fill and a bulk store takes away.  (Element stores of the same lines, shuffled or staged, took 5500
// cycles a row tile: the next S leaves the shared-memory pipe little time.)
// f32: a warp's 32 channels are a line, stored as they are.
// A part keeps f32 sums, four rows side by side.  Further segments of a run are
// added to what its first one left there, the same thread's words.
template <bool SPLIT_P, Deal DEAL>
__device__ void store(const Args &a, Misc *m, uint8_t *stage, const CUtensorMap *map_out)
{
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, mate = w & 1, group = w >> 1;
    const uint32_t tb = m->tmem + ((uint32_t)(32 * w) << 16) + O_COL;
    // matrix lane / 8 of a stmatrix: 8 channels, x the 8 rows whose addresses the lanes give
    const int put = (lane & 7) * 128 + (((4 * mate + (lane >> 3)) ^ (lane & 7)) << 4);
    for (uint32_t s = 0;; ++s) {
        const uint32_t r = s & 1;
        if (group_any(group, !wait(m, &m->seg_full[r], (s >> 1) & 1))) break;          // both warps leave, or none
        const int tile = m->seg[r].tile, slot = DEAL == SHARED ? m->seg[r].slot : -1;
        const bool boxed = m->seg[r].boxed;
        const uint32_t live[2] = {__ballot_sync(~0u, m->hi[r][lane] >= 0), __ballot_sync(~0u, m->hi[r][32 + lane] >= 0)};
        const bool again = CUTS<SPLIT_P, DEAL> && m->seg[r].again, more = CUTS<SPLIT_P, DEAL> && m->seg[r].more;
        const float *old_fac = reinterpret_cast<const float *>(m->lo[r]);      // softmax leaves them there
        if (!again) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[r]);
        }
        if (tile < 0) break;
        wait(m, &m->fac_full[r], (s >> 1) & 1);
        wait(m, &m->o_full, s & 1);
        fence_after_sync();
        const int64_t row0 = (int64_t)tile * RT;
        const float *fac = m->fac[r];
        if (slot >= 0 || SPLIT_P) {
#pragma unroll 1
            for (int ch = 0; ch < 2 * CHUNKS; ++ch) {
                const int c = ch >> 1, half = ch & 1, d = 128 * c + 32 * w + lane;
                uint32_t o[32];
                float *part = a.part_o + (size_t)max(slot, 0) * RT * D;
                float *out = (float *)a.out + (size_t)(row0 + 32 * half) * D + d;
                float old[32];
                if (again) {
                    if (slot >= 0) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(old + j) = *reinterpret_cast<const float4 *>(part + part_at(32 * half + j, d));
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) old[j] = live[half] >> j & 1 ? out[(size_t)j * D] : 0.0f;
                    }
                }
                tmem_ld32(tb + RT * c + 32 * half, o);
                tmem_ld_wait();
                if (again)
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(fmaf(old[j], old_fac[32 * half + j], __uint_as_float(o[j])));
                if (slot < 0 && !more)
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * fac[32 * half + j]);
                if (ch == 2 * CHUNKS - 1) o_read(m);
                if (slot >= 0) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4 *>(part + part_at(32 * half + j, d)) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (live[half] >> j & 1) out[(size_t)j * D] = __uint_as_float(o[j]);
                }
            }
            __syncwarp();
            if (again && lane == 0) mbar_arrive(&m->seg_empty[r]);
        } else {
            float2 f[8];                                               // of rows 8i + 2 (lane % 4) and the next
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = *reinterpret_cast<const float2 *>(fac + 8 * i + 2 * (lane & 3));
#pragma unroll 1
            for (int c = 0; c < CHUNKS; ++c) {
                uint32_t o[2][2][16];                                  // rows 0-31, 32-63; channels 0-15, 16-31 of the warp's
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tmem_ld_16x32(tb + ((16u * (i & 1)) << 16) + RT * c + 32 * (i >> 1), o[i >> 1][i & 1]);
                tmem_ld_wait();
                if (c == CHUNKS - 1) o_read(m);
                uint8_t *box = stage + group * (RT * 128);
                bulk_wait_read<0>();                                   // the last store has read the box
                group_sync(group);
#pragma unroll
                for (int i = 0; i < 8; ++i) {                          // rows 8i .. 8i+7
                    uint32_t v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = pack2(__uint_as_float(o[i >> 2][k >> 1][4 * (i & 3) + 2 * (k & 1)]) * f[i].x,
                                     __uint_as_float(o[i >> 2][k >> 1][4 * (i & 3) + 2 * (k & 1) + 1]) * f[i].y);
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                                     smem_addr(box + put) + 1024 * i),
                                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
                fence_proxy_async_smem();
                group_sync(group);
                if (boxed) {
                    if (mate == 0 && elect_one()) tma_store_3d(map_out, box, 0, tile * RT, 2 * c + group);
                } else {                                               // some rows belong to no request
#pragma unroll 1
                    for (int q = 32 * mate + (lane >> 3), i = 0; i < 8; ++i, q += 4)
                        if (live[mate] >> (q & 31) & 1)
                            *reinterpret_cast<uint4 *>((uint8_t *)a.out + ((size_t)row0 + q) * (2 * D) + 256 * c + 128 * group +
                                                       16 * (lane & 7)) =
                                *reinterpret_cast<const uint4 *>(box + q * 128 + (((lane & 7) ^ (q & 7)) << 4));
                }
            }
        }
    }
    bulk_wait();
}

template <bool SPLIT_P, Deal DEAL>
__device__ void softmax(const Args &a, Misc *m, uint8_t *sm)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = tid & (KT - 1), half = tid >> 7;                   // key of the tile, 32 of its 64 rows
    const uint32_t tb = m->tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float sl = a.scale == 0.0f ? 1e-30f : a.scale * LOG2E;       // not 0: a masked score stays -inf
    const float masked = sl > 0.0f ? -INFINITY : INFINITY;
    uint8_t *P = sm + P_OFF;
    uint8_t *bad_key = P;                                              // [2][KT], while P is not in use
    const float4 *muse4 = reinterpret_cast<const float4 *>(m->muse + 32 * half);
    uint32_t unit = 0;
    float kept = 0.0f, kept_at = 0.0f;                                 // CUTS: row tid's sum over the run's segments so far, its reference
    for (uint32_t s = 0;; ++s) {
        const uint32_t r = s & 1;
        if (soft_any(!wait(m, &m->seg_full[r], (s >> 1) & 1))) break;  // all eight warps leave, or none; muse and P are free
        const Segment g = m->seg[r];
        if (g.tile < 0) break;
        const int *lo = m->lo[r] + 32 * half, *hi = m->hi[r] + 32 * half;
        const bool again = CUTS<SPLIT_P, DEAL> && g.again, more = CUTS<SPLIT_P, DEAL> && g.more;
        float l[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) l[j] = 0.0f;
        if (!g.uniform && !again && tid < RT) m->muse[tid] = FRESH;

        int key0 = g.key0;
        for (int k = 0; k < g.n; ++k, ++unit, key0 = next_tile(g, m->lo[r], m->hi[r], key0)) {
            // With the segment's first S the factors of two segments ago are free too: its products follow the last
            // one's, which waited until the output warps had read O and those factors.
            wait(m, &m->s_full, unit & 1);                             // given up: finish the segment, then leave
            fence_after_sync();
            float x[32];
            bool exact = k == 0 && !again && !g.uniform;               // find the rows' maxima first
            for (;;) {
                {
                    uint32_t raw[32];
                    tmem_ld32(tb + S_COL + 32 * half, raw);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(raw[j]);
                }
                const bool cleared = DEAL == SLIDING && (m->cleared[0] | m->cleared[1] | m->cleared[2] | m->cleared[3]);
                if (key0 < g.max_lo || key0 + KT > g.min_hi || cleared) {
                    // A latent that is not finite gives no finite score at
                    // all.  A masked weight of zero would not keep it out of
                    // O, so it is cleared, and the rows that do see it become
                    // NaN.  (Queries that are not finite look the same, and
                    // become NaN by themselves.)
                    const int key = key0 + ((row - g.turn) & (KT - 1));
                    float least = INFINITY;
#pragma unroll
                    for (int j = 0; j < 32; ++j) least = fminf(least, fabsf(x[j]));
                    const bool all = !(least < INFINITY);
                    bool poison = cleared && (m->cleared[row >> 5] >> (row & 31) & 1);     // this key's latent is not finite
                    if (soft_any(all)) {
                        bad_key[half * KT + row] = all;
                        soft_sync();
                        bool found = bad_key[row] && bad_key[KT + row];
                        soft_sync();
                        if (DEAL == SLIDING) {                         // the ring goes on to tokens with other queries: look
                            for (int c = 0; c < CHUNKS; ++c) mbar_try_wait(&m->k_full[c], unit & 1);        // long true: orders the loads
                            uint32_t exponent = 0;                     // the largest ones of this half of the latent
                            if (found)
#pragma unroll 1
                                for (int i = 0; i < 4 * K_SLAB; i += i % 128 < 124 ? 4 : K_SLAB - 124) {
                                    const uint8_t *at = sm + K_OFF + 4 * half * K_SLAB + row * 128 + i;
                                    exponent = __vmaxu2(exponent, *reinterpret_cast<const uint32_t *>(at) & 0x7f807f80u);
                                }
                            bad_key[half * KT + row] = (exponent & 0xffffu) == 0x7f80u || exponent >> 16 == 0x7f80u;
                            soft_sync();
                            found = bad_key[row] || bad_key[KT + row];
                            soft_sync();
                        }
                        if (DEAL == SLIDING && found && half == 0) atomicOr(&m->cleared[row >> 5], 1u << (row & 31));
                        poison |= found;
                        if (found)
#pragma unroll 1
                            for (int i = 0; i < 4; ++i)
#pragma unroll 1
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4 *>(sm + K_OFF + (4 * half + i) * K_SLAB + row * 128 + 16 * c) =
                                        make_uint4(0, 0, 0, 0);
                    }
                    if (g.uniform) {                                   // one token's rows: the key is seen by all or none
                        if (poison || key < g.max_lo || key >= g.min_hi) {
                            const float v = key < g.max_lo || key >= g.min_hi ? masked : NAN;
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = v;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (poison) x[j] = NAN;
                            if (key < lo[j] || key >= hi[j]) x[j] = masked;
                        }
                    }
                }
                if (exact) {
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = x[j] * sl;
                    m->red[warp & 3][32 * half + lane] = columns<true>(v);
                    soft_sync();
                    if (tid < RT) {
                        const float top = fmaxf(fmaxf(m->red[0][tid], m->red[1][tid]), fmaxf(m->red[2][tid], m->red[3][tid]));
                        // Only a row whose own score is far above its reference moves it: what another row holds, also
                        // what is not finite, changes no bit of it.
                        const float old = m->muse[tid], now = top - old > RISE ? top : old;
                        m->fac[r][tid] = ex2(old - now);               // fresh and still fresh: 1; now seen: 0
                        m->muse[tid] = now;
                    }
                    soft_sync();
                    if (k > 0) {                                       // S follows the last O product: O is at rest
#pragma unroll
                        for (int j = 0; j < 32; ++j) l[j] *= m->fac[r][32 * half + j];
#pragma unroll 1
                        for (int c = 0; c < CHUNKS; ++c) {
                            uint32_t o[32];
                            tmem_ld32(tb + O_COL + RT * c + 32 * half, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                o[j] = __float_as_uint(__uint_as_float(o[j]) * m->fac[r][32 * half + j]);
                            tmem_st32(tb + O_COL + RT * c + 32 * half, o);
                        }
                        tmem_st_wait();
                    }
                } else if (k == 0 && !again) {
                    // A row's first reference: any score near the maximum will
                    // do, so where all rows see the same keys the first of
                    // them gives it.
                    if (((row - g.turn) & (KT - 1)) == max(key0, g.max_lo) - key0)
#pragma unroll
                        for (int j = 0; j < 32; ++j) m->muse[32 * half + j] = x[j] * sl;
                    soft_sync();
                }
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float4 ma = muse4[2 * c], mb = muse4[2 * c + 1];
                    const float mu[8] = {ma.x, ma.y, ma.z, ma.w, mb.x, mb.y, mb.z, mb.w};
                    uint32_t h[4], e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float &p0 = x[8 * c + 2 * i], &p1 = x[8 * c + 2 * i + 1];
                        p0 = fmaf(p0, sl, -mu[2 * i]);
                        p1 = fmaf(p1, sl, -mu[2 * i + 1]);
                        top = fmaxf(fmaxf(top, p0), p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        h[i] = pack2(p0, p1);
                        if (SPLIT_P) e[i] = pack2(p0 - __uint_as_float(h[i] << 16), p1 - __uint_as_float(h[i] & 0xffff0000u));
                    }
                    const uint32_t off = row * 128 + (((4 * half + c) ^ (row & 7)) << 4);
                    *reinterpret_cast<uint4 *>(P + off) = make_uint4(h[0], h[1], h[2], h[3]);
                    if (SPLIT_P) *reinterpret_cast<uint4 *>(P + P_BYTES + off) = make_uint4(e[0], e[1], e[2], e[3]);
                }
                // A score far above its reference, in any warp: once more, from the maxima.
                if (exact || !soft_any(top > RISE)) break;
                exact = true;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) l[j] += x[j];
            fence_proxy_async_smem();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->p_full);
        }

        // ---- the rows' sums
        m->red[warp & 3][32 * half + lane] = columns<false>(l);
        soft_sync();
        const int64_t row0 = (int64_t)g.tile * RT;
        if (tid < RT) {
            float sum = (m->red[0][tid] + m->red[1][tid]) + (m->red[2][tid] + m->red[3][tid]);
            if (CUTS<SPLIT_P, DEAL>) {
                if (again) {
                    const float old = ex2(kept_at - m->muse[tid]);
                    sum += old * kept;
                    m->lo[r][tid] = __float_as_int(old);               // nobody reads the rows' ranges any more
                }
                kept = sum;
                kept_at = m->muse[tid];
            }
            const bool none = m->muse[tid] == FRESH && !(sum != sum);  // no key seen (a NaN sum has seen one)
            if (!more && g.slot >= 0) {
                a.part_ml[(size_t)g.slot * RT + tid] = make_float2(none ? -INFINITY : m->muse[tid], none ? 0.0f : sum);
            } else if (!more) {
                m->fac[r][tid] = none ? 0.0f : 1.0f / sum;
                if (a.lse && m->hi[r][tid] >= 0)
                    a.lse[row0 + tid] = none ? -INFINITY : (m->muse[tid] + log2f(sum)) * LN2;
            }
        }
        __syncwarp();
        if (lane == 0 && warp < RT / 32) mbar_arrive(&m->fac_full[r]);
        if (lane == 0) mbar_arrive(&m->seg_empty[r]);
    }
}

// Split path: units before every row tile, and this CTA's share of them.
__device__ void deal_units(const Args &a, Misc *m, int *before)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int live = live_tokens(a);
    int n[2], key0;
#pragma unroll
    for (int i = 0; i < 2; ++i) n[i] = 2 * tid + i < a.tiles ? key_tiles(a, live, 2 * tid + i, 0, key0) : 0;
    int x = n[0] + n[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    int *sums = reinterpret_cast<int *>(m->red) + sizeof(Share) / sizeof(int);
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int add = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) add += sums[w];
        total += sums[w];
    }
    const int mine = add + x - n[0] - n[1];
    if (2 * tid < a.tiles) before[2 * tid] = mine;
    if (2 * tid + 1 < a.tiles) before[2 * tid + 1] = mine + n[0];
    if (tid == 0) before[a.tiles] = total;
    __syncthreads();
    // First unit of CTA c: its fair share's, or a near end of the row tile there.
    const int ctas = min((int)gridDim.x, total);
    auto start = [&](int c, int &tile) {
        const int u = c < ctas ? (int)((int64_t)total * c / ctas) : total;
        int b = 0, e = a.tiles;
        while (e - b > 1) {
            const int mid = (b + e) >> 1;
            if (before[mid] <= u) b = mid; else e = mid;
        }
        const int off = u - before[b], rest = before[b + 1] - u;
        const int at = off <= SNAP && off <= rest ? before[b] : rest <= SNAP ? before[b + 1] : u;
        while (b + 1 < a.tiles && before[b + 1] <= at) ++b;
        tile = b;
        return at;
    };
    if (tid == 0) {
        int tile, next;
        const int u0 = start(blockIdx.x, tile), u1 = start(blockIdx.x + 1, next);
        *reinterpret_cast<Share *>(m->red) = {u1 - u0, tile, u0 - before[tile]};
    }
    // For the join, by the first CTA: row tile after row tile, the CTAs that
    // begin inside it.  The one before them has its beginning, as a part in
    // the second of its slots unless it began there.
    int *tiles = before + a.tiles + 1, *starts = tiles + CTAS;
    if (blockIdx.x == 0 && tid < CTAS) {
        int tile;
        starts[tid] = start(tid, tile);
        tiles[tid] = starts[tid] > before[tile] && starts[tid] < total ? tile : -1;    // -1: at a border
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        const int tile = tid < CTAS ? tiles[tid] : -1;
        const bool opens = tile >= 0 && tiles[tid - 1] != tile;        // CTA 0 begins at a border
        const uint32_t mask = __ballot_sync(~0u, opens);
        if (lane == 0) sums[warp] = __popc(mask);
        if (tid < CTAS) a.shared[tid] = make_int4(0, 0, 0, 0);
        __syncthreads();
        if (opens) {
            int rank = __popc(mask & ((1u << lane) - 1)), n = 2;
            for (int w = 0; w < warp; ++w) rank += sums[w];
            while (tid + n - 1 < CTAS && tiles[tid + n - 1] == tile) ++n;
            a.shared[rank] = make_int4(tile, tid - 1, n, 2 * (tid - 1) + (starts[tid - 1] == before[tile] ? 0 : 1));
        }
        __syncthreads();
    }
}

template <bool SPLIT_P, Deal DEAL>
__global__ void __launch_bounds__(THREADS, 1)
prompt_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_out, const Args a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    Misc *m = reinterpret_cast<Misc *>(sm + P_OFF + 2 * P_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (smem_addr(sm) & 1023) {                                        // the swizzled tiles need it
        if (tid == 0) set_error(a.error, CSA2_DEV_BAD_REQUEST);
        return;
    }
    if (warp == MMA_WARP) tmem_alloc(&m->tmem, TMEM_COLS);
    if (tid == 0) {
        mbar_init(&m->q_full, 1);
        mbar_init(&m->q_empty, 1);
        for (int c = 0; c < CHUNKS; ++c) {
            mbar_init(&m->k_full[c], 1);
            mbar_init(&m->k_empty[c], 1);
        }
        mbar_init(&m->s_full, 1);
        mbar_init(&m->p_full, SOFT_WARPS);
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_empty, STORE_WARPS);
        mbar_init(&m->drain, 1);
        for (int r = 0; r < 2; ++r) {
            mbar_init(&m->seg_full[r], 1);
            mbar_init(&m->seg_empty[r], SOFT_WARPS + STORE_WARPS + 1);
            mbar_init(&m->fac_full[r], RT / 32);
        }
        mbar_fence_init();
        m->abort = 0;
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
        tma_prefetch_map(&map_out);
    }
    grid_dependency_wait();
    allow_dependents();
    if (blockIdx.x == 0)                                               // prefix sums that start at 0 and do not fall
        for (int b = tid; b < a.batch; b += THREADS)
            if ((b == 0 && (a.cu_q[0] != 0 || a.cu_k[0] != 0)) || a.cu_q[b + 1] < a.cu_q[b] || a.cu_k[b + 1] < a.cu_k[b] ||
                a.cu_q[b + 1] > a.n_q || a.cu_k[b + 1] > a.n_k)
                set_error(a.error, CSA2_DEV_BAD_REQUEST);
    if (DEAL == SHARED) deal_units(a, m, reinterpret_cast<int *>(sm));
    fence_before_sync();
    __syncthreads();
    fence_after_sync();

    if (warp < SOFT_WARPS) {
        softmax<SPLIT_P, DEAL>(a, m, sm);
    } else if (warp < LOAD_WARP) {
        store<SPLIT_P, DEAL>(a, m, sm + P_OFF + P_BYTES, &map_out);
    } else if (warp == LOAD_WARP) {
        if (DEAL == SHARED) fence_proxy_async_smem();                  // the plan's scratch lies where the latents land
        producer<SPLIT_P, DEAL>(a, m, sm, &map_q, &map_k);
    } else {
        if (elect_one()) {
            mma_issuer<SPLIT_P, DEAL>(m, sm);
            mma_commit(&m->drain);                                     // no MMA may be in flight at exit
            mbar_wait(&m->drain, 0);
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && m->abort) set_error(a.error, CSA2_DEV_TIMEOUT);
    if (warp == MMA_WARP) {
        fence_after_sync();
        tmem_dealloc(m->tmem, TMEM_COLS);
    }
}

// Joins the parts of the row tiles that several CTAs shared.  A CTA takes four
// rows x `chunks` times 128 channels; blockDim.y groups of threads share the
// parts.
constexpr int JOIN_GROUPS = 8;
template <bool F32>
__global__ void __launch_bounds__(128 * JOIN_GROUPS) prompt_join_kernel(const Args a, int chunks)
{
    grid_dependency_wait();
    allow_dependents();
    const int4 job = a.shared[blockIdx.x / (RT / 4)];
    const int tile = job.x, c0 = job.y, n = job.z, first = job.w;
    const int i = 4 * (blockIdx.x % (RT / 4)), group = threadIdx.y, groups = blockDim.y;
    const int64_t row = (int64_t)tile * RT + i, live = (int64_t)live_tokens(a) * a.heads;
    if (n == 0 || row >= live) return;
    // slot of part k; the CTAs behind the first began with theirs
    auto slot = [&](int k) { return (size_t)(k ? 2 * (c0 + k) : first); };
    auto part = [&](int k, int d) {
        return *reinterpret_cast<const float4 *>(a.part_o + slot(k) * RT * D + part_at(i, d));
    };
    int d = 128 * chunks * blockIdx.y + threadIdx.x;
    constexpr int EARLY = 6;                                           // on their way while the weights are formed
    float4 early[EARLY];
#pragma unroll
    for (int j = 0; j < EARLY; ++j) early[j] = group + j * groups < n ? part(group + j * groups, d) : make_float4(0.f, 0.f, 0.f, 0.f);
    __shared__ float weight[4][CTAS], inv[4];
    __shared__ float4 sums[JOIN_GROUPS][128];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (group == 0) {                                                  // warp w: weights of row i + w
        constexpr int N = (CTAS + 31) / 32;
        float2 ml[N];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int k = lane + 32 * j;
            ml[j] = k < n ? a.part_ml[slot(k) * RT + i + warp] : make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, ml[j].x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float w = ml[j].x == -INFINITY ? 0.0f : ex2(ml[j].x - top);
            if (lane + 32 * j < n) weight[warp][lane + 32 * j] = w;
            if (ml[j].x != -INFINITY) sum += w * ml[j].y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        if (lane == 0) {
            const bool none = top == -INFINITY && sum == 0.0f;         // a NaN has seen keys
            inv[warp] = none ? 0.0f : 1.0f / sum;
            if (blockIdx.y == 0 && a.lse && row + warp < live)
                a.lse[row + warp] = none ? -INFINITY : (top + log2f(sum)) * LN2;
        }
    }
    __syncthreads();
    for (int c = 0; c < chunks; ++c, d += 128) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &v, int k) {
            o.x += weight[0][k] * v.x;
            o.y += weight[1][k] * v.y;
            o.z += weight[2][k] * v.z;
            o.w += weight[3][k] * v.w;
        };
#pragma unroll
        for (int j = 0; j < EARLY; ++j)
            if (group + j * groups < n) add(early[j], group + j * groups);
#pragma unroll 8
        for (int k = group + EARLY * groups; k < n; k += groups) add(part(k, d), k);
        if (c + 1 < chunks)
#pragma unroll
            for (int j = 0; j < EARLY; ++j)
                early[j] = group + j * groups < n ? part(group + j * groups, d + 128) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (groups > 1) {
            sums[group][threadIdx.x] = o;
            __syncthreads();
            if (group == 0)
                for (int k = 1; k < groups; ++k) {                     // in order: the same result every time
                    const float4 v = sums[k][threadIdx.x];
                    o.x += v.x;
                    o.y += v.y;
                    o.z += v.z;
                    o.w += v.w;
                }
            __syncthreads();
        }
        if (group > 0) continue;
        const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (row + j >= live) break;
            const size_t at = (size_t)(row + j) * D + d;
            if (F32) ((float *)a.out)[at] = v[j] * inv[j];
            else ((__nv_bfloat16 *)a.out)[at] = __float2bfloat16_rn(v[j] * inv[j]);
        }
    }
}

constexpr int SLOTS = 2 * CTAS;

struct Layout {
    size_t o, ml, shared, bytes;
};
constexpr Layout layout()
{
    Layout l = {};
    l.ml = sizeof(float) * (size_t)SLOTS * RT * D;
    l.shared = l.ml + sizeof(float2) * (size_t)SLOTS * RT;
    l.bytes = (l.shared + sizeof(int4) * CTAS + 255) & ~(size_t)255;
    return l;
}

static_assert(layout().bytes == CSA2_PROMPT_WORKSPACE_MAX, "the most that any call needs");

int64_t row_tiles(int64_t n_q, int heads) { return (n_q * heads + RT - 1) / RT; }

// [rows][512] bf16 as 8 slabs of 64 channels, in boxes of box_rows x box_slabs
// that land slab by slab, 128-byte swizzled.  One load brings a whole chunk:
// a thread gets a load out every 150 cycles at best, and slab by slab the
// loop around them held a key tile back to 3200 cycles, against 1800 for
// 128 KB from L2 into every SM at once.
bool make_map(CUtensorMap *m, const void *p, int64_t rows, int64_t stride, int box_rows, int box_slabs)
{
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, D / 64};
    cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_slabs};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void *)p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <bool SPLIT_P, Deal DEAL>
cudaError_t launch_variant(const CUtensorMap &map_q, const CUtensorMap &map_k, const CUtensorMap &map_out, const Args &a, int grid, cudaStream_t st)
{
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = once.run(dev, [] {
            return cudaFuncSetAttribute(prompt_attend_kernel<SPLIT_P, DEAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)SMEM_BYTES);
        });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope(-1, st);
        e = launch_pdl(prompt_attend_kernel<SPLIT_P, DEAL>, dim3(grid), dim3(THREADS), SMEM_BYTES, st, map_q, map_k, map_out, a);
    }
    if (e != cudaSuccess || DEAL != SHARED) return e;
    LaunchScope scope(-1, st);
    // Few row tiles have many parts each: 148 for one token over 131072
    // latents, joined in 45 us in all by 8 groups (71 by one); 32 tokens'
    // about 5, for which one group is best (89 us, 118 with 8).
    const int tiles = std::min(a.tiles, CTAS - 1), groups = std::max(1, std::min(JOIN_GROUPS, grid / (8 * a.tiles)));
    const int chunks = tiles <= CTAS / 3 ? 1 : CHUNKS;                 // a wave or two of CTAs, most with nothing to do
    return launch_pdl(prompt_join_kernel<SPLIT_P>, dim3(tiles * (RT / 4), CHUNKS / chunks), dim3(128, groups), 0, st, a, chunks);
}

// Whole row tiles, at worst the longest ones on one SM, take about as long as
// planning and joining shared ones would.
bool few_keys(int64_t tiles, int64_t n_k, int window)
{
    return (tiles + CTAS - 1) / CTAS * n_k <= 10 * KT || (window > 0 && window <= 4 * KT);
}

}  // namespace

size_t prompt_workspace_bytes(int64_t n_q, int heads, int64_t n_k)
{
    const int64_t tiles = row_tiles(n_q, heads);
    return few_keys(tiles, n_k, 0) || tiles > MAX_SPLIT_TILES ? 256 : layout().bytes;
}

cudaError_t launch_prompt_attend(const PromptArgs &p, cudaStream_t st)
{
    const Layout l = layout();
    Args a = {};
    a.cu_q = p.cu_q;
    a.cu_k = p.cu_k;
    a.batch = p.batch;
    a.n_q = p.n_q;
    a.n_k = p.n_k;
    a.heads = p.heads;
    a.window = p.window;
    a.tiles = (int)row_tiles(p.n_q, p.heads);
    a.lat = p.lat;
    a.lat_stride = p.lat_stride;
    a.scale = p.scale;
    a.out = p.out;
    a.lse = p.lse;
    a.error = p.error;
    a.part_o = (float *)((char *)p.ws + l.o);
    a.part_ml = (float2 *)((char *)p.ws + l.ml);
    a.shared = (int4 *)((char *)p.ws + l.shared);
    CUtensorMap map_q, map_k, map_out;
    // Without keys the latents' map covers a row of q that every mask leaves out.
    if (!make_map(&map_q, p.q, (int64_t)p.n_q * p.heads, D, RT, 8) ||
        !make_map(&map_out, p.out, (int64_t)p.n_q * p.heads, D, RT, 1) ||        // f32 outputs do not use it
        !make_map(&map_k, p.n_k ? p.lat : p.q, p.n_k ? p.n_k : 1, p.n_k ? p.lat_stride : D, KT, 2))
        return cudaErrorInvalidValue;
    // Sharing evens out few rows or ragged pasts (50 tokens after 4000: 57 us
    // against 88 whole; 32 tokens with pasts of 32 to 16384: 34 against 244),
    // but plans and joins (100 tokens after 1000: 43 against 30); many row
    // tiles with like pasts are even enough dealt round robin (800 tokens after
    // 20000: 2.38 ms shared, 2.45 whole).  With one long past among many short
    // ones they are not, and past MAX_SPLIT_TILES that costs: 131072 latents in
    // one of 1000 requests with 500 each take 2.95 ms, in one of 800, shared,
    // 0.16.  Sliding: one token 9.5 us either way, 4000 tokens 110 against 120.
    const bool sliding = p.window > 0 && p.window <= KT && p.heads % RT == 0;
    if (sliding || few_keys(a.tiles, p.n_k, p.window) || a.tiles > MAX_SPLIT_TILES) {
        const int grid = std::min(a.tiles, CTAS);
        if (sliding)
            return p.out_is_fp32 ? launch_variant<true, SLIDING>(map_q, map_k, map_out, a, grid, st)
                                 : launch_variant<false, SLIDING>(map_q, map_k, map_out, a, grid, st);
        return p.out_is_fp32 ? launch_variant<true, WHOLE>(map_q, map_k, map_out, a, grid, st)
                             : launch_variant<false, WHOLE>(map_q, map_k, map_out, a, grid, st);
    }
    return p.out_is_fp32 ? launch_variant<true, SHARED>(map_q, map_k, map_out, a, CTAS, st)
                         : launch_variant<false, SHARED>(map_q, map_k, map_out, a, CTAS, st);
}

}  // namespace csa2
