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
// score passes it by 2^8, so the usual tile has no reduction over keys; the
// weights stay below 2^8, and l and O are fp32.  The sums l stay in registers
// per key slot and are reduced once per tile of rows.
//
// P is rounded to bf16 for the second product (relative 2^-9, below the bf16
// output's own step); for an fp32 output it is split into two bf16 parts
// (2^-17) and the product taken twice.
//
// Roles: eight warps do the softmax and the output, one warp plans the row
// tiles and issues the TMA loads, one issues the MMAs.  A 128-dim chunk of
// the latents is refilled as soon as its second product is done, and the next
// S starts on the chunks that have arrived.
//
// Few rows, many keys: the (row tile, key tile) units are dealt out evenly to
// the SMs, a row tile may be shared by several, and a second kernel joins the
// parts.  Many rows: whole row tiles, dealt round robin.
#include "common.cuh"
#include "serve.cuh"
#include "umma.cuh"

namespace csa2 {
using namespace umma;

namespace {

constexpr int D = CSA2_LATENT;
constexpr int KT = 128;                        // keys per tile
constexpr int RT = 64;                         // rows per tile
constexpr int SOFT_WARPS = 8;
constexpr int THREADS = (SOFT_WARPS + 2) * 32;
constexpr int K_SLAB = KT * 128;               // 64 channels of the keys: 16 KB
constexpr int Q_SLAB = RT * 128;               // 8 KB
constexpr int P_BYTES = KT * 128;              // [key][row] bf16, 16 KB
constexpr int CHUNKS = 4;                      // of 128 channels
constexpr int K_OFF = 0, Q_OFF = 8 * K_SLAB, P_OFF = Q_OFF + 8 * Q_SLAB;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t S_COL = 256, O_COL = 0;
constexpr uint32_t IDESC_S = idesc_f16(KT, RT, true, false, false);
constexpr uint32_t IDESC_O = idesc_f16(128, RT, true, true, true);
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float RISE = 8.0f;                   // how far (in log2) a score may pass the reference
constexpr int MAX_SPLIT_TILES = 2 * THREADS;   // row tiles that the split path plans in every CTA

struct Segment {                               // n consecutive key tiles of one row tile
    int tile, n, key0;                         // key0: first key of the first of them
    int max_lo, min_hi;                        // keys in [max_lo, min_hi) are seen by every live row
    int slot;                                  // partial result's slot, -1: the segment is the whole row tile
};

struct Misc {
    uint64_t q_full, q_empty, k_full[CHUNKS], k_empty[CHUNKS], s_full, p_full, o_full, seg_full[2], seg_empty[2], drain;
    Segment seg[2];
    int lo[2][RT], hi[2][RT];
    float muse[RT], lim[RT], fac[RT];
    uint32_t tmem;
    int abort;
    int64_t first_unit, n_units;               // split path: this CTA's share
    int first_tile, first_at;
    int scan[THREADS / 32];
};
constexpr size_t smem_bytes(bool split_p) { return P_OFF + (split_p ? 2 : 1) * P_BYTES + sizeof(Misc); }
static_assert(smem_bytes(true) <= 232448, "shared memory of one CTA");

struct Args {
    const int32_t *cu_q, *cu_k;
    int batch, n_q, n_k, heads, window, tiles;
    float scale;
    void *out;
    float *lse;
    int32_t *error;
    float *part_o;                             // [slots][RT][D]
    float2 *part_ml;                           // [slots][RT]
    int32_t *prefix;                           // [tiles + 1] units before a row tile
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

// Keys [lo, hi) of token t of request b: within [0, n_k] and hi >= lo however
// the prefix sums look, non-decreasing in t where they are sound.
__device__ __forceinline__ void key_range(const Args &a, int b, int t, int &lo, int &hi)
{
    const int64_t q1 = __ldg(a.cu_q + b + 1);
    const int64_t k0 = max(0, min(a.n_k, __ldg(a.cu_k + b))), k1 = max(0, min(a.n_k, __ldg(a.cu_k + b + 1)));
    const int64_t end = max(k0, min(k1, k1 - (q1 - t) + 1));
    hi = (int)end;
    lo = (int)(a.window > 0 ? max(k0, end - a.window) : k0);
}

// Key tiles of a row tile, 0 if it has no live row; key0 gets the first key
// of tile `which`.  The ranges of one request's tokens join without gaps, so
// the walk goes request by request and skips what lies between.
__device__ __forceinline__ int key_tiles(const Args &a, int live, int tile, int which, int &key0)
{
    int t = (int)((int64_t)tile * RT / a.heads);
    key0 = 0;
    if (t >= live) return 0;
    const int t1 = (int)min((int64_t)live - 1, ((int64_t)tile * RT + RT - 1) / a.heads);
    int n = 0, p = 0;
    for (int b = request_of(a, t); t <= t1; ++b) {
        if (b < a.batch - 1 && __ldg(a.cu_q + b + 1) <= t) continue;   // an empty request
        const int e = b < a.batch - 1 ? max(t, min(t1, __ldg(a.cu_q + b + 1) - 1)) : t1;
        int lo, hi, lo1;
        key_range(a, b, t, lo, hi);
        if (e > t) key_range(a, b, e, lo1, hi);
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

// The next key tile: behind this one, or where the first row with keys left begins.
__device__ __forceinline__ int next_tile(const int *lo, const int *hi, int key0, int &row)
{
    key0 += KT;
    while (row < RT && hi[row] <= key0) ++row;
    return row < RT ? max(key0, lo[row]) : key0;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait that gives up after a limit, or as soon as another role has.
__device__ __forceinline__ bool wait(Misc *m, uint64_t *bar, uint32_t parity)
{
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255) == 255 && *reinterpret_cast<volatile int *>(&m->abort)) return false;
    }
    *reinterpret_cast<volatile int *>(&m->abort) = 1;
    return false;
}

__device__ __forceinline__ bool warp_wait(Misc *m, uint64_t *bar, uint32_t parity)
{
    return __all_sync(~0u, wait(m, bar, parity));
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
template <bool SPLIT>
__device__ void producer(const Args &a, Misc *m, uint8_t *sm, const CUtensorMap *map_q, const CUtensorMap *map_k)
{
    const int lane = threadIdx.x & 31;
    const int live = live_tokens(a);
    int tile = SPLIT ? m->first_tile : a.tiles - 1 - (int)blockIdx.x, at = SPLIT ? m->first_at : 0;
    int64_t left = SPLIT ? m->n_units : 0;
    uint32_t unit = 0, s = 0;
    for (;; ++s) {
        Segment g = {-1, 0, 0, 0, 0, -1};
        if (SPLIT) {
            for (; left > 0 && tile < a.tiles; ++tile, at = 0) {
                const int total = key_tiles(a, live, tile, at, g.key0);
                if (total - at <= 0) continue;
                g.tile = tile;
                g.n = (int)min(left, (int64_t)(total - at));
                if (g.n < total) g.slot = 2 * blockIdx.x + (s == 0 ? 0 : 1);
                left -= g.n;
                ++tile;
                at = 0;
                break;
            }
        } else {
            for (; tile >= 0; tile -= gridDim.x) {
                const int total = key_tiles(a, live, tile, 0, g.key0);
                if (total == 0) continue;
                g.tile = tile;
                g.n = total;
                tile -= gridDim.x;
                break;
            }
        }
        const uint32_t r = s & 1;
        bool ok = warp_wait(m, &m->seg_empty[r], ((s >> 1) & 1) ^ 1);
        if (ok && g.tile >= 0) {
            int max_lo = 0, min_hi = INT32_MAX;
#pragma unroll
            for (int i = lane; i < RT; i += 32) {
                const int64_t row = (int64_t)g.tile * RT + i;
                const int t = (int)min(row / a.heads, (int64_t)INT32_MAX);
                int lo = 0, hi = -1;                                   // hi < 0: no such row
                if (t < live) {
                    key_range(a, request_of(a, t), t, lo, hi);
                    if (hi <= lo) lo = hi = 0;                         // no keys
                    max_lo = max(max_lo, lo);
                    min_hi = min(min_hi, hi);
                }
                m->lo[r][i] = lo;
                m->hi[r][i] = hi;
            }
            g.max_lo = __reduce_max_sync(~0u, max_lo);
            g.min_hi = __reduce_min_sync(~0u, min_hi);
        }
        if (ok && lane == 0) m->seg[r] = g;
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&m->seg_full[r]);
        if (ok && g.tile < 0) return;

        ok = ok && warp_wait(m, &m->q_empty, (s & 1) ^ 1);
        if (ok && lane == 0) {
            mbar_arrive_expect_tx(&m->q_full, 8 * Q_SLAB);
            for (int i = 0; i < 8; ++i) tma_load_2d(sm + Q_OFF + i * Q_SLAB, map_q, 64 * i, g.tile * RT, &m->q_full);
        }
        int key0 = g.key0, row = 0;
        for (int k = 0; ok && k < g.n; ++k, ++unit, key0 = next_tile(m->lo[r], m->hi[r], key0, row)) {
            for (int c = 0; c < CHUNKS; ++c) {
                ok = warp_wait(m, &m->k_empty[c], (unit & 1) ^ 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&m->k_full[c], 2 * K_SLAB);
                    for (int i = 2 * c; i < 2 * c + 2; ++i)
                        tma_load_2d(sm + K_OFF + i * K_SLAB, map_k, 64 * i, key0, &m->k_full[c]);
                }
            }
        }
        if (!ok) {                                                     // gave up: no copy may be in flight at exit
            for (int parity = 0; parity < 2; ++parity) {
                mbar_wait(&m->q_full, parity, 1u << 16);
                for (int c = 0; c < CHUNKS; ++c) mbar_wait(&m->k_full[c], parity, 1u << 16);
            }
            return;
        }
    }
}

template <bool SPLIT_P>
__device__ void mma_issuer(Misc *m, uint8_t *sm)
{
    const uint32_t ka = smem_addr(sm + K_OFF), qa = smem_addr(sm + Q_OFF), pa = smem_addr(sm + P_OFF), tb = m->tmem;
    uint32_t unit = 0;
    for (uint32_t s = 0;; ++s) {
        const uint32_t r = s & 1;
        if (!wait(m, &m->seg_full[r], (s >> 1) & 1)) return;
        const int n = m->seg[r].n;
        mbar_arrive(&m->seg_empty[r]);
        if (n == 0) return;
        if (!wait(m, &m->q_full, s & 1)) return;
        for (int k = 0; k < n; ++k, ++unit) {
            for (int c = 0; c < CHUNKS; ++c) {
                if (!wait(m, &m->k_full[c], unit & 1)) return;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int kk = 8 * c + i;
                    mma_ss(tb + S_COL, smem_desc(ka + (kk >> 2) * K_SLAB + (kk & 3) * 32, 16, 1024),
                           smem_desc(qa + (kk >> 2) * Q_SLAB + (kk & 3) * 32, 16, 1024), IDESC_S, kk > 0 ? 1u : 0u);
                }
            }
            mma_commit(&m->s_full);
            if (k == n - 1) mma_commit(&m->q_empty);
            if (!wait(m, &m->p_full, unit & 1)) return;
            fence_after_sync();
            for (int c = 0; c < CHUNKS; ++c) {
#pragma unroll
                for (int part = 0; part < (SPLIT_P ? 2 : 1); ++part)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_ss(tb + O_COL + RT * c, smem_desc(ka + 2 * c * K_SLAB + i * 2048, K_SLAB, 1024),
                               smem_desc(pa + part * P_BYTES + i * 2048, 8192, 1024), IDESC_O,
                               (k > 0 || part > 0 || i > 0) ? 1u : 0u);
                mma_commit(&m->k_empty[c]);
            }
            if (k == n - 1) mma_commit(&m->o_full);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <bool SPLIT_P>
__device__ void softmax(const Args &a, Misc *m, uint8_t *sm)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = tid & (KT - 1), half = tid >> 7;                   // key of the tile, 32 of its 64 rows
    const uint32_t tb = m->tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const float sl = a.scale * LOG2E;
    uint8_t *P = sm + P_OFF;
    float *red = reinterpret_cast<float *>(P);                         // [4][RT], while P is not in use
    uint8_t *bad_key = P + 4 * RT * 4;                                 // [2][KT], likewise
    uint32_t unit = 0;
    for (uint32_t s = 0;; ++s) {
        const uint32_t r = s & 1;
        if (soft_any(!wait(m, &m->seg_full[r], (s >> 1) & 1))) return;  // all eight warps leave, or none
        const Segment g = m->seg[r];
        if (g.tile < 0) return;
        const int *lo = m->lo[r] + 32 * half, *hi = m->hi[r] + 32 * half;
        float l[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) l[j] = 0.0f;
        if (tid < RT) {
            m->muse[tid] = 0.0f;
            m->lim[tid] = -INFINITY;
        }
        soft_sync();

        int key0 = g.key0, first_row = 0;
        for (int k = 0; k < g.n; ++k, ++unit, key0 = next_tile(m->lo[r], m->hi[r], key0, first_row)) {
            wait(m, &m->s_full, unit & 1);                             // given up: finish the segment, then leave
            fence_after_sync();
            float x[32];
            {
                uint32_t raw[32];
                tmem_ld32(tb + S_COL + 32 * half, raw);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(raw[j]) * sl;
            }
            const int key = key0 + row;
            bool poison = false;                                       // this key's latent is not finite
            if (key0 < g.max_lo || key0 + KT > g.min_hi) {
                // A latent that is not finite gives no finite score at all.
                // A masked weight of zero would not keep it out of O, so it
                // is cleared, and the rows that do see it become NaN.
                bool all = true;
#pragma unroll
                for (int j = 0; j < 32; ++j) all &= !(fabsf(x[j]) < INFINITY);
                if (soft_any(all)) {
                    bad_key[half * KT + row] = all;
                    soft_sync();
                    poison = bad_key[row] && bad_key[KT + row];
                    soft_sync();
                    if (poison)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4 *>(sm + K_OFF + (4 * half + i) * K_SLAB + row * 128 + 16 * c) =
                                    make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (poison) x[j] = NAN;
                    if (key < lo[j] || key >= hi[j]) x[j] = -INFINITY;
                }
            }
            bool rise = false;
#pragma unroll
            for (int j = 0; j < 32; ++j) rise |= x[j] - m->muse[32 * half + j] > m->lim[32 * half + j];
            if (soft_any(rise)) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = x[j];
                red[(warp & 3) * RT + 32 * half + lane] = columns<true>(v);
                soft_sync();
                if (tid < RT) {
                    const float top = fmaxf(fmaxf(red[tid], red[RT + tid]), fmaxf(red[2 * RT + tid], red[3 * RT + tid]));
                    const bool fresh = m->lim[tid] == -INFINITY;        // no key seen so far
                    const float old = fresh ? -INFINITY : m->muse[tid], now = fmaxf(old, top);
                    m->fac[tid] = now == -INFINITY ? 1.0f : ex2(old - now);
                    m->muse[tid] = now == -INFINITY ? 0.0f : now;
                    m->lim[tid] = now == -INFINITY ? -INFINITY : RISE;
                }
                soft_sync();
                if (k > 0) {                                           // S follows the last O product: O is at rest
#pragma unroll
                    for (int j = 0; j < 32; ++j) l[j] *= m->fac[32 * half + j];
                    for (int c = 0; c < CHUNKS; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tb + O_COL + RT * c + 32 * half, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * m->fac[32 * half + j]);
                        tmem_st32(tb + O_COL + RT * c + 32 * half, o);
                    }
                    tmem_st_wait();
                }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                x[j] = ex2(x[j] - m->muse[32 * half + j]);
                l[j] += x[j];
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t h[4], e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = x[8 * c + 2 * i], p1 = x[8 * c + 2 * i + 1];
                    h[i] = pack2(p0, p1);
                    if (SPLIT_P) e[i] = pack2(p0 - __uint_as_float(h[i] << 16), p1 - __uint_as_float(h[i] & 0xffff0000u));
                }
                const uint32_t off = row * 128 + (((4 * half + c) ^ (row & 7)) << 4);
                *reinterpret_cast<uint4 *>(P + off) = make_uint4(h[0], h[1], h[2], h[3]);
                if (SPLIT_P) *reinterpret_cast<uint4 *>(P + P_BYTES + off) = make_uint4(e[0], e[1], e[2], e[3]);
            }
            fence_proxy_async_smem();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->p_full);
        }

        // ---- output
        wait(m, &m->o_full, s & 1);
        fence_after_sync();
        red[(warp & 3) * RT + 32 * half + lane] = columns<false>(l);
        soft_sync();
        const int64_t row0 = (int64_t)g.tile * RT;
        if (tid < RT) {
            const float sum = (red[tid] + red[RT + tid]) + (red[2 * RT + tid] + red[3 * RT + tid]);
            const bool none = m->lim[tid] == -INFINITY && !(sum != sum);   // no key seen (a NaN sum has seen one)
            if (g.slot >= 0) {
                a.part_ml[(size_t)g.slot * RT + tid] = make_float2(none ? -INFINITY : m->muse[tid], none ? 0.0f : sum);
            } else {
                m->fac[tid] = none ? 0.0f : 1.0f / sum;
                if (a.lse && m->hi[r][tid] >= 0)
                    a.lse[row0 + tid] = none ? -INFINITY : (m->muse[tid] + log2f(sum)) * LN2;
            }
        }
        soft_sync();
        const bool bf16 = !SPLIT_P && g.slot < 0;
        float *out_f = g.slot >= 0 ? a.part_o + (size_t)g.slot * RT * D : (float *)a.out + row0 * D;
        __nv_bfloat16 *out_h = (__nv_bfloat16 *)a.out + row0 * D;
        for (int c = 0; c < CHUNKS; ++c) {
            uint32_t o[32];
            tmem_ld32(tb + O_COL + RT * c + 32 * half, o);
            tmem_ld_wait();
            const int d = 128 * c + (row & 127);
            if (bf16) {
#pragma unroll
                for (int j = 0; j < 32; j += 2) {                      // neighbours swap: two channels of one row each
                    const int q0 = 32 * half + j;
                    const float v0 = __uint_as_float(o[j]) * m->fac[q0], v1 = __uint_as_float(o[j + 1]) * m->fac[q0 + 1];
                    const bool odd = lane & 1;
                    const float got = __shfl_xor_sync(~0u, odd ? v0 : v1, 1);
                    const int q = q0 + odd;
                    if (m->hi[r][q] >= 0)
                        *reinterpret_cast<uint32_t *>(out_h + (size_t)q * D + (d & ~1)) =
                            odd ? pack2(got, v1) : pack2(v0, got);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int q = 32 * half + j;
                    if (m->hi[r][q] >= 0)
                        out_f[(size_t)q * D + d] = __uint_as_float(o[j]) * (g.slot >= 0 ? 1.0f : m->fac[q]);
                }
            }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->seg_empty[r]);
        soft_sync();                                                   // fac, muse and P's scratch are free again
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
    if (lane == 31) m->scan[warp] = x;
    __syncthreads();
    int add = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) add += m->scan[w];
        total += m->scan[w];
    }
    const int mine = add + x - n[0] - n[1];
    if (2 * tid < a.tiles) before[2 * tid] = mine;
    if (2 * tid + 1 < a.tiles) before[2 * tid + 1] = mine + n[0];
    if (tid == 0) before[a.tiles] = total;
    __syncthreads();
    if (blockIdx.x == 0)
        for (int i = tid; i <= a.tiles; i += THREADS) a.prefix[i] = before[i];
    if (tid == 0) {
        const int64_t ctas = min((int64_t)gridDim.x, (int64_t)total);
        int64_t u0 = 0, u1 = 0;
        if (blockIdx.x < ctas) {
            u0 = (int64_t)total * blockIdx.x / ctas;
            u1 = (int64_t)total * (blockIdx.x + 1) / ctas;
        }
        int b = 0, e = a.tiles;
        while (e - b > 1) {
            const int mid = (b + e) >> 1;
            if (before[mid] <= u0) b = mid; else e = mid;
        }
        m->first_tile = b;
        m->first_at = (int)(u0 - before[b]);
        m->n_units = u1 - u0;
    }
}

template <bool SPLIT_P, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
prompt_attend_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k, const Args a)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    Misc *m = reinterpret_cast<Misc *>(sm + P_OFF + (SPLIT_P ? 2 : 1) * P_BYTES);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (smem_addr(sm) & 1023) {                                        // the swizzled tiles need it
        if (tid == 0) set_error(a.error, CSA2_DEV_BAD_REQUEST);
        return;
    }
    if (warp == SOFT_WARPS + 1) tmem_alloc(&m->tmem, TMEM_COLS);
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
        mbar_init(&m->drain, 1);
        for (int r = 0; r < 2; ++r) {
            mbar_init(&m->seg_full[r], 1);
            mbar_init(&m->seg_empty[r], SOFT_WARPS + 1);
        }
        mbar_fence_init();
        m->abort = 0;
        tma_prefetch_map(&map_q);
        tma_prefetch_map(&map_k);
    }
    grid_dependency_wait();
    allow_dependents();
    if (blockIdx.x == 0)                                               // prefix sums that start at 0 and do not fall
        for (int b = tid; b < a.batch; b += THREADS)
            if ((b == 0 && (a.cu_q[0] != 0 || a.cu_k[0] != 0)) || a.cu_q[b + 1] < a.cu_q[b] || a.cu_k[b + 1] < a.cu_k[b] ||
                a.cu_q[b + 1] > a.n_q || a.cu_k[b + 1] > a.n_k)
                set_error(a.error, CSA2_DEV_BAD_REQUEST);
    if (SPLIT) deal_units(a, m, reinterpret_cast<int *>(sm));
    fence_before_sync();
    __syncthreads();
    fence_after_sync();

    if (warp < SOFT_WARPS) {
        softmax<SPLIT_P>(a, m, sm);
    } else if (warp == SOFT_WARPS) {
        if (SPLIT) fence_proxy_async_smem();                           // the plan's scratch lies where the latents land
        producer<SPLIT>(a, m, sm, &map_q, &map_k);
    } else {
        if ((tid & 31) == 0) {
            mma_issuer<SPLIT_P>(m, sm);
            mma_commit(&m->drain);                                     // no MMA may be in flight at exit
            mbar_wait(&m->drain, 0);
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    if (tid == 0 && m->abort) set_error(a.error, CSA2_DEV_TIMEOUT);
    if (warp == SOFT_WARPS + 1) {
        fence_after_sync();
        tmem_dealloc(m->tmem, TMEM_COLS);
    }
}

// Joins the parts of the row tiles that several CTAs of `grid` shared; one row per CTA.
template <bool F32>
__global__ void __launch_bounds__(D / 4) prompt_join_kernel(const Args a, int grid)
{
    grid_dependency_wait();
    allow_dependents();
    const int tile = blockIdx.x / RT, i = blockIdx.x % RT;
    const int64_t total = a.prefix[a.tiles], u0 = a.prefix[tile], u1 = a.prefix[tile + 1];
    const int64_t row = (int64_t)tile * RT + i;
    if (u1 == u0 || row / a.heads >= live_tokens(a)) return;
    const int64_t ctas = min((int64_t)grid, total);
    const int c0 = (int)(((u0 + 1) * ctas - 1) / total), c1 = (int)((u1 * ctas - 1) / total);
    if (c0 == c1) return;                                              // one CTA had all of it
    // A CTA keeps the part of the row tile that it began with in its first slot, a later one in its second.
    auto slot = [&](int c) { return (size_t)2 * c + (total * c / ctas >= u0 ? 0 : 1); };
    float top = -INFINITY;
    for (int c = c0; c <= c1; ++c) top = fmaxf(top, a.part_ml[slot(c) * RT + i].x);
    float sum = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
        const float2 ml = a.part_ml[slot(c) * RT + i];
        if (ml.x == -INFINITY) continue;
        const float w = ex2(ml.x - top);
        const float4 v = *reinterpret_cast<const float4 *>(a.part_o + (slot(c) * RT + i) * D + 4 * threadIdx.x);
        sum += w * ml.y;
        o.x += w * v.x;
        o.y += w * v.y;
        o.z += w * v.z;
        o.w += w * v.w;
    }
    const bool none = top == -INFINITY;
    const float f = none ? 0.0f : 1.0f / sum;
    const size_t at = (size_t)row * D + 4 * threadIdx.x;
    if (F32)
        *reinterpret_cast<float4 *>((float *)a.out + at) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    else
        *reinterpret_cast<uint2 *>((__nv_bfloat16 *)a.out + at) = make_uint2(pack2(o.x * f, o.y * f), pack2(o.z * f, o.w * f));
    if (a.lse && threadIdx.x == 0) a.lse[row] = none ? -INFINITY : (top + log2f(sum)) * LN2;
}

constexpr int CTAS = 148;                      // one per SM
constexpr int SLOTS = 2 * CTAS;

struct Layout {
    size_t o, ml, prefix, bytes;
};
constexpr Layout layout()
{
    Layout l = {};
    l.ml = sizeof(float) * (size_t)SLOTS * RT * D;
    l.prefix = l.ml + sizeof(float2) * (size_t)SLOTS * RT;
    l.bytes = (l.prefix + sizeof(int32_t) * (MAX_SPLIT_TILES + 1) + 255) & ~(size_t)255;
    return l;
}

int64_t row_tiles(int64_t n_q, int heads) { return (n_q * heads + RT - 1) / RT; }

// [rows][512] bf16 in boxes of 64 channels x box_rows, 128-byte swizzled.
bool make_map(CUtensorMap *m, const void *p, int64_t rows, int64_t stride, int box_rows)
{
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void *)p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <bool SPLIT_P, bool SPLIT>
cudaError_t launch_variant(const CUtensorMap &map_q, const CUtensorMap &map_k, const Args &a, int grid, cudaStream_t st)
{
    static DeviceOnce once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = once.run(dev, [] {
            return cudaFuncSetAttribute(prompt_attend_kernel<SPLIT_P, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)smem_bytes(SPLIT_P));
        });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope(-1, st);
        e = launch_pdl(prompt_attend_kernel<SPLIT_P, SPLIT>, dim3(grid), dim3(THREADS), smem_bytes(SPLIT_P), st, map_q, map_k, a);
    }
    if (e != cudaSuccess || !SPLIT) return e;
    LaunchScope scope(-1, st);
    return launch_pdl(prompt_join_kernel<SPLIT_P>, dim3(a.tiles * RT), dim3(D / 4), 0, st, a, grid);
}

}  // namespace

size_t prompt_workspace_bytes(int64_t n_q, int heads, int64_t n_k)
{
    // one key tile at most, or row tiles enough for every SM: nothing is shared
    return n_k <= KT || row_tiles(n_q, heads) > MAX_SPLIT_TILES ? 256 : layout().bytes;
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
    a.scale = p.scale;
    a.out = p.out;
    a.lse = p.lse;
    a.error = p.error;
    a.part_o = (float *)((char *)p.ws + l.o);
    a.part_ml = (float2 *)((char *)p.ws + l.ml);
    a.prefix = (int32_t *)((char *)p.ws + l.prefix);
    CUtensorMap map_q, map_k;
    // Without keys the latents' map covers a row of q that every mask leaves out.
    if (!make_map(&map_q, p.q, (int64_t)p.n_q * p.heads, D, RT) ||
        !make_map(&map_k, p.n_k ? p.lat : p.q, p.n_k ? p.n_k : 1, p.n_k ? p.lat_stride : D, KT))
        return cudaErrorInvalidValue;
    // Row tiles of one key tile each cannot be shared; many fill the SMs as they are.
    const bool one = p.n_k <= KT || (p.window > 0 && p.window <= KT && p.heads % RT == 0);
    if (!one && a.tiles <= MAX_SPLIT_TILES)
        return p.out_is_fp32 ? launch_variant<true, true>(map_q, map_k, a, CTAS, st)
                             : launch_variant<false, true>(map_q, map_k, a, CTAS, st);
    const int grid = std::min(a.tiles, CTAS);
    return p.out_is_fp32 ? launch_variant<true, false>(map_q, map_k, a, grid, st)
                         : launch_variant<false, false>(map_q, map_k, a, grid, st);
}

}  // namespace csa2
