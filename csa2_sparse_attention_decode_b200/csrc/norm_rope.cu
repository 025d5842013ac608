// Root-mean-square norm of every query head and latent of a token, with the
// position rotation of the last channels in the same pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w
//   (y_a, y_b) <- (y_a cos t - y_b sin t, y_a sin t + y_b cos t),  t = pos * inv_freq_i
//
// for the R/2 channel pairs of the last R channels: neighbours (2i, 2i+1),
// or halves (i, i + R/2).  Sums, norm and rotation are fp32 and each output
// is rounded once.  The angle is formed in fp64 and reduced to a turn before
// the fp32 sine: at position 2^20 an fp32 product is off by up to 0.06 rad.
//
// Bound: 4 bytes per element, read and written once.  A row stays in its
// warp's registers (16 bytes a lane and load), so there is nothing to re-read;
// a CTA computes a token's sines once, in shared memory, for all its heads.
#include "common.cuh"
#include "serve.cuh"

namespace csa2 {
namespace {

constexpr int THREADS = 256;
constexpr int MAX_TOKENS = 8;                  // tokens of one CTA

__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// DIM channels a row; UNROLL rows in flight per lane group.  A CTA takes
// `tokens` consecutive tokens and, of their rows, [y * rows_per_cta, ...).
template <int DIM, int UNROLL>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(NormRopeArgs a, int tokens, int rows_per_cta)
{
    constexpr int CHUNKS = DIM / 8;                                    // 16-byte chunks of a row
    constexpr int LANES = CHUNKS < 32 ? CHUNKS : 32;                   // lanes of a row
    constexpr int CPL = CHUNKS / LANES;                                // chunks a lane
    constexpr int GROUPS = THREADS / LANES;                            // rows in a pass of the CTA
    extern __shared__ float2 turn[];                                   // [tokens][R/2] cosine, sine
    const int l = threadIdx.x & (LANES - 1), g = threadIdx.x / LANES;
    const int half = a.rot_dim / 2;
    grid_dependency_wait();
    allow_dependents();

    const int n = a.n_valid ? max(0, min(a.n, *a.n_valid)) : a.n;
    const int t0 = blockIdx.x * tokens, nt = min(tokens, n - t0);
    if (nt <= 0) return;
    const int per_token = a.heads + a.kv_heads;
    const int r0 = blockIdx.y * rows_per_cta, r1 = min(nt * per_token, r0 + rows_per_cta);

    for (int i = threadIdx.x; i < nt * half; i += THREADS) {
        const int t = i / half;
        double x = (double)a.pos[t0 + t] * (double)a.inv_freq[i - t * half] * 0.15915494309189535;   // 1 / 2 pi
        x -= rint(x);
        float s, c;
        sincospif(2.0f * (float)x, &s, &c);
        if (a.flags & CSA2_ROPE_INVERSE) s = -s;
        turn[i] = make_float2(c, s);
    }
    __syncthreads();

    for (int rb = r0 + g * UNROLL; rb - g * UNROLL < r1; rb += GROUPS * UNROLL) {   // uniform in a warp: shuffles below
        uint4 raw[UNROLL][CPL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int r = rb + u;
            if (r < r1) {
                const int t = r / per_token, h = r - t * per_token;
                const uint16_t *src = h < a.heads ? a.q + (int64_t)(t0 + t) * a.q_stride + (int64_t)h * DIM
                                                  : a.k + (int64_t)(t0 + t) * a.k_stride + (int64_t)(h - a.heads) * DIM;
#pragma unroll
                for (int j = 0; j < CPL; ++j) raw[u][j] = *reinterpret_cast<const uint4 *>(src + 8 * (l + j * LANES));
            } else {
#pragma unroll
                for (int j = 0; j < CPL; ++j) raw[u][j] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int r = rb + u;
            const int t = r / per_token, h = r - t * per_token;
            const bool is_q = h < a.heads;
            float x[CPL][8], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                unpack8(raw[u][j], x[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[j][i] * x[j][i];
            }
            if (!(a.flags & CSA2_ROPE_NO_NORM)) {
#pragma unroll
                for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
                const float inv = rsqrtf(sum * (1.0f / DIM) + a.eps);
                const float *w = is_q ? a.q_weight : a.k_weight;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    const float4 *wp = reinterpret_cast<const float4 *>(w + 8 * (l + j * LANES));
                    const float4 wa = wp[0], wb = wp[1];
                    const float ww[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * inv * ww[i];
                }
            }
            if (half) {
                const float2 *cs = turn + min(t, nt - 1) * half;
                if (!(a.flags & CSA2_ROPE_HALVES)) {
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        const int p0 = (8 * (l + j * LANES) - (DIM - a.rot_dim)) / 2;      // the chunk's first pair
                        if (8 * (l + j * LANES) >= DIM - a.rot_dim) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 v = cs[p0 + i];
                                const float xa = x[j][2 * i], xb = x[j][2 * i + 1];
                                x[j][2 * i] = xa * v.x - xb * v.y;
                                x[j][2 * i + 1] = xa * v.y + xb * v.x;
                            }
                        }
                    }
                } else {
                    // The rotated range starts at a multiple of its own length,
                    // so a chunk's partner is half / 8 chunks away by exclusive or.
                    const int away = half / 8;
                    float y[CPL][8];
#pragma unroll
                    for (int j = 0; j < CPL; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            y[j][i] = away < LANES ? __shfl_xor_sync(~0u, x[j][i], away) : x[CPL - 1 - j][i];
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        const int c0 = 8 * (l + j * LANES) - (DIM - a.rot_dim);
                        if (c0 >= 0) {
                            const bool upper = c0 >= half;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 v = cs[(upper ? c0 - half : c0) + i];
                                x[j][i] = upper ? y[j][i] * v.y + x[j][i] * v.x : x[j][i] * v.x - y[j][i] * v.y;
                            }
                        }
                    }
                }
            }
            if (r >= r1) continue;
            const int64_t row = is_q ? (int64_t)(t0 + t) * a.heads + h : (int64_t)(t0 + t) * a.kv_heads + (h - a.heads);
            uint16_t *dst = is_q ? a.q_out : a.k_out;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const int64_t at = row * DIM + 8 * (l + j * LANES);
                if (dst)
                    *reinterpret_cast<uint4 *>(dst + at) =
                        make_uint4(pack2(x[j][0], x[j][1]), pack2(x[j][2], x[j][3]), pack2(x[j][4], x[j][5]),
                                   pack2(x[j][6], x[j][7]));
                if (!is_q && a.k_out_f32) {
                    float4 *f = reinterpret_cast<float4 *>(a.k_out_f32 + at);
                    f[0] = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
                    f[1] = make_float4(x[j][4], x[j][5], x[j][6], x[j][7]);
                }
            }
        }
    }
}

template <int DIM, int UNROLL>
cudaError_t launch_dim(const NormRopeArgs &a, cudaStream_t st)
{
    constexpr int GROUPS = THREADS / (DIM / 8 < 32 ? DIM / 8 : 32);
    const int per_token = a.heads + a.kv_heads;
    // Enough rows a CTA to pay for its start, few enough to fill 148 SMs.
    int tokens = std::max(1, std::min(MAX_TOKENS, 65536 / (per_token * DIM * 2)));
    tokens = std::max(1, std::min(tokens, a.n / (2 * 148)));
    int split = 1;
    if (a.n < 2 * 148) split = std::max(1, std::min(2 * 148 / a.n, (per_token + GROUPS - 1) / GROUPS));
    const int rows = (tokens * per_token + split - 1) / split;
    LaunchScope scope(-1, st);
    return launch_pdl(norm_rope_kernel<DIM, UNROLL>, dim3((a.n + tokens - 1) / tokens, split), dim3(THREADS),
                      sizeof(float2) * tokens * (a.rot_dim / 2), st, a, tokens, rows);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int dim, cudaStream_t st)
{
    switch (dim) {
    case 64: return launch_dim<64, 2>(a, st);
    case 128: return launch_dim<128, 2>(a, st);
    case 256: return launch_dim<256, 2>(a, st);
    case 512: return launch_dim<512, 2>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace csa2
