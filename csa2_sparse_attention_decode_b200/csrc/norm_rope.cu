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
// warp's registers, so nothing is read twice.  A warp has 2 KB of rows in
// flight (two rows of 512 channels, four of 256, ...), takes a slice of a
// token's rows, and forms the token's sines once for the slice, in its own
// shared memory.  8192 tokens x 65 rows of 512: 187 us, 5.8 TB/s, 0.90 of the
// measured copy rate; 16381 tokens x 33 rows of 128 in halves: 60 us, 4.7 TB/s
// (242 instructions of a warp a KB of rows, 184 with 512 channels, and more wait
// for shared memory; two of fp32 at a time took 3 us off).
#include "common.cuh"
#include "serve.cuh"

namespace csa2 {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

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

// Two fp32 products, or products and sums, in one instruction, each rounded as by itself.
__device__ __forceinline__ void mul2(float &a0, float &a1, float b0, float b1)
{
    asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nmul.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void multiply_add2(float &a0, float &a1, float b0, float b1, float c0, float c1)
{
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nmov.b64 z, {%4, %5};\nfma.rn.f32x2 x, x, y, z;\n"
        "mov.b64 {%0, %1}, x;\n}\n"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void square_add2(float &s0, float &s1, float b0, float b1)
{
    asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %3};\nfma.rn.f32x2 x, y, y, x;\nmov.b64 {%0, %1}, x;\n}\n"
        : "+f"(s0), "+f"(s1)
        : "f"(b0), "f"(b1));
}

// A read that may pass the stores before it, but not the wait for the kernel
// before this one.
__device__ __forceinline__ float4 load_constant(const float *p)
{
    float4 v;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// DIM channels a row.  A step is 1 KB of rows: a lane holds two 16-byte chunks
// of one row, l and l + LANES, so that a row's lanes read and write whole lines.
template <int DIM>
struct Shape {
    static constexpr int CHUNKS = DIM / 8;                             // of a row
    static constexpr int LANES = CHUNKS / 2;                           // of a row
    static constexpr int ROWS = 32 / LANES;                            // of a step
};

// The cosines and sines of two pairs (c, c, s, s) share 16 bytes, and lanes with
// neighbouring chunks, `per` pairs each, read neighbouring ones: the cosine of
// pair p is float turn_at(p), its sine two floats on.
__device__ __forceinline__ int turn_at(int p, int per, int half) { return ((p % per / 2) * (half / per) + p / per) * 4 + (p & 1); }

// A warp forms a token's cosines and sines.  Not inlined: its registers would
// crowd out the rows in flight.
__device__ __noinline__ void fill_turns(float *turn, const float *inv_freq, int half, int per, int pos, float sign)
{
    for (int i = threadIdx.x & 31; i < half; i += 32) {
        double t = (double)pos * (double)inv_freq[i] * 0.15915494309189535;            // 1 / 2 pi
        t -= rint(t);
        float sine, cosine;
        sincospif(2.0f * (float)t, &sine, &cosine);
        float *at = turn + turn_at(i, per, half);
        at[0] = cosine;
        at[2] = sign * sine;
    }
}

// Norm and rotation of one step: x holds chunks l and l + LANES of a row, w the
// weights there.  In halves a channel's partner lies R/2 on: in the lane's
// other chunk where the whole row turns, else, in the row's second half, in
// another lane.  (16381 tokens x 33 rows of 128: 60 us, 67 with 64 channels
// turned.  Lanes that hold both chunks of any pair: 66 either way.)
template <int DIM, bool HALVES>
__device__ __forceinline__ void finish(const NormRopeArgs &a, const uint4 (&raw)[2], float (&x)[2][8], const float (&held)[2][8],
                                       const float *weight, const float4 *turn, const int (&c)[2])
{
    unpack8(raw[0], x[0]);
    unpack8(raw[1], x[1]);
    if (!(a.flags & CSA2_ROPE_NO_NORM)) {
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 2) square_add2(sum[0], sum[1], x[k][i], x[k][i + 1]);
        sum[0] += sum[1];
#pragma unroll
        for (int d = Shape<DIM>::LANES / 2; d > 0; d >>= 1) sum[0] += __shfl_xor_sync(~0u, sum[0], d);
        const float inv = rsqrtf(sum[0] * (1.0f / DIM) + a.eps);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 w = HALVES ? make_float4(held[k][i], held[k][i + 1], held[k][i + 2], held[k][i + 3])
                                        : load_constant(weight + 8 * c[k] + i);
                mul2(x[k][i], x[k][i + 1], inv, inv);
                mul2(x[k][i], x[k][i + 1], w.x, w.y);
                mul2(x[k][i + 2], x[k][i + 3], inv, inv);
                mul2(x[k][i + 2], x[k][i + 3], w.z, w.w);
            }
    }
    if (a.rot_dim == 0) return;
    const int skip = (DIM - a.rot_dim) / 8;                            // chunks before the rotated range
    if (!HALVES) {
        const int chunks = a.rot_dim / 8;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (c[k] < skip) continue;
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float4 v = turn[i / 2 * chunks + c[k] - skip];
                const float a0 = x[k][2 * i], b0 = x[k][2 * i + 1], a1 = x[k][2 * i + 2], b1 = x[k][2 * i + 3];
                x[k][2 * i] = a0 * v.x - b0 * v.z;
                x[k][2 * i + 1] = a0 * v.z + b0 * v.x;
                x[k][2 * i + 2] = a1 * v.y - b1 * v.w;
                x[k][2 * i + 3] = a1 * v.w + b1 * v.y;
            }
        }
    } else if (a.rot_dim == DIM) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 v = turn[i / 2 * Shape<DIM>::LANES + c[0]];
            float s0 = x[0][i], s1 = x[0][i + 1], t0 = x[1][i], t1 = x[1][i + 1];      // a s and -b s
            mul2(s0, s1, v.z, v.w);
            mul2(t0, t1, -v.z, -v.w);
            multiply_add2(x[0][i], x[0][i + 1], v.x, v.y, t0, t1);
            multiply_add2(x[1][i], x[1][i + 1], v.x, v.y, s0, s1);
        }
    } else {
        const int chunks = a.rot_dim / 16, at = (c[1] - skip) & (chunks - 1);          // of half the range
        const bool turns = c[1] >= skip;
        const float sign = c[1] - skip < chunks ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float t0 = __shfl_xor_sync(~0u, x[1][i], chunks), t1 = __shfl_xor_sync(~0u, x[1][i + 1], chunks);
            if (!turns) continue;
            const float4 v = turn[i / 2 * chunks + at];
            mul2(t0, t1, sign * v.z, sign * v.w);
            multiply_add2(x[1][i], x[1][i + 1], v.x, v.y, t0, t1);
        }
    }
}

// `slices` warps share a token; a warp takes every slices-th of its steps,
// queries first, then latents.
template <int DIM, bool HALVES>
__global__ void __launch_bounds__(THREADS, 4) norm_rope_kernel(NormRopeArgs a, int slices, int q_steps, int steps)
{
    using S = Shape<DIM>;
    extern __shared__ __align__(16) float turns[];                     // [WARPS][R] cosines and sines
    const int lane = threadIdx.x & 31, l = lane & (S::LANES - 1), sub = lane / S::LANES;
    const int half = a.rot_dim / 2, per = HALVES ? 8 : 4;
    const int c[2] = {l, l + S::LANES};
    float *turn = turns + (threadIdx.x >> 5) * a.rot_dim;
    grid_dependency_wait();
    allow_dependents();

    const int n = a.n_valid ? max(0, min(a.n, *a.n_valid)) : a.n;
    const int64_t items = (int64_t)n * slices;
    // The weights: neighbours read them from L1 at each step, which leaves
    // registers (8192 tokens x 65 rows of 512: 186 us, held 194; 64 tokens
    // 4.3, held 4.1); halves, whose rotation fills the registers either way,
    // hold them (16381 tokens x 33 rows of 128: 60 us, from L1 64).
    float held[2][8] = {};
    int weights_of = -1;                                               // 1: of the queries, 0: of the latents
    for (int64_t item = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5); item < items; item += (int64_t)gridDim.x * WARPS) {
        const int token = (int)(item / slices), slice = (int)(item - (int64_t)token * slices);
        bool turned = half == 0;
        for (int step = slice; step < steps;) {
            const bool is_q = step < q_steps;
            const int heads = is_q ? a.heads : a.kv_heads, end = is_q ? q_steps : steps;
            // the lane's row of this step and of the slice's next
            const int h[2] = {(is_q ? step : step - q_steps) * S::ROWS + sub, (is_q ? step : step - q_steps) * S::ROWS + sub + slices * S::ROWS};
            const bool two = step + slices < end;
            const bool live[2] = {h[0] < heads, two && h[1] < heads};
            const uint16_t *src = is_q ? a.q + (int64_t)token * a.q_stride : a.k + (int64_t)token * a.k_stride;
            uint4 raw[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    raw[u][k] = live[u] ? *reinterpret_cast<const uint4 *>(src + h[u] * DIM + 8 * c[k]) : make_uint4(0, 0, 0, 0);
            if (HALVES && weights_of != (int)is_q && !(a.flags & CSA2_ROPE_NO_NORM)) {
                weights_of = is_q;
                const float *ws = is_q ? a.q_weight : a.k_weight;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 wa = *reinterpret_cast<const float4 *>(ws + 8 * c[k]), wb = *reinterpret_cast<const float4 *>(ws + 8 * c[k] + 4);
                    held[k][0] = wa.x, held[k][1] = wa.y, held[k][2] = wa.z, held[k][3] = wa.w;
                    held[k][4] = wb.x, held[k][5] = wb.y, held[k][6] = wb.z, held[k][7] = wb.w;
                }
            }
            if (!turned) {                                             // while the rows are on their way
                turned = true;
                __syncwarp();
                fill_turns(turn, a.inv_freq, half, per, a.pos[token], a.flags & CSA2_ROPE_INVERSE ? -1.0f : 1.0f);
                __syncwarp();
            }
            uint16_t *dst = is_q ? a.q_out : a.k_out;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (u == 1 && !two) break;
                float x[2][8];
                finish<DIM, HALVES>(a, raw[u], x, held, is_q ? a.q_weight : a.k_weight, reinterpret_cast<const float4 *>(turn), c);
                if (!live[u]) continue;
                const int64_t to = ((int64_t)token * heads + h[u]) * DIM;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (dst)
                        *reinterpret_cast<uint4 *>(dst + to + 8 * c[k]) = make_uint4(
                            pack2(x[k][0], x[k][1]), pack2(x[k][2], x[k][3]), pack2(x[k][4], x[k][5]), pack2(x[k][6], x[k][7]));
                    if (!is_q && a.k_out_f32) {
                        float4 *f = reinterpret_cast<float4 *>(a.k_out_f32 + to + 8 * c[k]);
                        f[0] = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
                        f[1] = make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
                    }
                }
            }
            step += two ? 2 * slices : slices;
        }
    }
}

template <int DIM>
cudaError_t launch_dim(const NormRopeArgs &a, cudaStream_t st)
{
    constexpr int SMS = 148, RESIDENT = 4 * WARPS * SMS;               // warps at once
    constexpr int ROWS = Shape<DIM>::ROWS;
    const int q_steps = (a.heads + ROWS - 1) / ROWS, steps = q_steps + (a.kv_heads + ROWS - 1) / ROWS;
    // A warp forms the sines for its slice of a token: 16 steps pay for them
    // (8192 tokens x 65 rows of 512: 188 us in 4 slices, 202 in 1, 188 in 8).
    // Fewer tokens than warps: down to one pass of two steps each (64 tokens:
    // 4.3 us in 32 slices, 7.4 in 8).
    int slices = std::max(1, steps / 16);
    if ((int64_t)a.n * slices < RESIDENT) slices = std::max(slices, std::min((steps + 1) / 2, RESIDENT / a.n));
    const int64_t blocks = ((int64_t)a.n * slices + WARPS - 1) / WARPS;
    LaunchScope scope(-1, st);
    return launch_pdl(a.flags & CSA2_ROPE_HALVES ? norm_rope_kernel<DIM, true> : norm_rope_kernel<DIM, false>, dim3((unsigned)std::min<int64_t>(blocks, RESIDENT / WARPS)), dim3(THREADS),
                      sizeof(float) * WARPS * a.rot_dim, st, a, slices, q_steps, steps);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, int dim, cudaStream_t st)
{
    switch (dim) {
    case 64: return launch_dim<64>(a, st);
    case 128: return launch_dim<128>(a, st);
    case 256: return launch_dim<256>(a, st);
    case 512: return launch_dim<512>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace csa2
