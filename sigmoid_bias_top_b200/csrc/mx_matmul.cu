// mx_matmul.cu -- the product of MXFP4 rows with the MXFP4 matrices of their
// experts (include/mx.h): out[r] = A[r] W_e^T, or silu(gate) * up of it.
//
// Tiles of 64 rows x 64 outputs on the CUDA cores: a K step is one block of 32
// values, whose codes are turned into fp32 values in shared memory once and
// used 64 times; each thread keeps a 4 x 4 corner of the sums. Every CTA finds
// its expert and row tile from the offsets itself.
#include <cuda_fp16.h>

#include "mx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

// 32 codes (16 bytes) times their scale into column `col` of a [32][kTile] tile.
__device__ __forceinline__ void spread(const uint4 &q, float f, float *tile, int col) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t c = (w[i >> 3] >> (4 * (i & 7))) & 15u;
        const uint32_t m = c & 7u;  // 0, 0.5, 1, 1.5, 2, 3, 4, 6
        const float v = m < 2u ? 0.5f * m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
        tile[i * kTile + col] = (c & 8u ? -v : v) * f;
    }
}

template <bool kSilu>
__global__ void __launch_bounds__(kThreads) mx_matmul_simt_kernel(MxMatmulParams p) {
    __shared__ float sa[32 * kTile], sw[(kSilu ? 2 : 1) * 32 * kTile];
    __shared__ int offs[kMaxExperts + 1];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i <= p.E; i += kThreads)
        offs[i] = p.offsets ? min(max(p.offsets[i], 0), p.rows) : i == 0 ? 0 : p.rows;
    __syncthreads();
    // the row tile blockIdx.x, counted over the experts
    int e = 0, tile = blockIdx.x;
    for (; e < p.E; ++e) {
        const int n = (max(offs[e + 1] - offs[e], 0) + kTile - 1) / kTile;
        if (tile < n) break;
        tile -= n;
    }
    if (e == p.E) return;
    const int r0 = offs[e] + tile * kTile, r1 = offs[e + 1];
    const int NO = kSilu ? p.N / 2 : p.N;
    const int n0 = blockIdx.y * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[kSilu ? 2 : 1][4][4] = {};
    for (int k = 0; k < p.K; k += 32) {
        const int t = threadIdx.x & 63, who = threadIdx.x >> 6;
        const bool is_a = who == 0;
        if (is_a || who == 1 || (kSilu && who == 2)) {
            const int r = is_a ? r0 + t : n0 + t;
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            float f = 0.f;
            if (r < (is_a ? r1 : NO)) {
                const size_t row = is_a ? r : static_cast<size_t>(e) * p.N + (who == 2 ? NO : 0) + r;
                q = *reinterpret_cast<const uint4 *>((is_a ? p.a : p.w) + row * (p.K / 2) + k / 2);
                f = e8m0_value((is_a ? p.as : p.ws)[row * (p.K / 32) + k / 32]);
            }
            spread(q, f, is_a ? sa : sw + (who - 1) * 32 * kTile, t);
        }
        __syncthreads();
#pragma unroll 8
        for (int kk = 0; kk < 32; ++kk) {
            const float4 a = *reinterpret_cast<const float4 *>(sa + kk * kTile + ty * 4);
            const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int g = 0; g < (kSilu ? 2 : 1); ++g) {
                const float4 b = *reinterpret_cast<const float4 *>(sw + (g * 32 + kk) * kTile + tx * 4);
                const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[g][i][j] = fmaf(av[i], bv[j], acc[g][i][j]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (r >= r1 || n >= NO) continue;
            float v = acc[0][i][j];
            if (kSilu) v = v / (1.0f + expf(-v)) * acc[kSilu ? 1 : 0][i][j];
            const size_t at = static_cast<size_t>(r) * NO + n;
            if (p.dtype == MOE_F32) static_cast<float *>(p.out)[at] = v;
            else static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(v);
        }
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

int launch_mx_matmul(const MxMatmulParams &p, cudaStream_t s) {
    const int NO = p.silu_mul ? p.N / 2 : p.N;
    const dim3 grid(p.rows / kTile + p.E, (NO + kTile - 1) / kTile);
    return p.silu_mul ? launch_k(mx_matmul_simt_kernel<true>, grid, dim3(kThreads), 0, s, p)
                      : launch_k(mx_matmul_simt_kernel<false>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_mx_matmul(const uint8_t *a_codes, const uint8_t *a_scales,
                             const uint8_t *w_codes, const uint8_t *w_scales,
                             const int32_t *offsets, int rows, int K, int n_experts, int N,
                             int silu_mul, void *out, int dtype, void *stream) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || (silu_mul != 0 && silu_mul != 1)) return MOE_ERR_INVALID_ARG;
    if (!offsets && n_experts != 1) return MOE_ERR_INVALID_ARG;
    if (K <= 0 || K % kMxWord != 0 || N <= 0 || N % (silu_mul ? 32 : 16) != 0)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (n_experts < 1 || n_experts > kMaxExperts) return MOE_ERR_UNSUPPORTED_SHAPE;
    // 32-bit row indices and TMA coordinates
    if (rows >= (1 << 30) || static_cast<int64_t>(n_experts) * N >= (INT64_C(1) << 30))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(out, 16) ||
        !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(offsets, 4))
        return MOE_ERR_ALIGNMENT;
    MxMatmulParams p = {};
    p.a = a_codes; p.as = a_scales; p.w = w_codes; p.ws = w_scales; p.offsets = offsets;
    p.out = out; p.rows = rows; p.K = K; p.E = n_experts; p.N = N; p.silu_mul = silu_mul;
    p.dtype = dtype;
    return launch_mx_matmul(p, static_cast<cudaStream_t>(stream));
}
