// mx_quantize.cu -- rows to MXFP4 and back (include/mx.h has the format and
// the rounding).
//
// Quantising reads every value once and writes 17/32 byte for it, with a few
// operations a value: the memory system bounds it. A lane takes 8 consecutive
// values (one 16-byte load of bf16, two of fp32), four lanes make a block of
// 32; a warp takes a run of 1024 values, so that its 32 scales leave as one
// 32-byte sector. amax is found on the bit patterns (magnitudes order like
// integers, NaN above infinity above every number), whose exponent field is
// the block's floor(log2 amax); dividing by the scale is a multiplication by
// a power of two and so exact, and the one rounding is that of the conversion
// to E2M1. 32768 x 2048 bf16: 30 us, 5.6 TB/s of the 6.5 that a copy reaches; the
// way back takes 25 us.
#include <cuda_fp16.h>

#include "mx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 1024;  // values per warp and step

// Four codes pairs of 8 values, the first value in the low bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The 8 values of the codes in r (all of them fp16 values).
__device__ __forceinline__ void e2m1x8_values(uint32_t r, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(r));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *reinterpret_cast<const __half2 *>(&h[i]);
        v[2 * i] = __low2float(p);
        v[2 * i + 1] = __high2float(p);
    }
}

template <bool kF32>
struct Raw {
    uint4 q[kF32 ? 2 : 1];
};

template <bool kF32>
__device__ __forceinline__ Raw<kF32> load8(const void *x, int64_t elem) {
    Raw<kF32> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) +
                                                     elem * (kF32 ? 4 : 2));
    r.q[0] = __ldg(p);
    if (kF32) r.q[kF32 ? 1 : 0] = __ldg(p + 1);
    return r;
}

// kStrided: rows of x are ld elements apart; otherwise x is one run.
// Six resident CTAs (42 registers) hide bf16's loads best: quantising and
// dequantising 32768 x 2048 takes 61.9 us at five, 55.8 at six and 57.7 at eight;
// fp32, with twice the data in flight per lane, loses what the spills cost (4099 x
// 1536: 15.1 us unlimited, 16.6 at six).
template <bool kF32, bool kStrided>
__global__ void __launch_bounds__(kThreads, kF32 ? 1 : 6)
    mx_quantize_kernel(const void *__restrict__ x, int64_t n, int K, int64_t ld,
                       uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    pdl_trigger();
    pdl_wait();
    for (int64_t run = warp * kRun; run < n; run += warps * kRun) {
        Raw<kF32> raw[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = run + u * 256 + lane * 8;
            const int64_t at = kStrided ? (i / K) * ld + i % K : i;
            if (i < n) raw[u] = load8<kF32>(x, at);
            else raw[u] = Raw<kF32>();
        }
        uint32_t sc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float v[8];
            uint32_t e;  // exponent field of the block's largest magnitude
            if constexpr (kF32) {
                const uint32_t b[8] = {raw[u].q[0].x, raw[u].q[0].y, raw[u].q[0].z, raw[u].q[0].w,
                                       raw[u].q[1].x, raw[u].q[1].y, raw[u].q[1].z, raw[u].q[1].w};
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m = max(m, b[i] & 0x7fffffffu);
                    v[i] = __uint_as_float(b[i]);
                }
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                e = m >> 23;
            } else {
                const uint32_t b[4] = {raw[u].q[0].x, raw[u].q[0].y, raw[u].q[0].z, raw[u].q[0].w};
                uint32_t m = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    m = __vmaxu2(m, b[i] & 0x7fff7fffu);
                    v[2 * i] = __uint_as_float(b[i] << 16);
                    v[2 * i + 1] = __uint_as_float(b[i] & 0xffff0000u);
                }
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                e = max(m & 0xffffu, m >> 16) >> 7;
            }
            sc[u] = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
            const float inv = __uint_as_float((254u - sc[u]) << 23);  // 2^(127 - s)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= inv;
            const uint32_t c = sc[u] == 255u ? 0u : e2m1x8(v);
            const int64_t i = run + u * 256 + lane * 8;
            if (i < n) *reinterpret_cast<uint32_t *>(codes + i / 2) = c;
        }
        // block b of the run is in step b / 8, lanes 4 (b % 8) ..: lane b stores it
        const int src = 4 * (lane & 7), u = lane >> 3;
        const uint32_t s0 = __shfl_sync(0xffffffffu, sc[0], src);
        const uint32_t s1 = __shfl_sync(0xffffffffu, sc[1], src);
        const uint32_t s2 = __shfl_sync(0xffffffffu, sc[2], src);
        const uint32_t s3 = __shfl_sync(0xffffffffu, sc[3], src);
        const uint32_t s = u == 0 ? s0 : u == 1 ? s1 : u == 2 ? s2 : s3;
        if (run + lane * kMxBlock < n) scales[run / kMxBlock + lane] = static_cast<uint8_t>(s);
    }
}

// The same runs the other way: lane b loads the scale of block b of the run.
template <bool kF32>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                         int64_t n, void *__restrict__ y) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
    pdl_trigger();
    pdl_wait();
    for (int64_t run = warp * kRun; run < n; run += warps * kRun) {
        uint32_t c[4], sc = 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = run + u * 256 + lane * 8;
            c[u] = i < n ? __ldg(reinterpret_cast<const uint32_t *>(codes + i / 2)) : 0u;
        }
        if (run + lane * kMxBlock < n) sc = __ldg(scales + run / kMxBlock + lane);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float f = e8m0_value(__shfl_sync(0xffffffffu, sc, u * 8 + lane / 4));
            const int64_t i = run + u * 256 + lane * 8;
            if (i >= n) continue;
            float v[8];
            e2m1x8_values(c[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= f;
            if constexpr (kF32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(y) + i);
                o[0] = make_float4(v[0], v[1], v[2], v[3]);
                o[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(y) + i) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// A run per warp: short CTAs that the scheduler places as others end spread the
// load better than a loop over a resident grid (whose last round is part empty).
int grid_of(int64_t n) {
    const int64_t want = (n + kThreads / 32 * kRun - 1) / (kThreads / 32 * kRun);
    return static_cast<int>(want < (INT64_C(1) << 30) ? want : (INT64_C(1) << 30));
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

int launch_mx_quantize(const void *x, int dtype, int64_t rows, int K, int64_t ld, uint8_t *codes,
                       uint8_t *scales, cudaStream_t s) {
    const int64_t n = rows * K;
    if (n == 0) return MOE_OK;
    const dim3 grid(grid_of(n)), block(kThreads);
    if (dtype == MOE_F32)
        return ld == K ? launch_k(mx_quantize_kernel<true, false>, grid, block, 0, s, x, n, K, ld,
                                  codes, scales)
                       : launch_k(mx_quantize_kernel<true, true>, grid, block, 0, s, x, n, K, ld,
                                  codes, scales);
    return ld == K ? launch_k(mx_quantize_kernel<false, false>, grid, block, 0, s, x, n, K, ld,
                              codes, scales)
                   : launch_k(mx_quantize_kernel<false, true>, grid, block, 0, s, x, n, K, ld,
                              codes, scales);
}

}  // namespace moe

using namespace moe;

static int check_rows(const void *x, int dtype, int64_t rows, int K, const void *codes,
                      const void *scales) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0) return MOE_ERR_INVALID_ARG;
    if (K <= 0 || K % kMxBlock != 0 || rows > (INT64_C(1) << 46) / K)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(codes, 16)) return MOE_ERR_ALIGNMENT;
    return MOE_OK;
}

extern "C" int moe_mx_quantize(const void *x, int dtype, int64_t rows, int K, int64_t ld,
                               uint8_t *codes, uint8_t *scales, void *stream) {
    const int rc = check_rows(x, dtype, rows, K, codes, scales);
    if (rc != MOE_OK || rows == 0) return rc;
    if (ld < K) return MOE_ERR_INVALID_ARG;
    if (ld * (dtype == MOE_F32 ? 4 : 2) % 16 != 0) return MOE_ERR_ALIGNMENT;
    return launch_mx_quantize(x, dtype, rows, K, rows == 1 ? K : ld, codes, scales,
                              static_cast<cudaStream_t>(stream));
}

extern "C" int moe_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K,
                                 void *y, int dtype, void *stream) {
    const int rc = check_rows(y, dtype, rows, K, codes, scales);
    if (rc != MOE_OK || rows == 0) return rc;
    const int64_t n = rows * K;
    const dim3 grid(grid_of(n)), block(kThreads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == MOE_F32 ? launch_k(mx_dequantize_kernel<true>, grid, block, 0, s, codes, scales, n, y)
                            : launch_k(mx_dequantize_kernel<false>, grid, block, 0, s, codes, scales, n, y);
}
