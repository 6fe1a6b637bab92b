// mx.cuh -- MXFP4: shared definitions of the quantiser and the product
// (include/mx.h has the format), and the launchers.
#pragma once

#include "../../include/mx.h"
#include "moe_internal.cuh"

namespace moe {

constexpr int kMxBlock = 32;    // values per shared scale
constexpr int kMxWord = 128;    // values per four scales: the product's K granule
// The product's largest K: a tile of it takes 16 ms at an SM's share of the HBM's
// rate, and the item dealer waits for 16 tiles within its second.
constexpr int kMxMaxK = 1 << 22;

struct MxMatmulParams {
    const uint8_t *a, *as;      // [rows][K/2], [rows][K/32]
    const uint8_t *w, *ws;      // [E][N][K/2], [E][N][K/32]
    const int32_t *offsets;     // [E+1], or null: one group of all rows
    void *out;                  // [rows][N], or [rows][N/2] with silu_mul
    int *status;                // a context's status word, or (counts) a count of time-outs
    int rows, K, E, N, silu_mul, dtype;
    int counts;                 // waits that run out are counted in *status
    int wait_us;                // a wait's limit (0: a second)
    int withheld;               // a kind of barrier that never completes, for the self-test
};

// The product's kinds of barriers (moe_mx_selftest_timeout).
enum { kMxFullA = 1, kMxScaledA, kMxEmptyA, kMxFullB, kMxScaledB, kMxEmptyB, kMxTFull, kMxTEmpty,
       kMxDealt, kMxTaken };

int launch_mx_quantize(const void *x, int dtype, int64_t rows, int K, int64_t ld, uint8_t *codes,
                       uint8_t *scales, cudaStream_t s);
int launch_mx_matmul(const MxMatmulParams &p, int n_sm, cudaStream_t s);

// The value of an E8M0 scale (2^-127 is an fp32 subnormal; 255 is NaN).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7fffffffu : s << 23);
}

}  // namespace moe
