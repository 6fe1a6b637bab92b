/*
 * mx.h -- C ABI of the microscaled 4-bit (MXFP4) operators on B200 (sm_100a):
 * quantising rows, the values of quantised rows, and the product of quantised
 * rows with the quantised matrices of their experts. Same library (libmoe.so),
 * conventions and error codes as moe.h.
 *
 * Format (OCP Microscaling Formats specification 1.0, MXFP4): along a row,
 * every 32 consecutive values share one E8M0 scale, a byte s standing for
 * 2^(s - 127) (255: NaN); each value is an E2M1 code (1 sign, 2 exponent bits
 * with bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times its scale. A
 * matrix [rows][K] is stored as codes[rows][K/2], value 2j of a row in the low
 * four bits of byte j and value 2j + 1 in the high four, and
 * scales[rows][K/32].
 *
 * All pointers are DEVICE pointers. The calls are asynchronous on `stream`,
 * allocate nothing and can be captured in a CUDA graph (a device's first call of
 * a kind sets its kernel up: make that one before a capture); the device must be
 * the calling thread's current one. Outputs must not overlap inputs.
 */
#ifndef SIGMOID_BIAS_TOP_MX_H
#define SIGMOID_BIAS_TOP_MX_H

#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* codes, scales = MXFP4 of x[rows][K] (dtype MOE_F32 or MOE_BF16), row r at
 * x + r * ld elements (ld >= K). Per block of 32: s = max(floor(log2 amax) - 2,
 * -127) + 127 and code = E2M1(v / 2^(s - 127)), rounded to nearest, ties to
 * the even code, saturating at 6 (amax in [6, 8) times a power of four may
 * saturate: the exponent follows amax alone, as the specification has it). A
 * block of zeros gets s = 0; a block that holds an infinity or a NaN gets
 * s = 255 and zero codes, so that its values are NaN. K % 32 == 0; x 16-byte
 * aligned and ld a multiple of 16 bytes; codes 16-byte aligned. rows == 0 is a
 * no-op. */
int moe_mx_quantize(const void *x, int dtype, int64_t rows, int K, int64_t ld, uint8_t *codes,
                    uint8_t *scales, void *stream);

/* y[rows][K] (dtype MOE_F32 or MOE_BF16, contiguous) = the values of the codes,
 * each product of code and scale rounded once (no rounding happens for scales
 * that moe_mx_quantize makes). y 16-byte aligned; codes and scales as above. */
int moe_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, void *y,
                      int dtype, void *stream);

/* out[r] = A[r] W_e^T for the rows r of every expert e:
 *   A [rows][K] and W [n_experts][N][K] in MXFP4,
 *   offsets [n_experts + 1] int32: expert e has rows offsets[e] ..
 *     offsets[e + 1] - 1 (as moe_debug_routing gives them); NULL with
 *     n_experts == 1 stands for {0, rows}.
 *   silu_mul == 0: out [rows][N];
 *   silu_mul == 1: N = 2I, W holds gate rows 0 .. I - 1, then up rows, and
 *     out [rows][I] = silu(gate) * up.
 * Products and sums are those of fp32; out (dtype MOE_F32 or MOE_BF16) is
 * rounded once. Rows of no expert are left as they were. Offsets that do not
 * ascend within [0, rows] give unspecified rows, with no access outside the
 * buffers. An expert may have no rows; rows == 0 is a no-op.
 * K % 128 == 0, K <= 2^22, N % 16 == 0 (N % 32 == 0 with silu_mul), n_experts <= 256,
 * rows < 2^30 and n_experts * N < 2^30; codes and out 16-byte, scales and
 * offsets 4-byte aligned. */
int moe_mx_matmul(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                  const uint8_t *w_scales, const int32_t *offsets, int rows, int K, int n_experts,
                  int N, int silu_mul, void *out, int dtype, void *stream);

/* moe_mx_matmul waits inside its kernel with a limit of a second. Waits for the
 * current device, then tells what the calls on it, of any thread, met since the
 * calling thread's last reading (its first: since the program's start): MOE_OK or
 * MOE_ERR_DEVICE_TIMEOUT (out of a call is then incomplete). A reading leaves what
 * other threads will be told as it is. */
int moe_mx_status(void);

/* For tests of the time-out: moe_mx_matmul with waits of at most timeout_us (1 to
 * 1000000) whose barriers of one kind (withheld: 1 to 10, 0 for none) wait for an
 * arrival that nothing makes. Where the call's size has that kind waited for, it
 * returns within a few times timeout_us plus 40 ms, moe_mx_status tells of it, and
 * out is unspecified; calls after it are not affected. */
int moe_mx_selftest_timeout(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const int32_t *offsets, int rows, int K,
                            int n_experts, int N, int silu_mul, void *out, int dtype, int timeout_us,
                            int withheld, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* SIGMOID_BIAS_TOP_MX_H */
