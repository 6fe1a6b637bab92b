// balance.cu -- the router's balance loss, its per-expert counts and the
// gradient of the logits (include/balance.h has the formulas).
//
// The logits are read once by each pass and a few operations are done per
// value, so the memory system bounds large batches and the launches small
// ones. A lane holds 8 consecutive experts of a row (one 16-byte load of bf16,
// two of fp32); a row takes TPR lanes, the power of two that covers E / 8, so
// a warp works on 32 / TPR rows at once and a row's sums are shuffles.
//
// Forward: the tokens are cut into chunks, one CTA each. A CTA walks the
// sequences that its chunk meets; for each it sums the normalised scores of
// its tokens per expert in registers (lanes, then row groups, then warps: a
// fixed order), counts the selected experts in shared memory, and stores both
// as one partial row. Chunk c and sequence b meet in slot c + b: along the
// tokens c and b only grow, and one of them does from each pair to the next,
// so the slots of all pairs differ and nchunk + B of them are enough. A second
// launch, one CTA per sequence, adds the sequence's slots in order (in fp64),
// forms prob, and the last CTA to finish adds the sequences' losses in order.
//
// Backward: with g_e = coef f_e / (B' T) of the token's sequence,
//   dloss/dl_e = (g_e - sum_j g_j p_j) / (sum s + eps) * s_e (1 - s_e),
// a row at a time from its logits, which are read again: the scores cost less
// to form than to store and load.
//
// 131072 tokens of 256 experts (fp32, 61 sequences): 44 us for the sums and the last
// reduction (36 and 8; a lane's two rows in flight are both worked on before the next
// are loaded), 47 for the gradient, which keeps a row ahead (5.7 TB/s; 64 with one row
// in flight and full-precision exponentials). 64 tokens take 19 us on the device, under
// the 109 that torch's autograd and the calls take on the host.
#include "../../include/balance.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFinishThreads = 1024;
constexpr int kV = 8;               // experts per lane
constexpr int kMinChunk = 8;        // tokens
constexpr int kMaxChunk = 1024;     // tokens: a lane's fp32 sums stay under 128 terms
constexpr int kMaxChunks = 148 * 4; // chunks of a large batch: four CTAs an SM
constexpr int kMaxCount = 1 << 30;  // tokens, sequences: a chunk, a step or both together past the
                                    // last one still fit an int

struct FwdParams {
    const void *logits;
    int64_t ld;
    const int32_t *idx, *seq;
    float *part;        // [nchunk + B][E] sums of normalised scores
    int32_t *part_n;    // [nchunk + B][E] counts
    double *seq_loss;   // [B]
    int32_t *ticket;    // finished CTAs of the second launch
    float *loss, *prob, *scale;
    int32_t *counts, *kept;  // kept: a second copy of counts, or null
    int N, E, k, B, chunk, nchunk;
    float coef, eps;
    bool vec;           // rows start on 16 bytes and E % 8 == 0
};

struct BwdParams {
    const void *logits;
    int64_t ld;
    const int32_t *counts, *seq;
    const float *scale, *gout;
    void *grad;
    int N, E, k, B, chunk;
    float eps;
    bool vec, vec_out;
};

__device__ __forceinline__ int seq_at(const int32_t *seq, int b, int B, int N) {
    if (!seq) return b == 0 ? 0 : N;
    const int v = seq[b];
    return v < 0 ? 0 : v > N ? N : v;
}

// The last sequence that starts at or before token t (sequences without
// tokens, which start where the next one does, are passed over).
__device__ __forceinline__ int find_seq(const int32_t *seq, int B, int N, int t) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_at(seq, mid, B, N) <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One lane's 8 logits of a row, experts e0 .. e0 + 7; -inf (a score of 0) past E.
template <bool kF32>
__device__ __forceinline__ void load_logits(const void *logits, int64_t row, int e0, int E, bool vec,
                                            float (&v)[kV]) {
    const float ninf = __int_as_float(0xff800000);
    if (vec) {
        if (e0 >= E) {
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] = ninf;
        } else if constexpr (kF32) {
            const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(logits) + row + e0);
            const float4 a = __ldg(p), b = __ldg(p + 1);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(
                static_cast<const uint16_t *>(logits) + row + e0));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int e = e0 + i;
        v[i] = e >= E ? ninf
               : kF32 ? static_cast<const float *>(logits)[row + e]
                      : bf16_to_f32(static_cast<const uint16_t *>(logits)[row + e]);
    }
}

// The exponential and the reciprocal are the fast ones: 2^-22 relative plus
// |v| 2^-23 from the rounded product with log2(e), no more than what an fp32 sum
// over the experts loses, and half the kernels' time.
// v = sigmoid(v) per value; returns the row's sum of scores plus eps. slope, if
// given, gets sigmoid's derivative: with t = exp(-|v|) it is t / (1 + t)^2,
// which keeps its relative accuracy where 1 - s would cancel.
// Shares and gradients only see scores, slopes and eps relative to the total, so
// all may be in any common scale. Totals under kTiny, whose scores may be subnormal
// and whose reciprocal may overflow, get the scale e^80: every logit of such a row
// lies under -22, s and its derivative are exp(v) to 2^-31, and exp(v + 80) is an
// ordinary number down to the -104 below which fp32 rounds a score to 0 (v + 80 is
// exact). Only eps < kTiny can have them; the branch costs a compare otherwise, and
// no registers, because it has the logits loaded again.
constexpr float kTiny = 0x1p-32f;
constexpr float kTinyShift = 80.f, kTinyScale = 5.5406223843935098e34f;  // e^80
constexpr float kLowest = -104.f;
template <int TPR>
__device__ __forceinline__ float row_sum(const float (&v)[kV]) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) sum += v[i];
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

template <int TPR, typename Reload>
__device__ __forceinline__ float scores(float (&v)[kV], float eps, float *slope, Reload reload) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const float t = __expf(-fabsf(v[i]));
        const float r = __fdividef(1.0f, 1.0f + t);
        v[i] = v[i] < 0.f ? t * r : r;   // a NaN stays one through t
        if (slope) slope[i] = t * r * r;
    }
    float total = row_sum<TPR>(v) + eps;
    if (eps < kTiny && __any_sync(0xffffffffu, total < kTiny)) {
        float u[kV];
        reload(u);
#pragma unroll
        for (int i = 0; i < kV; ++i) u[i] = u[i] < kLowest ? 0.f : __expf(u[i] + kTinyShift);
        const float scaled = row_sum<TPR>(u) + eps * kTinyScale;
        if (total < kTiny) {
            total = scaled;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                v[i] = u[i];
                if (slope) slope[i] = u[i];
            }
        }
    }
    return total;
}

template <bool kF32, int TPR>
__global__ void __launch_bounds__(kThreads) balance_partial_kernel(FwdParams p) {
    constexpr int G = 32 / TPR;          // rows per warp and step
    __shared__ float acc_s[kWarps][kMaxExperts];
    __shared__ int hist[kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / TPR, e0 = (lane % TPR) * kV;
    const int c = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    if (c == 0 && threadIdx.x == 0) *p.ticket = 0;
    int t = c * p.chunk;
    const int t_end = min(p.N, t + p.chunk);
    t = max(t, seq_at(p.seq, 0, p.B, p.N));
    while (t < t_end) {
        const int b = find_seq(p.seq, p.B, p.N, t);
        const int stop = min(t_end, seq_at(p.seq, b + 1, p.B, p.N));
        if (stop <= t) break;            // tokens behind the last sequence
        for (int e = threadIdx.x; e < p.E; e += kThreads) hist[e] = 0;
        float acc[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) acc[i] = 0.f;
        __syncthreads();
        // the rows of two steps are loaded before the first is worked on
        for (int r0 = t + warp * G; r0 < stop; r0 += 2 * kWarps * G) {
            float v[2][kV];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = r0 + u * kWarps * G + grp;
                load_logits<kF32>(p.logits, (r < stop ? r : r0) * p.ld, e0, p.E, p.vec, v[u]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = r0 + u * kWarps * G + grp;
                const float total = scores<TPR>(v[u], p.eps, nullptr, [&](float (&l)[kV]) {
                    load_logits<kF32>(p.logits, (r < stop ? r : r0) * p.ld, e0, p.E, p.vec, l);
                });
                if (r < stop) {
                    // eps may be 0 and every score may have underflowed: no share then
                    const float inv = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
                    for (int i = 0; i < kV; ++i) acc[i] += v[u][i] * inv;
                }
            }
        }
        for (int64_t i = static_cast<int64_t>(t) * p.k + threadIdx.x; i < static_cast<int64_t>(stop) * p.k;
             i += kThreads) {
            const int e = __ldg(p.idx + i);
            if (e >= 0 && e < p.E) atomicAdd(&hist[e], 1);  // integers: any order, one sum
        }
#pragma unroll
        for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < kV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (grp == 0)
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (e0 + i < p.E) acc_s[warp][e0 + i] = acc[i];
        __syncthreads();
        const size_t slot = static_cast<size_t>(c + b) * p.E;
        for (int e = threadIdx.x; e < p.E; e += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += acc_s[w][e];
            p.part[slot + e] = s;
            p.part_n[slot + e] = hist[e];
        }
        __syncthreads();
        t = stop;
    }
}

// Sums of f and n over the block in a fixed order, in thread 0.
__device__ __forceinline__ void block_sum(double &f, int &n, double *fs, int *ns) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        f += __shfl_down_sync(0xffffffffu, f, o);
        n += __shfl_down_sync(0xffffffffu, n, o);
    }
    __syncthreads();
    if (lane == 0) {
        fs[warp] = f;
        ns[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        f = fs[lane];
        n = ns[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            f += __shfl_down_sync(0xffffffffu, f, o);
            n += __shfl_down_sync(0xffffffffu, n, o);
        }
    }
}

__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(FwdParams p) {
    static_assert(kFinishThreads == 1024, "block_sum takes 32 warps");
    __shared__ double sum_s[kFinishThreads];
    __shared__ int cnt_s[kFinishThreads];
    __shared__ bool last;
    const int b = blockIdx.x, tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int t0 = seq_at(p.seq, b, p.B, p.N), t1 = seq_at(p.seq, b + 1, p.B, p.N);
    const int T = t1 - t0;
    const int c0 = T > 0 ? t0 / p.chunk : 0, c1 = T > 0 ? (t1 - 1) / p.chunk + 1 : 0;
    // kFinishThreads / e_pad slots at a time, each thread one expert of them
    int e_pad = 1;
    while (e_pad < p.E) e_pad <<= 1;
    const int groups = kFinishThreads / e_pad, e = tid % e_pad, g = tid / e_pad;
    double s = 0.0;
    int n = 0;
    if (e < p.E) {
        for (int c = c0 + g; c < c1; c += 4 * groups) {  // four slots' loads at a time
            float f[4];
            int m[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int cu = c + u * groups;
                const size_t slot = static_cast<size_t>(cu + b) * p.E + e;
                f[u] = cu < c1 ? p.part[slot] : 0.f;
                m[u] = cu < c1 ? p.part_n[slot] : 0;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s += static_cast<double>(f[u]);
                n += m[u];
            }
        }
    }
    sum_s[tid] = s;
    cnt_s[tid] = n;
    __syncthreads();
    double mine = 0.0;
    if (g == 0 && e < p.E) {
        for (int i = 1; i < groups; ++i) {
            s += sum_s[i * e_pad + e];
            n += cnt_s[i * e_pad + e];
        }
        const double prob = T > 0 ? s / T : 0.0;
        p.prob[static_cast<size_t>(b) * p.E + e] = static_cast<float>(prob);
        p.counts[static_cast<size_t>(b) * p.E + e] = n;
        if (p.kept) p.kept[static_cast<size_t>(b) * p.E + e] = n;
        if (T > 0) mine = static_cast<double>(p.E) * n / (static_cast<double>(p.k) * T) * prob;
    }
    int none = 0;
    block_sum(mine, none, sum_s, cnt_s);
    if (tid == 0) {
        p.seq_loss[b] = mine;
        __threadfence();
        last = atomicAdd(p.ticket, 1) == p.B - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double total = 0.0;
    int live = 0;
    for (int i = tid; i < p.B; i += kFinishThreads) {
        total += *reinterpret_cast<volatile double *>(p.seq_loss + i);
        live += seq_at(p.seq, i + 1, p.B, p.N) > seq_at(p.seq, i, p.B, p.N);
    }
    block_sum(total, live, sum_s, cnt_s);
    if (tid == 0) {
        const double sc = live > 0 ? static_cast<double>(p.coef) / live : 0.0;
        *p.loss = static_cast<float>(sc * total);
        *p.scale = static_cast<float>(sc);
    }
}

template <bool kF32, int TPR>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(BwdParams p) {
    constexpr int G = 32 / TPR;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / TPR, e0 = (lane % TPR) * kV;
    pdl_trigger();
    pdl_wait();
    const float scale = *p.scale * *p.gout;
    const int first = seq_at(p.seq, 0, p.B, p.N);
    // each row group walks its own contiguous tokens and keeps their sequence's g
    const int r_begin = blockIdx.x * p.chunk;
    const int r_end = min(p.N, r_begin + p.chunk);
    const int per = (p.chunk + kWarps * G - 1) / (kWarps * G);
    const int mine = r_begin + (warp * G + grp) * per;
    int stop = first;      // end of the sequence that g belongs to
    bool inside = false;   // whether there is one
    float g[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) g[i] = 0.f;
    float ahead[kV];       // the next token's logits, in flight during this one's work
    load_logits<kF32>(p.logits, (mine < r_end ? mine : 0) * p.ld, e0, p.E, p.vec, ahead);
    for (int j = 0; j < per; ++j) {
        const int r = mine + j;
        const bool live = r < r_end;     // the shuffles below want whole warps
        float v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = ahead[i];
        load_logits<kF32>(p.logits, (j + 1 < per && r + 1 < r_end ? r + 1 : 0) * p.ld, e0, p.E, p.vec, ahead);
        if (live && (r >= stop || j == 0)) {
            inside = false;
            if (r >= first) {
                const int b = find_seq(p.seq, p.B, p.N, r);
                const int t0 = seq_at(p.seq, b, p.B, p.N), t1 = seq_at(p.seq, b + 1, p.B, p.N);
                inside = r < t1;
                stop = inside ? t1 : p.N;
                if (inside) {
                    const float T = static_cast<float>(t1 - t0);
                    const float u = scale * static_cast<float>(p.E) / (static_cast<float>(p.k) * T) / T;
#pragma unroll
                    for (int i = 0; i < kV; ++i)
                        g[i] = e0 + i < p.E
                                   ? u * static_cast<float>(__ldg(p.counts + static_cast<size_t>(b) * p.E + e0 + i))
                                   : 0.f;
                }
            } else {
                stop = first;
            }
        }
        float slope[kV];
        const float total = scores<TPR>(v, p.eps, slope, [&](float (&l)[kV]) {
            load_logits<kF32>(p.logits, (live ? r : 0) * p.ld, e0, p.E, p.vec, l);
        });
        const float inv = total == 0.f ? 0.f : 1.0f / total;
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < kV; ++i) dot = fmaf(g[i], v[i], dot);
#pragma unroll
        for (int o = TPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        dot *= inv;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < kV; ++i)
            v[i] = inside ? (g[i] - dot) * inv * slope[i] : 0.f;
        const size_t at = static_cast<size_t>(r) * p.E + e0;
        if (p.vec_out) {
            if (e0 < p.E) {
                if constexpr (kF32) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.grad) + at);
                    o[0] = make_float4(v[0], v[1], v[2], v[3]);
                    o[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t *>(&h);
                    }
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.grad) + at) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (e0 + i < p.E) {
                    if constexpr (kF32) static_cast<float *>(p.grad)[at + i] = v[i];
                    else static_cast<__nv_bfloat16 *>(p.grad)[at + i] = __float2bfloat16_rn(v[i]);
                }
        }
    }
}

// Tokens per chunk: enough chunks for every SM, kMinChunk to kMaxChunk tokens each.
int chunk_of(int N) {
    const int c = static_cast<int>((static_cast<int64_t>(N) + kMaxChunks - 1) / kMaxChunks);
    return c < kMinChunk ? kMinChunk : c > kMaxChunk ? kMaxChunk : c;
}

int lanes_per_row(int E) {
    int t = 1;
    while (t * kV < E) t <<= 1;
    return t;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define BALANCE_LAUNCH(kern, f32, tpr, grid, s, p)                                        \
    switch (tpr) {                                                                         \
        case 1: return launch_k(kern<f32, 1>, dim3(grid), dim3(kThreads), 0, s, p);       \
        case 2: return launch_k(kern<f32, 2>, dim3(grid), dim3(kThreads), 0, s, p);       \
        case 4: return launch_k(kern<f32, 4>, dim3(grid), dim3(kThreads), 0, s, p);       \
        case 8: return launch_k(kern<f32, 8>, dim3(grid), dim3(kThreads), 0, s, p);       \
        case 16: return launch_k(kern<f32, 16>, dim3(grid), dim3(kThreads), 0, s, p);     \
        default: return launch_k(kern<f32, 32>, dim3(grid), dim3(kThreads), 0, s, p);     \
    }

int launch_partial(const FwdParams &p, int dtype, cudaStream_t s) {
    const int tpr = lanes_per_row(p.E);
    if (dtype == MOE_F32) {
        BALANCE_LAUNCH(balance_partial_kernel, true, tpr, p.nchunk, s, p)
    }
    BALANCE_LAUNCH(balance_partial_kernel, false, tpr, p.nchunk, s, p)
}

int launch_backward(const BwdParams &p, int dtype, int grid, cudaStream_t s) {
    const int tpr = lanes_per_row(p.E);
    if (dtype == MOE_F32) {
        BALANCE_LAUNCH(balance_backward_kernel, true, tpr, grid, s, p)
    }
    BALANCE_LAUNCH(balance_backward_kernel, false, tpr, grid, s, p)
}

int check_shape(int dtype, int64_t ld, const void *seq, int N, int E, int k, int B, float eps) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (N < 0 || B < 1 || !(eps >= 0.f) || (!seq && B != 1)) return MOE_ERR_INVALID_ARG;
    if (E < 1 || E > kMaxExperts || k < 1 || k > kMaxTopK || k > E) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (N >= kMaxCount || B >= kMaxCount) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (static_cast<int64_t>(N) * E >= (INT64_C(1) << 31) ||
        static_cast<int64_t>(B) * E >= (INT64_C(1) << 31))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (ld < E) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

bool rows_vec(const void *logits, int dtype, int64_t ld, int E) {
    return aligned16(logits) && ld * (dtype == MOE_F32 ? 4 : 2) % 16 == 0 && E % kV == 0;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_workspace(int n_tokens, int n_experts, int n_seqs) {
    if (n_tokens < 0 || n_experts < 1 || n_seqs < 1 || n_tokens >= kMaxCount || n_seqs >= kMaxCount)
        return 0;
    const int chunk = chunk_of(n_tokens);
    const size_t slots = static_cast<size_t>((n_tokens + chunk - 1) / chunk) + n_seqs;
    return 256 + static_cast<size_t>(n_seqs) * 8 + slots * n_experts * 8;
}

static int forward(const void *logits, int dtype, int64_t ld, const int32_t *idx,
                   const int32_t *seq_offsets, int n_tokens, int n_experts, int top_k, int n_seqs,
                   float coef, float eps, void *workspace, float *loss, int32_t *counts, float *prob,
                   float *scale, int32_t *kept, void *stream) {
    int rc = check_shape(dtype, ld, seq_offsets, n_tokens, n_experts, top_k, n_seqs, eps);
    if (rc != MOE_OK) return rc;
    if (!workspace || !loss || !counts || !prob || !scale || (n_tokens > 0 && (!logits || !idx)))
        return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MOE_ERR_ALIGNMENT;
    FwdParams p = {};
    p.logits = logits; p.ld = ld; p.idx = idx; p.seq = seq_offsets;
    p.N = n_tokens; p.E = n_experts; p.k = top_k; p.B = n_seqs;
    p.chunk = chunk_of(n_tokens);
    p.nchunk = (n_tokens + p.chunk - 1) / p.chunk;
    uint8_t *w = static_cast<uint8_t *>(workspace);
    const size_t slots = static_cast<size_t>(p.nchunk) + n_seqs;
    p.ticket = reinterpret_cast<int32_t *>(w);
    p.seq_loss = reinterpret_cast<double *>(w + 256);
    p.part = reinterpret_cast<float *>(w + 256 + static_cast<size_t>(n_seqs) * 8);
    p.part_n = reinterpret_cast<int32_t *>(p.part + slots * n_experts);
    p.loss = loss; p.counts = counts; p.kept = kept; p.prob = prob; p.scale = scale;
    p.coef = coef; p.eps = eps;
    p.vec = rows_vec(logits, dtype, ld, n_experts);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.nchunk > 0) {
        if ((rc = launch_partial(p, dtype, s)) != MOE_OK) return rc;
    } else if (cudaMemsetAsync(p.ticket, 0, 4, s) != cudaSuccess) {
        return MOE_ERR_CUDA;
    }
    return launch_k(balance_finish_kernel, dim3(n_seqs), dim3(kFinishThreads), 0, s, p);
}

extern "C" int moe_balance_forward(const void *logits, int dtype, int64_t ld, const int32_t *idx,
                                   const int32_t *seq_offsets, int n_tokens, int n_experts,
                                   int top_k, int n_seqs, float coef, float eps, void *workspace,
                                   float *loss, int32_t *counts, float *prob, float *scale,
                                   void *stream) {
    return forward(logits, dtype, ld, idx, seq_offsets, n_tokens, n_experts, top_k, n_seqs, coef, eps,
                   workspace, loss, counts, prob, scale, nullptr, stream);
}

extern "C" int moe_balance_forward_kept(const void *logits, int dtype, int64_t ld,
                                        const int32_t *idx, const int32_t *seq_offsets,
                                        int n_tokens, int n_experts, int top_k, int n_seqs,
                                        float coef, float eps, void *workspace, float *loss,
                                        int32_t *counts, float *prob, float *scale, int32_t *kept,
                                        void *stream) {
    if (!kept) return MOE_ERR_INVALID_ARG;
    return forward(logits, dtype, ld, idx, seq_offsets, n_tokens, n_experts, top_k, n_seqs, coef, eps,
                   workspace, loss, counts, prob, scale, kept, stream);
}

extern "C" int moe_balance_backward(const void *logits, int dtype, int64_t ld,
                                    const int32_t *counts, const int32_t *seq_offsets,
                                    const float *scale, const float *grad_loss, int n_tokens,
                                    int n_experts, int top_k, int n_seqs, float eps, void *grad,
                                    void *stream) {
    const int rc = check_shape(dtype, ld, seq_offsets, n_tokens, n_experts, top_k, n_seqs, eps);
    if (rc != MOE_OK) return rc;
    if (n_tokens == 0) return MOE_OK;
    if (!logits || !counts || !scale || !grad_loss || !grad) return MOE_ERR_INVALID_ARG;
    BwdParams p = {};
    p.logits = logits; p.ld = ld; p.counts = counts; p.seq = seq_offsets; p.scale = scale;
    p.gout = grad_loss; p.grad = grad;
    p.N = n_tokens; p.E = n_experts; p.k = top_k; p.B = n_seqs; p.eps = eps;
    p.chunk = chunk_of(n_tokens);
    p.vec = rows_vec(logits, dtype, ld, n_experts);
    p.vec_out = n_experts % kV == 0 && aligned16(grad);
    return launch_backward(p, dtype, (n_tokens + p.chunk - 1) / p.chunk,
                           static_cast<cudaStream_t>(stream));
}
