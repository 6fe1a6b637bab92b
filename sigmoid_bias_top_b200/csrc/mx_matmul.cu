// mx_matmul.cu -- the product of MXFP4 rows with the MXFP4 matrices of their
// experts (include/mx.h): out[r] = A[r] W_e^T, or silu(gate) * up of it, on the
// block-scaled tensor-core instructions (tcgen05.mma kind::mxf4).
//
// The product is computed transposed, D[output][row] = W_e[output] . A[row]:
//   * M = 128 weight rows per tile. With silu_mul a tile covers 64 outputs:
//     one 4-D TMA box stages their gate and up rows interleaved in groups of
//     16, so TMEM lanes l and l + 16 of every 32-lane quarter hold gate and up
//     of one output.
//   * N = up to NT rows of one expert, rounded up to 16. An expert's rows are
//     split into tiles of equal size, so at most 15 padded columns per tile are
//     computed; padded columns are never stored.
// A stage holds K = 256: 128 bytes of codes per row in the 128-byte swizzle,
// loaded by TMA, and the two 4-byte words of scales of every row, which the
// tensor core takes from TMEM in a layout of its own: a 512-byte block per 128
// rows and 128 values of K, word r at (r % 32) * 16 + (r / 32) * 4. Two warps
// scatter the words there from their row-major place by 4-byte cp.async (rows
// start anywhere, so no bulk copy can), and the MMA thread copies the blocks
// on to TMEM (tcgen05.cp) before the stage's four MMAs. Every stage has TMEM
// columns of its own for them: a stage is refilled only after its MMAs have
// completed, so nothing is overwritten early.
// Roles (384 threads): a thread of warp 0 issues TMA, one of warp 1 copies
// scales and issues MMAs, warps 2 and 3 load the scales of the weights and of the
// rows, warps 4..11 drain the accumulators (two in TMEM, so that a tile's
// epilogue runs under the next tile's MMAs). Items (expert, weight tile, row
// tile) are dealt out in a fixed order; every CTA forms the plan from the
// offsets by itself. All waits are bounded (1 s) and report a time-out in the
// status word; the kernel then drains its copies and MMAs, frees TMEM and
// returns.
#include "mx.cuh"

namespace moe {
namespace {

constexpr int WM = 128;               // weight rows per tile
constexpr int BK = 256;               // K per stage (128 bytes of codes per row)
constexpr int UK = 64;                // K per MMA
constexpr int A_BYTES = WM * BK / 2;  // 16 KB
constexpr int SF_BLOCK = 512;         // scales of 128 rows x 128 values
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint64_t kWaitNs = 1000000000ull;

template <int NT>
struct Cfg {
    static constexpr int NB = (NT + 127) / 128;        // 128-row scale blocks of the rows
    static constexpr int B_BYTES = NT * BK / 2;
    static constexpr int SFA_BYTES = 2 * SF_BLOCK;
    static constexpr int SFB_BYTES = 2 * NB * SF_BLOCK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGES = NT <= 32 ? 9 : 5;
    static constexpr int SF_COLS = 8 + 8 * NB;         // TMEM columns of a stage's scales
    static constexpr int USED_COLS = 2 * NT + STAGES * SF_COLS;
    static constexpr int TMEM_COLS = USED_COLS <= 256 ? 256 : 512;
    static_assert(USED_COLS <= 512, "TMEM");
    static_assert(B_BYTES % 1024 == 0 && (SFA_BYTES + SFB_BYTES) % 1024 == 0, "swizzle atoms");
};

struct Ctl {
    uint64_t full[9];
    uint64_t empty[9];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Ctl *ctl, int *status) {
    if (mbar_try_wait(bar, parity)) return true;
    if (mbar_wait(bar, parity, globaltimer_ns() + kWaitNs)) return true;
    set_status(status, kStatusTimeout);
    atomicExch(&ctl->abort, 1);
    return false;
}

__device__ __forceinline__ bool aborted(Ctl *ctl) {
    return *reinterpret_cast<volatile int *>(&ctl->abort) != 0;
}

// True in one lane of the (converged) warp. The compiler knows that a region
// under it runs in a single thread and feeds the tcgen05 and TMA instructions'
// operands through uniform registers directly; under a test of the lane index
// every such instruction costs about 70 cycles to issue, which at four MMAs and
// six scale copies a stage was the kernel's bound.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// 4 bytes global -> shared; src_bytes == 0 writes zeros.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, uint32_t src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
                 : "memory");
}

// Box {64 two-byte columns, 16 rows, gate|up, 4 row groups} of the paired view.
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *m, int x, int group,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(0), "r"(0), "r"(group), "r"(smem_u32(bar))
        : "memory");
}

// Descriptor of a 512-byte scale block: no swizzle, 8-row groups of 16-byte
// rows 128 bytes apart, descriptor version 1.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 32 |
           static_cast<uint64_t>(1) << 46;
}

// 32 rows x 16 bytes of shared memory to 4 TMEM columns, repeated in the four
// 32-lane quarters.
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 A and B (K-major), E8M0 scales,
// M x N; the scales of the MMA's K = 64 are bytes 2h, 2h + 1 of their words.
__host__ __device__ constexpr uint32_t idesc_mxf4(int M, int N, int h) {
    return (static_cast<uint32_t>(2 * h) << 4)           // B scale byte
           | (1u << 7) | (1u << 10)                      // A, B: E2M1
           | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23)  // N / 8; E8M0
           | (static_cast<uint32_t>(M >> 4) << 24)
           | (static_cast<uint32_t>(2 * h) << 29);       // A scale byte
}

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
            "r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Work item: expert e, weight tile wt, `rows` rows from t0, computed with N.
struct Item {
    int e, wt, t0, rows, N;
};

__device__ __forceinline__ int find_expert(const int32_t *mts, int E, int q) {
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mts[mid] <= q) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Items run expert by expert, the row tiles of a weight tile one after another.
__device__ __forceinline__ Item decode(int item, int NW, const int32_t *mts,
                                       const int32_t *offs, int E) {
    Item it;
    it.e = find_expert(mts, E, item / NW);
    const int ntt = mts[it.e + 1] - mts[it.e];
    const int local = item - mts[it.e] * NW;
    it.wt = local / ntt;
    const int tt = local - it.wt * ntt;
    const int c = offs[it.e + 1] - offs[it.e];
    const int ts = ((c + ntt - 1) / ntt + 15) & ~15;
    it.t0 = offs[it.e] + tt * ts;
    it.rows = min(ts, c - tt * ts);
    it.N = (it.rows + 15) & ~15;
    return it;
}

// silu(g) * u. For a bf16 result the fast exponential and division (2^-20
// relative) leave its rounding alone; fp32 results take the full ones.
template <bool kFast>
__device__ __forceinline__ float silu_mul(float g, float u) {
    if (kFast) return __fdividef(g, 1.0f + __expf(-g)) * u;
    return g / (1.0f + expf(-g)) * u;
}

template <typename T>
__device__ __forceinline__ void store(T *p, float v);
template <>
__device__ __forceinline__ void store<float>(float *p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store<__nv_bfloat16>(__nv_bfloat16 *p, float v) {
    *p = __float2bfloat16_rn(v);
}

template <int NT, bool kSilu, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                     MxMatmulParams p) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + C::STAGES * C::STAGE_BYTES);
    int32_t *mts = reinterpret_cast<int32_t *>(ctl + 1);  // [E+1] prefix of row tiles
    int32_t *offs = mts + (p.E + 1);                        // [E+1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&ctl->full[s], 1 + 64);  // the TMA thread, and every lane of two warps
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], kEpiWarps);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&ctl->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmA);
    }
    pdl_trigger();
    pdl_wait();
    if (warp == 0) {
        // the plan: offsets brought into [0, rows], and the prefix of row tiles
        int run = 0;
        for (int i0 = 0; i0 <= E; i0 += 32) {
            const int i = i0 + lane;
            auto at = [&](int j) {
                return p.offsets ? min(max(p.offsets[j], 0), p.rows) : j == 0 ? 0 : p.rows;
            };
            const int beg = i <= E ? at(i) : 0;
            int tiles = i < E ? (max(at(i + 1) - beg, 0) + NT - 1) / NT : 0;
            int x = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i <= E) {
                mts[i] = run + x - tiles;
                offs[i] = beg;
            }
            run += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const uint32_t tmem_sf = tmem_base + 2 * NT;

    const int NO = kSilu ? p.N / 2 : p.N;                  // outputs
    const int NW = (NO + (kSilu ? 63 : 127)) / (kSilu ? 64 : 128);
    const int nk = (p.K + BK - 1) / BK;
    const int total = mts[E] * NW;  // out fits in memory: far below 2^31

    if (warp == 0) {
        if (elect_one()) {
            // ------------------------- TMA producer -------------------------
            int s = 0;
            uint32_t ph = 0;
            bool issued[C::STAGES];
            uint32_t issued_parity[C::STAGES];
            for (int i = 0; i < C::STAGES; ++i) issued[i] = false;
            bool ok = true;
            for (int item = blockIdx.x; ok && item < total && !aborted(ctl); item += gridDim.x) {
                const Item it = decode(item, NW, mts, offs, E);
                const int wrow = it.e * p.N + it.wt * (kSilu ? 64 : 128);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar(&ctl->empty[s], ph ^ 1u, ctl, p.status)) { ok = false; break; }
                    uint8_t *sa = smem + s * C::STAGE_BYTES;
                    mbar_arrive_expect_tx(&ctl->full[s], A_BYTES + C::B_BYTES);
                    // the maps count two-byte columns: 64 of them are K = 256
                    if (kSilu) tma_load_4d(sa, &tmW, kb * 64, wrow / 16, &ctl->full[s]);
                    else tma_load_2d(sa, &tmW, kb * 64, wrow, &ctl->full[s]);
                    tma_load_2d(sa + A_BYTES, &tmA, kb * 64, it.t0, &ctl->full[s]);
                    issued[s] = true;
                    issued_parity[s] = ph;
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (!ok || aborted(ctl)) {  // let the other roles leave and our own copies land
                atomicExch(&ctl->abort, 1);
                const uint64_t dl = globaltimer_ns() + kWaitNs;
                for (int i = 0; i < C::STAGES; ++i)
                    if (issued[i]) mbar_wait(&ctl->full[i], issued_parity[i], dl);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            // ----------------------------- MMA ------------------------------
            int s = 0, tile = 0;
            uint32_t ph = 0;
            bool any = false;
            for (int item = blockIdx.x; item < total && !aborted(ctl); item += gridDim.x, ++tile) {
                const Item it = decode(item, NW, mts, offs, E);
                const int buf = tile & 1;
                const uint32_t use = static_cast<uint32_t>(tile >> 1);
                if (!wait_bar(&ctl->tempty[buf], (use & 1u) ^ 1u, ctl, p.status)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * NT);
                const uint32_t idesc[2] = {idesc_mxf4(WM, it.N, 0), idesc_mxf4(WM, it.N, 1)};
                bool ok = true;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar(&ctl->full[s], ph, ctl, p.status)) { ok = false; break; }
                    tc_fence_after();
                    fence_proxy_async_smem();  // the scales were written by cp.async
                    const uint32_t a0 = smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t b0 = a0 + A_BYTES, sf = b0 + C::B_BYTES;
                    const uint32_t ta = tmem_sf + static_cast<uint32_t>(s * C::SF_COLS), tb = ta + 8;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        scales_to_tmem(ta + 4 * j, scale_desc(sf + j * SF_BLOCK));
#pragma unroll
                        for (int b = 0; b < C::NB; ++b)
                            scales_to_tmem(tb + 4 * (j * C::NB + b),
                                           scale_desc(sf + C::SFA_BYTES + (j * C::NB + b) * SF_BLOCK));
                    }
#pragma unroll
                    for (int kk = 0; kk < BK / UK; ++kk)
                        umma_mxf4(d_tmem, sw128_kmajor_desc(a0 + kk * UK / 2),
                                  sw128_kmajor_desc(b0 + kk * UK / 2), idesc[kk & 1],
                                  ta + 4 * (kk >> 1), tb + 4 * C::NB * (kk >> 1),
                                  (kb | kk) != 0 ? 1u : 0u);
                    any = true;
                    umma_commit(&ctl->empty[s]);
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                umma_commit(&ctl->tfull[buf]);
            }
            if (any) {
                umma_commit(&ctl->drain);
                mbar_wait(&ctl->drain, 0, globaltimer_ns() + kWaitNs);
            }
        }
    } else if (warp < 4) {
        // ------------- scales: warp 2 the weights', warp 3 the rows' -------------
        const bool weights = warp == 2;
        const size_t pitch = static_cast<size_t>(p.K / kMxBlock);
        constexpr int RA = WM / 32, RB = NT / 32;   // rows per lane
        constexpr int R = RA > RB ? RA : RB;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int item = blockIdx.x; ok && item < total && !aborted(ctl); item += gridDim.x) {
            const Item it = decode(item, NW, mts, offs, E);
            const uint8_t *src[R];
            uint32_t n[R];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = i * 32 + lane;
                n[i] = 0u;
                src[i] = weights ? p.ws : p.as;
                if (weights && i < RA) {
                    // with silu_mul, 16 gate rows and their 16 up rows in turn
                    const int o = kSilu ? it.wt * 64 + i * 16 + (lane & 15) : it.wt * 128 + r;
                    if (o < NO) {
                        n[i] = 4u;
                        src[i] += (static_cast<size_t>(it.e) * p.N + o + (kSilu && lane >= 16 ? NO : 0)) * pitch;
                    }
                } else if (!weights && i < RB && r < it.rows) {
                    n[i] = 4u;
                    src[i] += static_cast<size_t>(it.t0 + r) * pitch;
                }
            }
            for (int kb = 0; kb < nk; ++kb) {
                if (!wait_bar(&ctl->empty[s], ph ^ 1u, ctl, p.status)) { ok = false; break; }
                const uint32_t sf = smem_u32(smem + s * C::STAGE_BYTES) + A_BYTES + C::B_BYTES +
                                    (weights ? 0 : C::SFA_BYTES) + lane * 16;
                const bool two = kb * BK + kMxWord < p.K;  // K may end inside the stage
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (i < (weights ? RA : RB)) {
                        const uint32_t dst = sf + (i >> 2) * SF_BLOCK + (i & 3) * 4;
                        const uint32_t next = (weights ? 1 : C::NB) * SF_BLOCK;
                        cp_async_4(dst, src[i] + kb * 8, n[i]);
                        cp_async_4(dst + next, src[i] + kb * 8 + (two ? 4 : 0), two ? n[i] : 0u);
                    }
                }
                cp_async_arrive_noinc(&ctl->full[s]);
                if (++s == C::STAGES) { s = 0; ph ^= 1u; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // --------------------------- epilogue ---------------------------
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        const int c_first = ((warp - 4) >> 2) * 32;
        T *out = static_cast<T *>(p.out);
        int tile = 0;
        for (int item = blockIdx.x; item < total && !aborted(ctl); item += gridDim.x, ++tile) {
            const int buf = tile & 1;
            const uint32_t use = static_cast<uint32_t>(tile >> 1);
            if (!wait_bar(&ctl->tfull[buf], use & 1u, ctl, p.status)) break;
            tc_fence_after();
            const Item it = decode(item, NW, mts, offs, E);
            const uint32_t t_lane = tmem_base + static_cast<uint32_t>(buf * NT) +
                                    (static_cast<uint32_t>(q * 32) << 16);
            // lanes 0..15: gate of outputs f, lanes 16..31: up of the same f
            const int f = kSilu ? it.wt * 64 + q * 16 + (lane & 15) : it.wt * 128 + q * 32 + lane;
#pragma unroll 1
            for (int c0 = c_first; c0 < it.rows; c0 += 32 * (kEpiWarps / 4)) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(t_lane + c0, v);
                tmem_ld_wait(v);
                if constexpr (kSilu) {
                    // the gate lane finishes rows 0..15 of the chunk, the up lane 16..31
                    const bool is_gate = lane < 16;
                    const int rb = c0 + (is_gate ? 0 : 16);
                    const int lim = f < NO ? it.rows - rb : 0;
                    T *dst = out + static_cast<size_t>(it.t0 + rb) * NO + f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float lo = __uint_as_float(v[j]), hi = __uint_as_float(v[16 + j]);
                        const float got = __shfl_xor_sync(0xffffffffu, is_gate ? hi : lo, 16);
                        const float r = silu_mul<sizeof(T) == 2>(is_gate ? lo : got, is_gate ? got : hi);
                        if (j < lim) store<T>(dst, r);
                        dst += NO;
                    }
                } else {
                    const int lim = f < NO ? it.rows - c0 : 0;
                    T *dst = out + static_cast<size_t>(it.t0 + c0) * NO + f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j < lim) store<T>(dst, __uint_as_float(v[j]));
                        dst += NO;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tempty[buf]);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

// Device-side failures of calls without a context (moe_mx_status).
__device__ int g_mx_status;

template <int NT, bool kSilu, typename T>
int launch(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    using C = Cfg<NT>;
    CUtensorMap w, a;
    int rc;
    const uint64_t wrows = static_cast<uint64_t>(p.E) * p.N;
    if (kSilu) rc = tc_encode_pair_4d(&w, p.w, wrows, p.K / 4, p.N / 2);
    else rc = tc_encode_2d(&w, p.w, wrows, p.K / 4, WM);
    if (rc != MOE_OK) return rc;
    if ((rc = tc_encode_2d(&a, p.a, p.rows, p.K / 4, NT)) != MOE_OK) return rc;
    auto kern = mx_matmul_kernel<NT, kSilu, T>;
    const size_t smem = 1024 + C::STAGES * C::STAGE_BYTES + sizeof(Ctl) + 2 * (p.E + 1) * sizeof(int32_t);
    if (ensure_smem(kern, smem) != MOE_OK) return MOE_ERR_CUDA;
    // no more CTAs than there can be items
    const int64_t tiles = static_cast<int64_t>(p.rows / NT + p.E) *
                          ((p.N + (WM - 1)) / WM);
    const int grid = static_cast<int>(tiles < n_sm ? tiles : n_sm);
    return launch_k(kern, dim3(grid), dim3(kThreads), smem, s, w, a, p);
}

template <int NT>
int launch_nt(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    if (p.dtype == MOE_F32)
        return p.silu_mul ? launch<NT, true, float>(p, n_sm, s) : launch<NT, false, float>(p, n_sm, s);
    return p.silu_mul ? launch<NT, true, __nv_bfloat16>(p, n_sm, s)
                      : launch<NT, false, __nv_bfloat16>(p, n_sm, s);
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int status_address(int **out) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(out), g_mx_status) == cudaSuccess ? MOE_OK
                                                                                       : MOE_ERR_CUDA;
}

}  // namespace

int launch_mx_matmul(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    return p.rows <= 32 * p.E ? launch_nt<32>(p, n_sm, s) : launch_nt<192>(p, n_sm, s);
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
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_NO_DEVICE;
    if (status_address(&p.status) != MOE_OK) return MOE_ERR_CUDA;
    return launch_mx_matmul(p, n_sm, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_mx_status(void) {
    int *status = nullptr, v = 0;
    if (status_address(&status) != MOE_OK || cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&v, status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(status, 0, sizeof(int)) != cudaSuccess)
        return MOE_ERR_CUDA;
    return v & kStatusTimeout ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}
