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
// rows and 128 values of K, word r at (r % 32) * 16 + (r / 32) * 4. Rows start
// anywhere, so no bulk copy can bring the scales there. Warps do: a lane loads four words, K = 512, of rows
// lane, lane + 32, ... at once, and the transpose of its 4 x 4 words is its
// 16-byte piece of four blocks (4-byte cp.async per word instead took 45 cycles
// of the load unit per instruction, 900 a stage where the MMAs need 350). The
// MMA thread copies the blocks on to TMEM (tcgen05.cp) before the stage's four
// MMAs. Every stage has TMEM columns of its own for them: a stage is refilled
// only after its MMAs have completed, so nothing is overwritten early.
// Roles (480 threads): a thread of warp 0 issues TMA, one of warp 1 copies
// scales and issues MMAs, warps 2..3 and 4..5 bring the scales of the weights
// and of the rows, warps 6..13 drain the accumulators (two in TMEM, so that a
// tile's epilogue runs under the next tile's MMAs), warp 14 works out the CTA's
// items (expert, weight tile, row tile; dealt out in a fixed order), 32 at a
// time, one a lane: divisions and searches that would cost every other role
// 2000 cycles per item. All waits are bounded (1 s) and report a time-out in the
// status word; the kernel then drains its copies and MMAs, frees TMEM and
// returns.
#include <cooperative_groups.h>

#include "mx.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int WM = 128;               // weight rows per CTA and tile
constexpr int BK = 256;               // K per stage (128 bytes of codes per row)
constexpr int UK = 64;                // K per MMA
constexpr int A_BYTES = WM * BK / 2;  // 16 KB
constexpr int SF_BLOCK = 512;         // scales of 128 rows x 128 values
constexpr int kEpiWarps = 8;
constexpr int kScaleWarps = 2;        // per operand
constexpr int kThreads = 64 + 64 * kScaleWarps + 32 * kEpiWarps + 64;
constexpr int kDeal = 32;             // items worked out at a time
constexpr int kMaxStages = 9;
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kPeerBitMask = 0xFEFFFFFFu;  // shared::cluster address in the pair's even CTA

// NT: rows of a tile at most. kPair: a tile is shared by two CTAs.
template <int NT, bool kPair>
struct Cfg {
    static constexpr int NB = (NT + 127) / 128;        // 128-row scale blocks of the rows
    static constexpr int B_ROWS = kPair ? NT / 2 : NT;
    static constexpr int B_BYTES = B_ROWS * BK / 2;
    static constexpr int SFA_BYTES = 2 * SF_BLOCK;
    static constexpr int SFB_BYTES = 2 * NB * SF_BLOCK;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
    static constexpr int STAGES = NT <= 32 ? 9 : 5;
    static constexpr int SF_COLS = 8 + 8 * NB;         // TMEM columns of a stage's scales
    static constexpr int USED_COLS = 2 * NT + STAGES * SF_COLS;
    static constexpr int TMEM_COLS = USED_COLS <= 256 ? 256 : 512;
    static constexpr int N_STEP = kPair ? 32 : 16;     // the MMA's N is a multiple of it
    static_assert(USED_COLS <= 512 && STAGES <= kMaxStages, "TMEM");
    static_assert(B_BYTES % 1024 == 0 && (SFA_BYTES + SFB_BYTES) % 1024 == 0, "swizzle atoms");
};

struct __align__(16) Ctl {  // the items behind it are read 16 bytes at a time
    uint64_t full[kMaxStages];    // codes and scales are in place
    uint64_t scaled[kMaxStages];  // pairs: this CTA's scales are in shared memory
    uint64_t peer[kMaxStages];    // leader: the other CTA's are
    uint64_t empty[kMaxStages];   // the stage's MMAs are done
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t dealt[2];            // a set of kDeal items is in place
    uint64_t taken[2];            // every role has read the set
    uint64_t drain, copied;
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

// Arrival on the barrier at the same offset in the pair's leader. What it has to
// order is local to this SM and done by then: TMEM reads that the caller fenced,
// or scales in this CTA's shared memory, which their writers fenced towards the
// async proxy and this thread has seen (an mbarrier wait in this CTA). No global
// access has to be ordered, so there is no release to the cluster, which waits
// for all of the SM's accesses in flight: 1300 cycles a stage.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t *bar) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(smem_u32(bar)));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// wait_bar on a barrier that threads of the other CTA arrive on.
__device__ __forceinline__ bool wait_bar_cluster(uint64_t *bar, uint32_t parity, Ctl *ctl, int *status) {
    const uint32_t addr = smem_u32(bar);
    uint64_t deadline = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 0u) {
            const uint64_t now = globaltimer_ns();
            if (deadline == 0) deadline = now + kWaitNs;
            else if (now > deadline) break;
        }
    }
    set_status(status, kStatusTimeout);
    atomicExch(&ctl->abort, 1);
    return false;
}

// The instructions of one CTA, or of a pair (cta_group::2: issued by the
// leader; loads of both CTAs complete on the leader's barrier, commits arrive
// in both).
template <bool kPair>
struct Tc {
    static __device__ __forceinline__ void alloc(uint32_t *dst, uint32_t cols) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(dst)),
                         "r"(cols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            tmem_alloc(dst, cols);
            tmem_relinquish();
        }
    }
    static __device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t cols) {
        if constexpr (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols)
                         : "memory");
        else
            tmem_dealloc(taddr, cols);
    }
    static __device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *m, int x, int y,
                                                   uint64_t *bar) {
        if constexpr (kPair)
            asm volatile(
                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(smem_u32(bar) & kPeerBitMask)
                : "memory");
        else
            tma_load_2d(dst, m, x, y, bar);
    }
    // Box {64 two-byte columns, 16 rows, gate|up, 4 row groups} of the paired-row view.
    static __device__ __forceinline__ void load_4d(void *dst, const CUtensorMap *m, int x, int group,
                                                   uint64_t *bar) {
        if constexpr (kPair)
            asm volatile(
                "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(0), "r"(0), "r"(group),
                "r"(smem_u32(bar) & kPeerBitMask)
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(0), "r"(0), "r"(group),
                "r"(smem_u32(bar))
                : "memory");
    }
    // 32 rows x 16 bytes of shared memory (each CTA's own) to 4 TMEM columns,
    // repeated in the four 32-lane quarters.
    static __device__ __forceinline__ void scales(uint32_t taddr, uint64_t desc) {
        if constexpr (kPair)
            asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
        else
            asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    }
    static __device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                               uint32_t accumulate) {
        if constexpr (kPair)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.b32 p, %6, 0;\n\t"
                "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                    "r"(d_tmem),
                "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
                : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.b32 p, %6, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
                    "r"(d_tmem),
                "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
                : "memory");
    }
    // one arrival on `bar`, in both CTAs of a pair, when this thread's tcgen05 work is done
    static __device__ __forceinline__ void commit(uint64_t *bar) {
        if constexpr (kPair)
            asm volatile(
                "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                " [%0], m;\n\t}" ::"r"(smem_u32(bar))
                : "memory");
        else
            umma_commit(bar);
    }
    // the same on this CTA's barrier alone
    static __device__ __forceinline__ void commit_here(uint64_t *bar) {
        if constexpr (kPair)
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                             smem_u32(bar))
                         : "memory");
        else
            umma_commit(bar);
    }
};

// Descriptor of a 512-byte scale block: no swizzle, 8-row groups of 16-byte
// rows 128 bytes apart, descriptor version 1.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128 >> 4) << 32 |
           static_cast<uint64_t>(1) << 46;
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

// Work item: weight rows from wrow on (tile wt of its expert), `rows` rows from
// t0; rows == 0 ends the list.
struct __align__(16) Item {
    int wrow, wt, t0, rows;
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
__device__ __forceinline__ Item decode(int item, int NW, const int32_t *mts, const int32_t *offs,
                                       int E, int N, int tile_outputs, int n_step) {
    Item it;
    const int e = find_expert(mts, E, item / NW);
    const int ntt = mts[e + 1] - mts[e];
    const int local = item - mts[e] * NW;
    it.wt = local / ntt;
    const int tt = local - it.wt * ntt;
    const int c = offs[e + 1] - offs[e];
    const int ts = ((c + ntt - 1) / ntt + n_step - 1) / n_step * n_step;
    it.t0 = offs[e] + tt * ts;
    it.rows = min(ts, c - tt * ts);
    it.wrow = e * N + it.wt * tile_outputs;
    return it;
}

// A role's walk along the dealt items. kWarp: the whole warp walks together.
template <bool kWarp>
struct Walk {
    Ctl *ctl;
    const Item *items;  // [2][kDeal]
    int *status;
    int i;

    __device__ __forceinline__ Walk(Ctl *c, const Item *it, int *st)
        : ctl(c), items(it), status(st), i(0) {}

    // false at the end of the list, or after a time-out
    __device__ __forceinline__ bool next(Item &it) {
        const int set = (i / kDeal) & 1;
        if (i % kDeal == 0 &&
            !wait_bar(&ctl->dealt[set], (i / (2 * kDeal)) & 1u, ctl, status))
            return false;
        const int4 v = *reinterpret_cast<const int4 *>(items + set * kDeal + i % kDeal);
        it.wrow = v.x; it.wt = v.y; it.t0 = v.z; it.rows = v.w;
        if (i % kDeal == kDeal - 1) {
            if (kWarp) __syncwarp();
            if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&ctl->taken[set]);
        }
        ++i;
        return it.rows > 0 && !aborted(ctl);
    }
};

// silu(g) * u. For a bf16 result the fast exponential and division (2^-20
// relative) leave its rounding alone; fp32 results take the full ones.
template <bool kFast>
__device__ __forceinline__ float silu_mul(float g, float u) {
    if (kFast) return __fdividef(g, 1.0f + __expf(-g)) * u;
    return g / (1.0f + expf(-g)) * u;
}

// Scale warp `mine` of kScaleWarps of an operand. ROWS: WM for the weights (NO =
// outputs of the layer, o_base = first of the CTA's outputs in the tile), the
// row tile NT for the rows (NO < 0). base: the operand's scale blocks in stage
// 0. A chunk is K = 512, two stages; the operand's warps take the chunks in
// turn, each with two in registers, so that their loads are in flight while
// earlier ones are stored. Rows past the tile's end take the last one's scales:
// their products are never stored. kVec: rows of scales are whole 16-byte words.
template <typename C, int ROWS, bool kPaired, bool kPair, bool kVec>
__device__ __forceinline__ void bring_scales(const MxMatmulParams &p, Ctl *ctl, const Item *items,
                                             uint8_t *base, int NO, int o_base, int tile_outputs,
                                             int nk, int mine) {
    constexpr int R = (ROWS + 31) / 32;        // rows per lane
    constexpr int NB = (ROWS + 127) / 128;     // blocks per 128 values of K
    struct Chunk {
        uint4 w[R];                            // four words of each of the lane's rows
        int stages, first;                     // its stages, counted from the kernel's first
    };
    const int lane = threadIdx.x & 31;
    const bool weights = NO >= 0;
    const uint8_t *src = weights ? p.ws : p.as;
    const size_t pitch = static_cast<size_t>(p.K / kMxBlock);
    const int words = p.K / kMxWord, nch = (words + 3) / 4;
    Walk<true> walk(ctl, items, p.status);
    const uint8_t *row[R];
    int kc = nch, turn = 0, stage = 0;
    bool more = true;

    auto fetch = [&](Chunk &c) {
        c.stages = 0;
        for (; more; ++kc, turn = turn + 1 == kScaleWarps ? 0 : turn + 1) {
            if (kc == nch) {
                Item it;
                more = walk.next(it);
                if (!more) return;
                kc = 0;
                const uint8_t *first = src + static_cast<size_t>(weights ? it.wrow : it.t0) * pitch;
                const int last = weights ? NO - 1 - it.wt * tile_outputs : it.rows - 1;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    // paired: 16 gate rows and their 16 up rows in turn
                    int o = weights ? o_base + (kPaired ? i * 16 + (lane & 15) : i * 32 + lane) : i * 32 + lane;
                    o = min(o, last) + (kPaired && lane >= 16 ? NO : 0);
                    row[i] = first + static_cast<size_t>(o) * pitch;
                }
            }
            const int n = min(2, nk - 2 * kc);
            if (turn == mine) {
                c.stages = n;
                c.first = stage;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if constexpr (kVec) {
                        c.w[i] = __ldg(reinterpret_cast<const uint4 *>(row[i] + kc * 16));
                    } else {
                        const uint32_t *u = reinterpret_cast<const uint32_t *>(row[i] + kc * 16);
                        const int left = words - kc * 4;
                        c.w[i].x = __ldg(u);
                        c.w[i].y = left > 1 ? __ldg(u + 1) : 0u;
                        c.w[i].z = left > 2 ? __ldg(u + 2) : 0u;
                        c.w[i].w = left > 3 ? __ldg(u + 3) : 0u;
                    }
                }
                stage += n;
                ++kc;
                turn = turn + 1 == kScaleWarps ? 0 : turn + 1;
                return;
            }
            stage += n;
        }
    };
    auto put = [&](const Chunk &c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h >= c.stages) break;
            const int s = (c.first + h) % C::STAGES;
            const uint32_t ph = static_cast<uint32_t>((c.first + h) / C::STAGES) & 1u;
            if (!wait_bar(&ctl->empty[s], ph ^ 1u, ctl, p.status)) return false;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t v[4];  // word 2h + j of the lane's four rows of the block
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 &w = c.w[4 * b + i < R ? 4 * b + i : R - 1];
                        v[i] = h == 0 ? (j == 0 ? w.x : w.y) : (j == 0 ? w.z : w.w);
                    }
                    *reinterpret_cast<uint4 *>(base + s * C::STAGE_BYTES + (j * NB + b) * SF_BLOCK + lane * 16) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                }
            fence_proxy_async_smem();  // before the tensor core's copy reads them
            __syncwarp();
            if (lane == 0) mbar_arrive(kPair ? &ctl->scaled[s] : &ctl->full[s]);
        }
        return true;
    };

    Chunk c0, c1;
    fetch(c0);
    for (;;) {
        fetch(c1);
        if (c0.stages == 0 || !put(c0)) break;
        fetch(c0);
        if (c1.stages == 0 || !put(c1)) break;
    }
}

// tcgen05.ld .16x256b.x4: 16 TMEM lanes x 32 columns; thread t gets lane t/4
// (registers 4i, 4i+1) and lane t/4 + 8 (4i+2, 4i+3) of columns 8i + 2 (t % 4)
// + {0, 1}.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// tcgen05.wait::ld that names the loads' destinations.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Four 8 x 8 bf16 tiles in fragment layout, stored transposed: lane l names the
// 16-byte row l % 8 of tile l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                  uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One warp's 32 accumulator columns (rows c0.. of the tile) x its 32 TMEM lanes
// to out. The fragments hold gate (lanes 0..15) and up (16..31) of an output in
// the same thread and register. bf16: pairs of rows are packed, stored
// transposed to the warp's staging rows (one per row of the tile, kPitch apart:
// no bank conflicts) and leave as 16-byte pieces; fp32 leaves from the
// fragments, 32 bytes of four rows at a time.
template <bool kSilu, typename T>
struct Drain {
    static constexpr int kOutputs = kSilu ? 16 : 32;   // per warp
    static constexpr int kPitch = kOutputs * 2 + 16;   // bytes
    static constexpr int kStage = sizeof(T) == 2 ? 32 * kPitch : 0;

    static __device__ __forceinline__ void run(uint32_t taddr, uint32_t stage, T *out, int f0, int NO,
                                               int lim, int lane) {
        uint32_t lo[16], hi[16];
        tmem_ld_16x256b_x4(taddr, lo);
        tmem_ld_16x256b_x4(taddr + (16u << 16), hi);
        tmem_ld_wait(lo);
        tmem_ld_wait(hi);
        if constexpr (kSilu) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                lo[i] = __float_as_uint(
                    silu_mul<sizeof(T) == 2>(__uint_as_float(lo[i]), __uint_as_float(hi[i])));
        }
        if constexpr (sizeof(T) == 2) {
            const uint32_t at = stage + lane * kPitch;
#pragma unroll
            for (int h = 0; h < kOutputs / 16; ++h) {
                const uint32_t(&v)[16] = h ? hi : lo;
                uint32_t q[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    q[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                stmatrix_x4_trans(at + h * 32, q[0], q[2], q[4], q[6]);
                stmatrix_x4_trans(at + h * 32 + 16, q[1], q[3], q[5], q[7]);
            }
            __syncwarp();
            constexpr int kPieces = kOutputs / 8;       // 16-byte pieces of a row
            const int col = f0 + (lane % kPieces) * 8;  // NO % 16 == 0: all 8 outputs or none
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int r = (i * 32 + lane) / kPieces;
                uint4 v;
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "r"(stage + r * kPitch + (lane % kPieces) * 16)
                             : "memory");
                if (r < lim && col < NO)
                    *reinterpret_cast<uint4 *>(out + static_cast<size_t>(r) * NO + col) = v;
            }
            __syncwarp();  // the staging rows are read before the next chunk's are written
        } else {
#pragma unroll
            for (int h = 0; h < kOutputs / 16; ++h) {
                const uint32_t(&v)[16] = h ? hi : lo;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int f = f0 + h * 16 + lane / 4 + ((i >> 1) & 1) * 8;
                    const int r = (i >> 2) * 8 + (lane & 3) * 2 + (i & 1);
                    if (r < lim && f < NO)
                        out[static_cast<size_t>(r) * NO + f] = __uint_as_float(v[i]);
                }
            }
        }
    }
};

template <typename C>
__device__ __forceinline__ int mma_n(const Item &it) {
    return (it.rows + C::N_STEP - 1) / C::N_STEP * C::N_STEP;
}

// A stage's scale blocks (shared address sf) to its TMEM columns; two: the rows
// fill more than one block.
template <typename C, bool kPair>
__device__ __forceinline__ void copy_scales(uint32_t sf, uint32_t taddr, bool two) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        Tc<kPair>::scales(taddr + 4 * j, scale_desc(sf + j * SF_BLOCK));
#pragma unroll
        for (int b = 0; b < C::NB; ++b)
            if (b == 0 || two)
                Tc<kPair>::scales(taddr + 8 + 4 * (j * C::NB + b),
                                  scale_desc(sf + C::SFA_BYTES + (j * C::NB + b) * SF_BLOCK));
    }
}

template <int NT, bool kPair, bool kSilu, typename T>
__device__ __forceinline__ void mx_matmul_body(const CUtensorMap &tmW, const CUtensorMap &tmA,
                                               const MxMatmulParams &p) {
    using C = Cfg<NT, kPair>;
    using X = Tc<kPair>;
    constexpr int kCtas = kPair ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *stages_out = smem + C::STAGES * C::STAGE_BYTES;  // the epilogue's staging rows
    Ctl *ctl = reinterpret_cast<Ctl *>(stages_out + kEpiWarps * Drain<kSilu, T>::kStage);
    Item *items = reinterpret_cast<Item *>(ctl + 1);       // [2][kDeal]
    int32_t *mts = reinterpret_cast<int32_t *>(items + 2 * kDeal);  // [E+1] prefix of row tiles
    int32_t *offs = mts + (p.E + 1);                        // [E+1]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;
    const int half = kPair ? static_cast<int>(blockIdx.x & 1) : 0;  // rank in the cluster of two
    const bool leader = half == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            // the TMA thread, and a scale warp of each operand or, for pairs, the
            // commit of the scales' copies
            mbar_init(&ctl->full[s], kPair ? 2 : 3);
            mbar_init(&ctl->scaled[s], 2);  // a scale warp of each operand
            mbar_init(&ctl->peer[s], 1);
            mbar_init(&ctl->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&ctl->tfull[b], 1);
            mbar_init(&ctl->tempty[b], kCtas * kEpiWarps);
            mbar_init(&ctl->dealt[b], 1);
            // TMA, scale and epilogue warps; MMA thread of the leader, copy threads of pairs
            mbar_init(&ctl->taken[b], 1 + 2 * kScaleWarps + kEpiWarps + (kPair ? leader ? 2 : 1 : 1));
        }
        mbar_init(&ctl->drain, 1);
        mbar_init(&ctl->copied, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) X::alloc(&ctl->tmem_base, C::TMEM_COLS);
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
    if constexpr (kPair) cg::this_cluster().sync();  // barriers and TMEM of both CTAs are ready
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    const uint32_t tmem_sf = tmem_base + 2 * NT;

    const int NO = kSilu ? p.N / 2 : p.N;                  // outputs
    constexpr int kCtaOutputs = kSilu ? 64 : 128;
    constexpr int kOutputs = kCtaOutputs * kCtas;          // outputs of a tile
    const int NW = (NO + kOutputs - 1) / kOutputs;
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
            Walk<false> walk(ctl, items, p.status);
            Item it;
            while (ok && walk.next(it)) {
                const int wrow = it.wrow + half * kCtaOutputs;
                const int trow = it.t0 + half * (mma_n<C>(it) / 2);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar(&ctl->empty[s], ph ^ 1u, ctl, p.status)) { ok = false; break; }
                    uint8_t *sa = smem + s * C::STAGE_BYTES;
                    if (leader) mbar_arrive_expect_tx(&ctl->full[s], kCtas * (A_BYTES + C::B_BYTES));
                    // the maps count two-byte columns: 64 of them are K = 256
                    if (kSilu) X::load_4d(sa, &tmW, kb * 64, wrow / 16, &ctl->full[s]);
                    else X::load_2d(sa, &tmW, kb * 64, wrow, &ctl->full[s]);
                    X::load_2d(sa + A_BYTES, &tmA, kb * 64, trow, &ctl->full[s]);
                    issued[s] = true;
                    issued_parity[s] = ph;
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            // (a pair's copies complete on the leader's barriers)
            if (!ok || aborted(ctl)) {  // let the other roles leave and our own copies land
                atomicExch(&ctl->abort, 1);
                const uint64_t dl = globaltimer_ns() + kWaitNs;
                for (int i = 0; leader && i < C::STAGES; ++i)
                    if (issued[i]) mbar_wait(&ctl->full[i], issued_parity[i], dl);
            }
        }
    } else if (warp == 1) {
        if (leader && elect_one()) {
            // ----------------------------- MMA ------------------------------
            int s = 0, tile = 0;
            uint32_t ph = 0;
            bool any = false;
            Walk<false> walk(ctl, items, p.status);
            Item it;
            for (; walk.next(it); ++tile) {
                const int buf = tile & 1;
                const uint32_t use = static_cast<uint32_t>(tile >> 1);
                if (kPair ? !wait_bar_cluster(&ctl->tempty[buf], (use & 1u) ^ 1u, ctl, p.status)
                          : !wait_bar(&ctl->tempty[buf], (use & 1u) ^ 1u, ctl, p.status))
                    break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * NT);
                const int n = mma_n<C>(it);
                const uint32_t idesc[2] = {idesc_mxf4(kCtas * WM, n, 0), idesc_mxf4(kCtas * WM, n, 1)};
                bool ok = true;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar(&ctl->full[s], ph, ctl, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(smem + s * C::STAGE_BYTES);
                    const uint32_t b0 = a0 + A_BYTES;
                    const uint32_t ta = tmem_sf + static_cast<uint32_t>(s * C::SF_COLS), tb = ta + 8;
                    if constexpr (!kPair) copy_scales<C, kPair>(b0 + C::B_BYTES, ta, n > 128);
#pragma unroll
                    for (int kk = 0; kk < BK / UK; ++kk)
                        X::mma(d_tmem, sw128_kmajor_desc(a0 + kk * UK / 2),
                               sw128_kmajor_desc(b0 + kk * UK / 2), idesc[kk & 1],
                               ta + 4 * (kk >> 1), tb + 4 * C::NB * (kk >> 1),
                               (kb | kk) != 0 ? 1u : 0u);
                    any = true;
                    X::commit(&ctl->empty[s]);
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                X::commit(&ctl->tfull[buf]);
            }
            if (any) {
                X::commit_here(&ctl->drain);
                mbar_wait(&ctl->drain, 0, globaltimer_ns() + kWaitNs);
            }
        }
    } else if (warp < 2 + 2 * kScaleWarps) {
        // ---------------------------- scales ----------------------------
        const bool weights = warp < 2 + kScaleWarps;
        const int mine = (warp - 2) % kScaleWarps;
        uint8_t *sf = smem + A_BYTES + C::B_BYTES;
        const bool vec = p.K % 512 == 0 &&
                         (reinterpret_cast<uintptr_t>(weights ? p.ws : p.as) & 15u) == 0;
        if (weights && vec)
            bring_scales<C, WM, kSilu, kPair, true>(p, ctl, items, sf, NO, half * kCtaOutputs, kOutputs, nk, mine);
        else if (weights)
            bring_scales<C, WM, kSilu, kPair, false>(p, ctl, items, sf, NO, half * kCtaOutputs, kOutputs, nk, mine);
        else if (vec)
            bring_scales<C, NT, false, kPair, true>(p, ctl, items, sf + C::SFA_BYTES, -1, 0, 0, nk, mine);
        else
            bring_scales<C, NT, false, kPair, false>(p, ctl, items, sf + C::SFA_BYTES, -1, 0, 0, nk, mine);
    } else if (warp == kThreads / 32 - 1) {
        if (kPair && elect_one()) {
            // ---- pairs: scales on to TMEM by the leader, told by the other CTA ----
            int s = 0;
            uint32_t ph = 0;
            bool any = false, ok = true;
            Walk<false> walk(ctl, items, p.status);
            Item it;
            while (ok && walk.next(it)) {
                const bool two = mma_n<C>(it) > 128;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar(&ctl->scaled[s], ph, ctl, p.status)) { ok = false; break; }
                    if (leader) {
                        if (!wait_bar_cluster(&ctl->peer[s], ph, ctl, p.status)) { ok = false; break; }
                        tc_fence_after();
                        copy_scales<C, kPair>(smem_u32(smem + s * C::STAGE_BYTES) + A_BYTES + C::B_BYTES,
                                              tmem_sf + static_cast<uint32_t>(s * C::SF_COLS), two);
                        X::commit_here(&ctl->full[s]);
                        any = true;
                    } else {
                        mbar_arrive_leader(&ctl->peer[s]);
                    }
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                }
            }
            if (any) {  // no copy is in flight when the kernel ends
                X::commit_here(&ctl->copied);
                mbar_wait(&ctl->copied, 0, globaltimer_ns() + kWaitNs);
            }
        }
    } else if (warp == kThreads / 32 - 2) {
        // ------------------------- item dealer --------------------------
        for (int c = 0;; ++c) {
            if (c >= 2 && !wait_bar(&ctl->taken[c & 1], ((c >> 1) & 1u) ^ 1u, ctl, p.status)) break;
            const int64_t item = blockIdx.x / kCtas +
                                 (static_cast<int64_t>(c) * kDeal + lane) * (gridDim.x / kCtas);
            Item it = {0, 0, 0, 0};
            if (item < total)
                it = decode(static_cast<int>(item), NW, mts, offs, E, p.N, kOutputs, C::N_STEP);
            items[(c & 1) * kDeal + lane] = it;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->dealt[c & 1]);
            if (__any_sync(0xffffffffu, it.rows == 0) || aborted(ctl)) break;
        }
    } else {
        // --------------------------- epilogue ---------------------------
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        const int ew = warp - 2 - 2 * kScaleWarps;
        const int c_first = (ew >> 2) * 32;       // its 32-column chunks, every second
        const uint32_t stage = smem_u32(stages_out) + ew * Drain<kSilu, T>::kStage;
        T *out = static_cast<T *>(p.out);
        int tile = 0;
        Walk<true> walk(ctl, items, p.status);
        Item it;
        for (; walk.next(it); ++tile) {
            const int buf = tile & 1;
            const uint32_t use = static_cast<uint32_t>(tile >> 1);
            if (!wait_bar(&ctl->tfull[buf], use & 1u, ctl, p.status)) break;
            tc_fence_after();
            const uint32_t t_lane = tmem_base + static_cast<uint32_t>(buf * NT) +
                                    (static_cast<uint32_t>(q * 32) << 16);
            const int f0 = it.wt * kOutputs + half * kCtaOutputs + q * (kSilu ? 16 : 32);
#pragma unroll 1
            for (int c0 = c_first; c0 < it.rows; c0 += 32 * (kEpiWarps / 4))
                Drain<kSilu, T>::run(t_lane + c0, stage, out + static_cast<size_t>(it.t0 + c0) * NO, f0,
                                     NO, it.rows - c0, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) mbar_arrive_leader(&ctl->tempty[buf]);
                else mbar_arrive(&ctl->tempty[buf]);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cg::this_cluster().sync();  // the leader's work in both CTAs has drained
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        X::dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <int NT, bool kSilu, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                     MxMatmulParams p) {
    mx_matmul_body<NT, false, kSilu, T>(tmW, tmA, p);
}

template <int NT, bool kSilu, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_matmul_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmA, MxMatmulParams p) {
    mx_matmul_body<NT, true, kSilu, T>(tmW, tmA, p);
}

// Device-side failures of calls without a context (moe_mx_status).
__device__ int g_mx_status;

// CTA pairs that can be resident at once (an SM without a partner in its GPC
// cannot host half a pair), at most one pair per two SMs.
int resident_pairs(const void *kern, size_t smem, int n_sm) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_sm / 2 * 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = n_sm / 2;
    }
    return n < n_sm / 2 ? n : n_sm / 2;
}

template <int NT, bool kPair, bool kSilu, typename T>
int launch(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    using C = Cfg<NT, kPair>;
    CUtensorMap w, a;
    int rc;
    const uint64_t wrows = static_cast<uint64_t>(p.E) * p.N;
    if (kSilu) rc = tc_encode_pair_4d(&w, p.w, wrows, p.K / 4, p.N / 2);
    else rc = tc_encode_2d(&w, p.w, wrows, p.K / 4, WM);
    if (rc != MOE_OK) return rc;
    if ((rc = tc_encode_2d(&a, p.a, p.rows, p.K / 4, C::B_ROWS)) != MOE_OK) return rc;
    const size_t smem = 1024 + C::STAGES * C::STAGE_BYTES + kEpiWarps * Drain<kSilu, T>::kStage +
                        sizeof(Ctl) + 2 * kDeal * sizeof(Item) + 2 * (p.E + 1) * sizeof(int32_t);
    // no more CTAs than there can be items
    const int64_t items = static_cast<int64_t>(p.rows / NT + p.E) *
                          ((p.N + (kPair ? 2 : 1) * WM - 1) / ((kPair ? 2 : 1) * WM));
    if constexpr (kPair) {
        auto kern = mx_matmul_pair_kernel<NT, kSilu, T>;
        if (ensure_smem(kern, smem) != MOE_OK) return MOE_ERR_CUDA;
        static int resident = 0;  // per kernel, for the device model of the process
        if (resident == 0) resident = resident_pairs(reinterpret_cast<const void *>(kern), smem, n_sm);
        const int pairs = static_cast<int>(items < resident ? items : resident);
        return launch_k(kern, dim3(2 * pairs), dim3(kThreads), smem, s, w, a, p);
    } else {
        auto kern = mx_matmul_kernel<NT, kSilu, T>;
        if (ensure_smem(kern, smem) != MOE_OK) return MOE_ERR_CUDA;
        return launch_k(kern, dim3(static_cast<int>(items < n_sm ? items : n_sm)), dim3(kThreads), smem,
                        s, w, a, p);
    }
}

template <int NT, bool kPair>
int launch_nt(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    if (p.dtype == MOE_F32)
        return p.silu_mul ? launch<NT, kPair, true, float>(p, n_sm, s)
                          : launch<NT, kPair, false, float>(p, n_sm, s);
    return p.silu_mul ? launch<NT, kPair, true, __nv_bfloat16>(p, n_sm, s)
                      : launch<NT, kPair, false, __nv_bfloat16>(p, n_sm, s);
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int status_address(int **out) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(out), g_mx_status) == cudaSuccess ? MOE_OK
                                                                                       : MOE_ERR_CUDA;
}

}  // namespace

int launch_mx_matmul(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    return p.rows <= 32 * p.E ? launch_nt<32, false>(p, n_sm, s) : launch_nt<192, true>(p, n_sm, s);
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
