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
// A tile is one CTA's (few rows per expert) or shared by two CTAs
// (cta_group::2): 256 weight rows, each CTA staging its own 128 of them and half
// of the tile's rows, which the MMA reads from both.
// A stage holds K = 512: two TMA boxes of 256 values (128 bytes of codes) per
// operand in the 128-byte swizzle, and the scales. Pairs keep the weights in a
// ring of their own: where all of K fits it (K <= 2048), the row tiles of a weight
// tile, which a pair takes one after another, share one load of it.
// The scales, four 4-byte words per row and stage, the tensor core takes from
// TMEM: column c, lane r of every 32-lane quarter holds the word of row 32 c + r.
// TMA brings a stage's 16 bytes of every row to shared memory; four warps, one
// per quarter, read them (rows lane, lane + 32, ...) and store the words, whose
// transpose is a matter of register names, to their quarter (tcgen05.st). What
// was slower: loads of the words by warps (a 16-byte load of 32 rows took 150
// cycles of the load unit's time, 4-byte cp.async 45), and copies from shared
// memory to TMEM (tcgen05.cp), which run in the MMAs' pipe, 30 cycles for 128
// words, 360 a stage where the MMAs need 768. Scale rows that TMA cannot address
// (K % 512, unaligned) are loaded by the four warps themselves.
// Roles (512 threads): a thread of warp 0 loads the weights, one of warp 15 the
// rows, one of warp 1 issues the MMAs, warps 2..5 bring the scales to TMEM, warps
// 6..13 drain the accumulators (two in TMEM, so that a tile's epilogue runs under
// the next tile's MMAs), warp 14 works out the items (expert, weight tile, row
// tile), 16 at a time, one a lane: divisions and searches that would cost every
// other role 2000 cycles per item. All waits are bounded (1 s). One that runs out
// reports it in the status word and tells every role of the CTA, or of both, whose
// waits then end as well (a warp's for all of its lanes at once, since what follows
// in it are warp-wide instructions); the kernel drains its copies and MMAs, frees
// TMEM and returns.
//
// What bounds it. Few rows: the weights' stream from HBM; 128 rows of 64 experts,
// gate/up (K 2048, I 1536), three sets of weights in turn: 35 us, 81% of what a copy
// reaches, about 4 us of them the launch's own latencies. Many rows: waits between the
// roles; 32768 rows: 107 us in short runs, with MMAs in half of the cycles (the MMAs
// alone would take 52 at that clock). Known of them: the first weights of a run wait
// for the last row tile of the run before where K fills the ring (K 2048; without the
// weights' loads, as a bound, 20% less), pairs get equal numbers of items and not
// equal work, and above K 2048 nothing is shared. The 1000 W power cap comes on top:
// 127 us in long runs (SMs at 1.4 GHz instead of 1.6). The shared load of the weights
// took 6% off both; half the tile's rows per SM (pairs), 7%. One row tile's shape, 192
// rows: two accumulators and the scales fill TMEM (512 columns).
#include <cooperative_groups.h>
#include <stddef.h>

#include <atomic>

#include "mx.cuh"

namespace cg = cooperative_groups;

namespace moe {
namespace {

constexpr int WM = 128;               // weight rows per CTA and tile
constexpr int SUBK = 256;             // K per TMA box (128 bytes of codes per row)
constexpr int KSUB = 2;               // boxes per operand and stage
constexpr int BK = SUBK * KSUB;       // K per stage
constexpr int KWORDS = BK / kMxWord;  // 4-byte words of scales per row and stage
constexpr int UK = 64;                // K per MMA
constexpr int A_SUB = WM * SUBK / 2;  // 16 KB
constexpr int A_BYTES = A_SUB * KSUB;
constexpr int kEpiWarps = 8;
constexpr int kScaleWarps = 4;        // one per 32-lane quarter of TMEM
constexpr int kThreads = 32 * (4 + kScaleWarps + kEpiWarps);
constexpr int kDeal = 16;             // items worked out at a time
constexpr int kMaxStages = 4;
constexpr int NA = 4;                 // weight stages
constexpr int A_SLOT = A_BYTES + WM * 16;  // codes and scales
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint64_t kDrainNs = 20000000ull;  // after a time-out, for copies in flight: over a
                                            // thousand times what one takes
constexpr uint32_t kPeerBitMask = 0xFEFFFFFFu;  // shared::cluster address in the pair's even CTA

struct MxKernelParams : MxMatmulParams {
    bool sf_tma;                  // the scales come by TMA
    uint64_t wait_ns;             // a wait's limit
};

// NT: rows of a tile at most. kPair: a tile is shared by two CTAs.
template <int NT, bool kPair>
struct Cfg {
    static constexpr int NB = (NT + 127) / 128;        // 128-row scale blocks of the rows
    static constexpr int R = (NT + 31) / 32;           // rows of a tile per lane
    static constexpr int B_ROWS = kPair ? NT / 2 : NT;
    static constexpr int B_SUB = B_ROWS * SUBK / 2;
    static constexpr int B_BYTES = B_SUB * KSUB;
    static constexpr int B_SLOT = B_BYTES + (NT + 63) / 64 * 64 * 16;  // codes and scales
    static constexpr int STAGES = kPair ? 3 : 4;       // of the rows
    static constexpr int SLOTS_BYTES = NA * A_SLOT + STAGES * B_SLOT;
    static constexpr int SFA_COLS = 4 * KWORDS;        // TMEM columns of a weight stage's scales
    static constexpr int SFB_COLS = 4 * KWORDS * NB;   // of a row stage's
    static constexpr int SF_SLOTS = kPair ? 2 : 4;     // sets of the latter
    static constexpr int USED_COLS = 2 * NT + NA * SFA_COLS + SF_SLOTS * SFB_COLS;
    static constexpr int TMEM_COLS = USED_COLS <= 256 ? 256 : 512;
    static constexpr int N_STEP = 16;                  // the MMA's N is a multiple of it
    static_assert(USED_COLS <= 512 && STAGES <= kMaxStages, "TMEM");
    static_assert(kPair || (STAGES == NA && SF_SLOTS == NA), "one ring of stages");
    // a slot's last MMAs are waited for on their stage's barrier, which a later
    // stage must not have gone through again by then
    static_assert(SF_SLOTS <= STAGES, "slots");
    static_assert(A_SLOT % 1024 == 0 && B_SUB % 1024 == 0 && B_SLOT % 1024 == 0, "swizzle atoms");
};

struct __align__(16) Ctl {  // the items behind it are read 16 bytes at a time
    // pairs, whose weight stages outlive an item; single CTAs move both operands
    // on together and count the weights' loads on the rows' barriers
    uint64_t fulla[NA];            // the weights' codes are in place
    uint64_t scaleda[NA];          // their scales are in shared memory
    uint64_t emptya[NA];           // the MMAs of all items that share them are done
    uint64_t fullb[kMaxStages];    // the rows' codes and all scales are in place
    uint64_t scaledb[kMaxStages];  // the rows' scales are in shared memory
    uint64_t emptyb[kMaxStages];   // the stage's MMAs are done
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t dealt[2];            // a set of kDeal items is in place
    uint64_t taken[2];            // every role has read the set
    uint64_t drain;
    uint64_t wait_ns;
    uint32_t tmem_base;
    uint32_t peer_abort;          // cluster address of the pair's other abort word (0: none)
    int counts;                   // the status word counts time-outs
    int abort;
};

// Barriers by their shared addresses (one register, no conversion from generic
// pointers: the roles' loops are bound by their instructions' latencies).
__device__ __forceinline__ bool try_bar(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool aborted(Ctl *ctl) {
    return *reinterpret_cast<volatile int *>(&ctl->abort) != 0;
}

// kWarp: the whole warp waits, and all of its lanes get one answer.
template <bool kWarp>
__device__ __noinline__ bool wait_bar_slow(uint32_t bar, uint32_t parity, Ctl *ctl, int *status) {
    const uint64_t deadline = globaltimer_ns() + ctl->wait_ns;
    for (uint32_t i = 0;; ++i) {
        const bool ok = try_bar(bar, parity);
        if (kWarp ? __all_sync(0xffffffffu, ok) : ok) return true;
        if ((i & 15u) == 15u) {
            bool stop = aborted(ctl);
            if (!stop && globaltimer_ns() > deadline) {
                stop = true;
                if (ctl->counts) atomicAdd(status, 1);
                else set_status(status, kStatusTimeout);
                atomicExch(&ctl->abort, 1);
                if (ctl->peer_abort != 0u)  // it cannot exit before this CTA
                    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(ctl->peer_abort)
                                 : "memory");
            }
            if (kWarp ? __any_sync(0xffffffffu, stop) : stop) return false;
        }
    }
}

template <bool kWarp>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl *ctl, int *status) {
    // a try suspends the thread for a while by itself; a few of them cover any
    // wait of a running pipeline
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        const bool ok = try_bar(bar, parity);
        if (kWarp ? __all_sync(0xffffffffu, ok) : ok) return true;
    }
    return wait_bar_slow<kWarp>(bar, parity, ctl, status);
}

__device__ __forceinline__ void arrive_bar(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void arrive_bar_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 ld_shared(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
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

// Arrival on the barrier at the same offset in the pair's leader. It orders this
// thread's TMEM accesses, which the caller has fenced, and nothing else: a
// release to the cluster would wait for all of the thread's global accesses in
// flight (over 700 cycles a stage).
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}

// sw128_kmajor_desc in its two words; the low word moves by bytes / 16.
constexpr uint32_t kDescHigh = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) {
    return ((saddr & 0x3FFFFu) >> 4) | 1u << 16;
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
    // dst and bar are shared addresses
    static __device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *m, int x, int y,
                                                   uint32_t bar) {
        if constexpr (kPair)
            asm volatile(
                "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar & kPeerBitMask)
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
                : "memory");
    }
    // Box {two-byte columns, 16 rows, gate|up, 4 row groups} of the paired-row view.
    static __device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap *m, int x, int group,
                                                   uint32_t bar) {
        if constexpr (kPair)
            asm volatile(
                "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(0), "r"(0), "r"(group),
                "r"(bar & kPeerBitMask)
                : "memory");
        else
            asm volatile(
                "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
                "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(0), "r"(0), "r"(group), "r"(bar)
                : "memory");
    }
    // a, b: low words of the operands' descriptors (kDescHigh: the high word of both)
    static __device__ __forceinline__ void mma(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
        if constexpr (kPair)
            asm volatile(
                "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
                "mov.b64 x, {%1, %7};\n\t"
                "mov.b64 y, {%2, %7};\n\t"
                "setp.ne.b32 p, %6, 0;\n\t"
                "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %3, [%4], [%5], p;\n\t}" ::
                    "r"(d_tmem),
                "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHigh)
                : "memory");
        else
            asm volatile(
                "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
                "mov.b64 x, {%1, %7};\n\t"
                "mov.b64 y, {%2, %7};\n\t"
                "setp.ne.b32 p, %6, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], x, y, %3, [%4], [%5], p;\n\t}" ::
                    "r"(d_tmem),
                "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHigh)
                : "memory");
    }
    // one arrival on `bar`, in both CTAs of a pair, when this thread's tcgen05 work is done
    static __device__ __forceinline__ void commit(uint32_t bar) {
        if constexpr (kPair)
            asm volatile(
                "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
                "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                " [%0], m;\n\t}" ::"r"(bar)
                : "memory");
        else
            commit_here(bar);
    }
    // the same on this CTA's barrier alone
    static __device__ __forceinline__ void commit_here(uint32_t bar) {
        if constexpr (kPair)
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                         : "memory");
        else
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                         : "memory");
    }
};

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
// t0; first, last: of a run of items that share the weights' stages. rows == 0
// ends the list.
struct Item {
    int wrow, wt, t0, rows;
    bool first, last;
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
// A CTA (pair) takes the items [begin, end), packed for shared memory. reuse:
// the row tiles of a weight tile share its stages.
__device__ __forceinline__ int4 decode(int item, int begin, int end, bool reuse, int NW,
                                       const int32_t *mts, const int32_t *offs, int E, int N,
                                       int tile_outputs, int n_step) {
    const int e = find_expert(mts, E, item / NW);
    const int ntt = mts[e + 1] - mts[e];
    const int local = item - mts[e] * NW;
    const int wt = local / ntt, tt = local - wt * ntt;
    const int c = offs[e + 1] - offs[e];
    const int ts = ((c + ntt - 1) / ntt + n_step - 1) / n_step * n_step;
    const bool first = !reuse || tt == 0 || item == begin;
    const bool last = !reuse || tt == ntt - 1 || item == end - 1;
    return make_int4(e * N + wt * tile_outputs, wt, offs[e] + tt * ts,
                     min(ts, c - tt * ts) | (first ? 1 << 16 : 0) | (last ? 1 << 17 : 0));
}

// The shared addresses of a barrier of Ctl, at base `bars` (that of the Ctl).
#define MX_BAR(field, i) (bars + static_cast<uint32_t>(offsetof(Ctl, field)) + 8u * static_cast<uint32_t>(i))

// A role's walk along the dealt items, which follow the Ctl. kWarp: the whole
// warp walks together.
template <bool kWarp>
struct Walk {
    Ctl *ctl;
    int *status;
    uint32_t bars;
    int i;

    __device__ __forceinline__ Walk(Ctl *c, uint32_t b, int *st) : ctl(c), status(st), bars(b), i(0) {}

    // false at the end of the list, or after a time-out
    __device__ __forceinline__ bool next(Item &it) {
        const int set = (i / kDeal) & 1;
        if (i % kDeal == 0 && !wait_bar<kWarp>(MX_BAR(dealt, set), (i / (2 * kDeal)) & 1u, ctl, status)) return false;
        const uint4 v = ld_shared(bars + static_cast<uint32_t>(sizeof(Ctl)) +
                                  (set * kDeal + i % kDeal) * static_cast<uint32_t>(sizeof(int4)));
        it.wrow = static_cast<int>(v.x);
        it.wt = static_cast<int>(v.y);
        it.t0 = static_cast<int>(v.z);
        it.rows = static_cast<int>(v.w & 0xffffu);
        it.first = v.w >> 16 & 1u;
        it.last = v.w >> 17 & 1u;
        if (i % kDeal == kDeal - 1) {
            if (kWarp) __syncwarp();
            if (!kWarp || (threadIdx.x & 31) == 0) arrive_bar(MX_BAR(taken, set));
        }
        ++i;
        return it.rows > 0;
    }
};

// silu(g) * u = g / (1 + exp(-g)) * u. exp(-g) is infinite from -88.7 on, and 1 over
// it a subnormal number before, while u may be large: a negative gate's factor exp(g),
// as the square of exp(g / 2), is taken half with g and half with u, so that it
// underflows only where the result does. 2^-20 relative and |g| 2^-23.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float h = expf(-0.5f * fabsf(g));
    const float f = g < 0.f ? h : 1.0f;
    return g * f / (1.0f + h * h) * (u * f);
}

// The same for a bf16 result and gates not below kFarGate: the divisor is at most
// 2^116, so the exponential and the reciprocal may be the fast ones that flush
// subnormal numbers. 2^-20 relative and |g| 2^-23 from the rounded product with
// log2(e), 2^-16 at most, which leaves the result's rounding alone. (The form above
// for every gate cost gate/up prefill 5%.)
constexpr float kFarGate = -80.f;
__device__ __forceinline__ float silu_mul_near(float g, float u) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504f));  // log2(e)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return g * r * u;
}

// 32 TMEM lanes x 4 R columns: column 4 j + i of row group count R, i.e. word j
// of the R rows of this lane in turn.
__device__ __forceinline__ void store_words(uint32_t taddr, const uint4 (&w)[4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(w[0].x), "r"(w[1].x), "r"(w[2].x), "r"(w[3].x), "r"(w[0].y), "r"(w[1].y), "r"(w[2].y),
        "r"(w[3].y), "r"(w[0].z), "r"(w[1].z), "r"(w[2].z), "r"(w[3].z), "r"(w[0].w), "r"(w[1].w),
        "r"(w[2].w), "r"(w[3].w)
        : "memory");
}
__device__ __forceinline__ void store_words(uint32_t taddr, const uint4 (&w)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(w[0].x), "r"(w[1].x), "r"(w[2].x), "r"(w[3].x), "r"(w[4].x), "r"(w[5].x), "r"(w[6].x),
        "r"(w[7].x), "r"(w[0].y), "r"(w[1].y), "r"(w[2].y), "r"(w[3].y), "r"(w[4].y), "r"(w[5].y),
        "r"(w[6].y), "r"(w[7].y), "r"(w[0].z), "r"(w[1].z), "r"(w[2].z), "r"(w[3].z), "r"(w[4].z),
        "r"(w[5].z), "r"(w[6].z), "r"(w[7].z), "r"(w[0].w), "r"(w[1].w), "r"(w[2].w), "r"(w[3].w),
        "r"(w[4].w), "r"(w[5].w), "r"(w[6].w), "r"(w[7].w)
        : "memory");
}

// A stage's 16 bytes of scale row `row` (of `rows` in the matrix), loaded word by
// word; zeros past K.
__device__ __forceinline__ uint4 load_words(const uint8_t *src, size_t row, int K, int kb) {
    const uint32_t *u = reinterpret_cast<const uint32_t *>(src + row * (K / kMxBlock) + kb * 16);
    const int left = K / kMxWord - kb * KWORDS;
    return make_uint4(__ldg(u), left > 1 ? __ldg(u + 1) : 0u, left > 2 ? __ldg(u + 2) : 0u,
                      left > 3 ? __ldg(u + 3) : 0u);
}

// A scale warp: the words of the CTA's 128 weight rows (first output o_base of
// the tile's; once for a run of items) and of the tile's rows, stage by stage, to
// its TMEM quarter. Rows past the tile's end have any scales; their products are
// never stored.
template <typename C, bool kPair, bool kSilu>
__device__ __forceinline__ void bring_scales(const MxKernelParams &p, Ctl *ctl, uint32_t bars,
                                             uint32_t smem, uint32_t tmem_sf, int NO, int o_base,
                                             int tile_outputs, int nk) {
    static_assert(KWORDS == 4, "a row's 16 bytes are a stage");
    const int lane = threadIdx.x & 31;
    const uint32_t taddr = tmem_sf + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21);
    Walk<true> walk(ctl, bars, p.status);
    Item it;
    int as = 0, s = 0, slot = 0;       // of the rings of weight stages, row stages, TMEM columns
    int os = 0, warmup = C::SF_SLOTS;  // the row stage that used the columns before, if one did
    uint32_t aph = 0, ph = 0, oph = 0;
    while (walk.next(it)) {
        const int o_last = NO - 1 - it.wt * tile_outputs;
        for (int kb = 0; kb < nk; ++kb) {
            uint4 a[4], b[4 * C::NB];
            const bool load_a = !kPair || it.first;
            if (p.sf_tma) {
                if (kPair && it.first && !wait_bar<true>(MX_BAR(scaleda, as), aph, ctl, p.status)) return;
                if (!wait_bar<true>(MX_BAR(scaledb, s), ph, ctl, p.status)) return;
                const uint32_t sfa = smem + as * A_SLOT + A_BYTES + lane * 16;
                const uint32_t sfb = smem + NA * A_SLOT + s * C::B_SLOT + C::B_BYTES + lane * 16;
                if (load_a) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = ld_shared(sfa + i * 512);
                }
#pragma unroll
                for (int i = 0; i < 4 * C::NB; ++i) b[i] = i < C::R ? ld_shared(sfb + i * 512) : b[0];
            } else {
                if (load_a) {
                    if (kPair && !wait_bar<true>(MX_BAR(emptya, as), aph ^ 1u, ctl, p.status)) return;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // gate/up: 16 gate rows and their 16 up rows in turn
                        const int o = min(o_base + (kSilu ? i * 16 + (lane & 15) : i * 32 + lane), o_last);
                        a[i] = load_words(p.ws, static_cast<size_t>(it.wrow) + o + (kSilu && lane >= 16 ? NO : 0),
                                          p.K, kb);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4 * C::NB; ++i)
                    b[i] = i < C::R ? load_words(p.as, static_cast<size_t>(it.t0) + min(i * 32 + lane, it.rows - 1),
                                                 p.K, kb)
                                    : b[0];
            }
            // the MMAs that read the columns' last scales are done
            if (warmup > 0) {
                --warmup;
            } else {
                if (!wait_bar<true>(MX_BAR(emptyb, os), oph, ctl, p.status)) return;
                if (++os == C::STAGES) { os = 0; oph ^= 1u; }
            }
            tc_fence_after();
            if (load_a) {
                // a weight stage's columns are free with the stage itself; those of
                // single CTAs, whose SF_SLOTS are as many, with the rows'
                store_words(taddr + static_cast<uint32_t>(as * C::SFA_COLS), a);
                if (++as == NA) { as = 0; aph ^= 1u; }
            }
            store_words(taddr + static_cast<uint32_t>(NA * C::SFA_COLS + slot * C::SFB_COLS), b);
            if (++slot == C::SF_SLOTS) slot = 0;
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (kPair) arrive_leader(MX_BAR(fullb, s));
                else arrive_bar(MX_BAR(fullb, s));
            }
            if (++s == C::STAGES) { s = 0; ph ^= 1u; }
        }
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
// transposed to the warp's staging rows (kSub rows of the tile at a time, kPitch
// apart: no bank conflicts) and leave as 16-byte pieces, one a lane; fp32 leaves
// from the fragments, 32 bytes of four rows at a time.
template <bool kSilu, typename T>
struct Drain {
    static constexpr int kOutputs = kSilu ? 16 : 32;   // per warp
    static constexpr int kPieces = kOutputs / 8;       // 16-byte pieces of a row
    static constexpr int kSub = 32 / kPieces;          // rows: one piece a lane
    static constexpr int kPitch = kOutputs * 2 + 16;   // bytes
    static constexpr int kStage = sizeof(T) == 2 ? kSub * kPitch : 0;

    static __device__ __forceinline__ void run(uint32_t taddr, uint32_t stage, T *out, int f0, int NO,
                                               int lim, int lane) {
        uint32_t lo[16], hi[16];
        tmem_ld_16x256b_x4(taddr, lo);
        tmem_ld_16x256b_x4(taddr + (16u << 16), hi);
        tmem_ld_wait(lo);
        tmem_ld_wait(hi);
        if constexpr (kSilu) {
            // which form a value takes depends on its own gate alone; the branch only
            // saves the second form where no value of the thread needs it
            float least = 0.f;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < 16; ++i) least = fminf(least, __uint_as_float(lo[i]));
            }
            if (sizeof(T) == 2 && least >= kFarGate) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    lo[i] = __float_as_uint(silu_mul_near(__uint_as_float(lo[i]), __uint_as_float(hi[i])));
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float g = __uint_as_float(lo[i]), u = __uint_as_float(hi[i]);
                    lo[i] = __float_as_uint(sizeof(T) == 2 && !(g < kFarGate) ? silu_mul_near(g, u)
                                                                              : silu_mul(g, u));
                }
            }
            __syncwarp();  // the stores below are the whole warp's
        }
        if constexpr (sizeof(T) == 2) {
            // fragment registers 4g, 4g + 1 are rows 8g.. of outputs 0..7, 4g + 2
            // and 4g + 3 of outputs 8..15 (and hi of 16..31)
            auto pair_of = [](const uint32_t(&v)[16], int i) {
                return pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
            };
            const int m = lane >> 3;  // the 8 x 8 tile whose row this lane names
            const uint32_t at = kSilu ? stage + ((m >> 1) * 8 + (lane & 7)) * kPitch + (m & 1) * 16
                                      : stage + (lane & 7) * kPitch + m * 16;
            const uint32_t from = stage + lane / kPieces * kPitch + (lane % kPieces) * 16;
            const int col = f0 + (lane % kPieces) * 8;  // NO % 16 == 0: all 8 outputs or none
#pragma unroll
            for (int u = 0; u < 32 / kSub; ++u) {
                if constexpr (kSilu)
                    stmatrix_x4_trans(at, pair_of(lo, 4 * u), pair_of(lo, 4 * u + 1), pair_of(lo, 4 * u + 2),
                                      pair_of(lo, 4 * u + 3));
                else
                    stmatrix_x4_trans(at, pair_of(lo, 2 * u), pair_of(lo, 2 * u + 1), pair_of(hi, 2 * u),
                                      pair_of(hi, 2 * u + 1));
                __syncwarp();
                const uint4 v = ld_shared(from);
                const int r = u * kSub + lane / kPieces;
                if (r < lim && col < NO)
                    *reinterpret_cast<uint4 *>(out + static_cast<size_t>(r) * NO + col) = v;
                __syncwarp();  // the staging rows are read before the next are written
            }
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

template <int NT, bool kPair, bool kSilu, typename T>
__device__ __forceinline__ void mx_matmul_body(const CUtensorMap &tmW, const CUtensorMap &tmA,
                                               const CUtensorMap &tmSW, const CUtensorMap &tmSA,
                                               const MxKernelParams &p) {
    using C = Cfg<NT, kPair>;
    using X = Tc<kPair>;
    constexpr int kCtas = kPair ? 2 : 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *stages_out = smem + C::SLOTS_BYTES;           // the epilogue's staging rows
    Ctl *ctl = reinterpret_cast<Ctl *>(stages_out + kEpiWarps * Drain<kSilu, T>::kStage);
    int4 *items = reinterpret_cast<int4 *>(ctl + 1);       // [2][kDeal]
    int32_t *mts = reinterpret_cast<int32_t *>(items + 2 * kDeal);  // [E+1] prefix of row tiles
    int32_t *offs = mts + (p.E + 1);                        // [E+1]
    const uint32_t base = smem_u32(smem), bars = smem_u32(ctl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.E;
    const int half = kPair ? static_cast<int>(blockIdx.x & 1) : 0;  // rank in the cluster of two
    const bool leader = half == 0;

    if (threadIdx.x == 0) {
        // one kind of barrier may wait for an arrival that nothing makes (p.withheld)
        auto init = [&](uint64_t *bar, int count, int kind) { mbar_init(bar, count + (p.withheld == kind)); };
        for (int s = 0; s < C::STAGES; ++s) {
            // the rows' TMA thread (of the leader; both of a single CTA), the scale
            // warps (of both CTAs)
            init(&ctl->fullb[s], (kPair ? 1 : 2) + kCtas * kScaleWarps, kMxFullB);
            init(&ctl->scaledb[s], kPair ? 1 : 2, kMxScaledB);
            init(&ctl->emptyb[s], 1, kMxEmptyB);
        }
        for (int s = 0; s < NA; ++s) {
            init(&ctl->fulla[s], 1, kMxFullA);  // the weights' TMA thread (of the leader)
            init(&ctl->scaleda[s], 1, kMxScaledA);
            init(&ctl->emptya[s], 1, kMxEmptyA);
        }
        for (int b = 0; b < 2; ++b) {
            init(&ctl->tfull[b], 1, kMxTFull);
            init(&ctl->tempty[b], kCtas * kEpiWarps, kMxTEmpty);
            init(&ctl->dealt[b], 1, kMxDealt);
            // every role but the dealer; one CTA of a pair has no MMA thread
            init(&ctl->taken[b], 2 + kScaleWarps + kEpiWarps + (leader ? 1 : 0), kMxTaken);
        }
        mbar_init(&ctl->drain, 1);
        ctl->wait_ns = p.wait_ns;
        ctl->counts = p.counts;
        ctl->peer_abort = 0;
        if constexpr (kPair)
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(ctl->peer_abort)
                         : "r"(smem_u32(&ctl->abort)), "r"(half ^ 1));
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) X::alloc(&ctl->tmem_base, C::TMEM_COLS);
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmA);
        if (p.sf_tma) {
            tma_prefetch_desc(&tmSW);
            tma_prefetch_desc(&tmSA);
        }
    }
    pdl_trigger();
    pdl_wait();
    if (warp == 0) {
        // the plan: offsets brought into [0, rows], and the prefix of row tiles;
        // all offsets are loaded at once (one memory round trip)
        constexpr int kSets = (kMaxExperts + 32) / 32;
        int off[kSets];
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            const int i = u * 32 + lane;
            off[u] = i > E ? 0 : !p.offsets ? (i == 0 ? 0 : p.rows) : min(max(p.offsets[i], 0), p.rows);
        }
        int run = 0;
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            if (u * 32 > E) break;
            const int i = u * 32 + lane;
            int next = __shfl_down_sync(0xffffffffu, off[u], 1);
            const int first = __shfl_sync(0xffffffffu, off[u + 1 < kSets ? u + 1 : u], 0);
            if (lane == 31) next = first;
            const int tiles = i < E ? (max(next - off[u], 0) + NT - 1) / NT : 0;
            int x = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (i <= E) {
                mts[i] = run + x - tiles;
                offs[i] = off[u];
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
    // an out that fits in memory has far fewer tiles; offsets out of order may not
    const int total = static_cast<int>(min(static_cast<int64_t>(mts[E]) * NW, INT64_C(0x7fffffff)));
    // a run's weights stay in shared memory where all their stages fit
    const bool reuse = kPair && nk <= NA;
    // a pair takes a block of items, which holds the runs together; a single CTA
    // every gridDim.x-th one
    const int crew = gridDim.x / kCtas, member = blockIdx.x / kCtas;
    const int begin = kPair ? static_cast<int>(static_cast<int64_t>(total) * member / crew) : member;
    const int end = kPair ? static_cast<int>(static_cast<int64_t>(total) * (member + 1) / crew) : total;

    if (warp == 0 || warp == kThreads / 32 - 1) {
        if (elect_one()) {
            // ----------- TMA producers: the weights', the rows' -----------
            const bool weights = warp == 0;
            const int stages = weights ? NA : C::STAGES;
            int s = 0;
            uint32_t ph = 0;
            bool issued[kMaxStages];
            uint32_t issued_parity[kMaxStages];
            for (int i = 0; i < kMaxStages; ++i) issued[i] = false;
            bool ok = true;
            Walk<false> walk(ctl, bars, p.status);
            Item it;
            while (ok && walk.next(it)) {
                if (kPair && weights && !it.first) continue;
                const int wrow = it.wrow + half * kCtaOutputs;
                const int trow = it.t0 + half * (mma_n<C>(it) / 2);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!wait_bar<false>(kPair && weights ? MX_BAR(emptya, s) : MX_BAR(emptyb, s), ph ^ 1u, ctl, p.status)) {
                        ok = false;
                        break;
                    }
                    // the maps count two-byte columns: 64 of them are a box; what lies
                    // past K arrives as zeros. Scales: every CTA its own weight rows'
                    // and all of the tile's rows'
                    const int x = kb * KSUB * 64;
                    if (weights) {
                        const uint32_t sa = base + s * A_SLOT, full = kPair ? MX_BAR(fulla, s) : MX_BAR(fullb, s),
                                       scaled = kPair ? MX_BAR(scaleda, s) : MX_BAR(scaledb, s);
                        if (leader) arrive_bar_tx(full, kCtas * A_BYTES);
#pragma unroll
                        for (int j = 0; j < KSUB; ++j) {
                            if (kSilu) X::load_4d(sa + j * A_SUB, &tmW, x + j * 64, wrow / 16, full);
                            else X::load_2d(sa + j * A_SUB, &tmW, x + j * 64, wrow, full);
                        }
                        if (p.sf_tma) {
                            arrive_bar_tx(scaled, WM * 16);
                            if (kSilu) Tc<false>::load_4d(sa + A_BYTES, &tmSW, kb * 8, wrow / 16, scaled);
                            else Tc<false>::load_2d(sa + A_BYTES, &tmSW, kb * 8, wrow, scaled);
                        }
                    } else {
                        const uint32_t sb = base + NA * A_SLOT + s * C::B_SLOT, full = MX_BAR(fullb, s),
                                       scaled = MX_BAR(scaledb, s);
                        if (leader) arrive_bar_tx(full, kCtas * C::B_BYTES);
#pragma unroll
                        for (int j = 0; j < KSUB; ++j) X::load_2d(sb + j * C::B_SUB, &tmA, x + j * 64, trow, full);
                        if (p.sf_tma) {
                            arrive_bar_tx(scaled, NT * 16);
                            Tc<false>::load_2d(sb + C::B_BYTES, &tmSA, kb * 8, it.t0, scaled);
                        }
                    }
                    issued[s] = true;
                    issued_parity[s] = ph;
                    if (++s == stages) { s = 0; ph ^= 1u; }
                }
            }
            // (a pair's copies complete on the leader's barriers)
            if (!ok || aborted(ctl)) {  // our own copies land
                const uint64_t dl = globaltimer_ns() + kDrainNs;
                for (int i = 0; i < stages; ++i)
                    if (issued[i]) {
                        const bool a = kPair && weights;
                        if (leader) mbar_wait(a ? &ctl->fulla[i] : &ctl->fullb[i], issued_parity[i], dl);
                        if (p.sf_tma) mbar_wait(a ? &ctl->scaleda[i] : &ctl->scaledb[i], issued_parity[i], dl);
                    }
            }
        }
    } else if (warp == 1) {
        if (leader && elect_one()) {
            // ----------------------------- MMA ------------------------------
            const uint32_t desc0 = desc_low(base);
            int s = 0, tile = 0, slot = 0;
            int run_as = 0;               // first weight stage of the run
            uint32_t ph = 0, run_aph = 0;
            bool any = false;
            Walk<false> walk(ctl, bars, p.status);
            Item it;
            for (; walk.next(it); ++tile) {
                const int buf = tile & 1;
                const uint32_t use = static_cast<uint32_t>(tile >> 1);
                if (!wait_bar<false>(MX_BAR(tempty, buf), (use & 1u) ^ 1u, ctl, p.status)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * NT);
                const int n = mma_n<C>(it);
                const uint32_t idesc[2] = {idesc_mxf4(kCtas * WM, n, 0), idesc_mxf4(kCtas * WM, n, 1)};
                bool ok = true;
                int as = run_as;
                uint32_t aph = run_aph;
                for (int kb = 0; kb < nk; ++kb) {
                    if (kPair && it.first && !wait_bar<false>(MX_BAR(fulla, as), aph, ctl, p.status)) { ok = false; break; }
                    if (!wait_bar<false>(MX_BAR(fullb, s), ph, ctl, p.status)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = desc0 + static_cast<uint32_t>(as) * (A_SLOT / 16);
                    const uint32_t b0 = desc0 + (NA * A_SLOT + static_cast<uint32_t>(s) * C::B_SLOT) / 16;
                    const uint32_t ta = tmem_sf + static_cast<uint32_t>(as * C::SFA_COLS);
                    const uint32_t tb = tmem_sf + static_cast<uint32_t>(NA * C::SFA_COLS + slot * C::SFB_COLS);
#pragma unroll
                    for (int kk = 0; kk < BK / UK; ++kk)
                        X::mma(d_tmem, a0 + ((kk >> 2) * A_SUB + (kk & 3) * (UK / 2)) / 16,
                               b0 + ((kk >> 2) * C::B_SUB + (kk & 3) * (UK / 2)) / 16, idesc[kk & 1],
                               ta + 4 * (kk >> 1), tb + 4 * C::NB * (kk >> 1), (kb | kk) != 0 ? 1u : 0u);
                    if (++slot == C::SF_SLOTS) slot = 0;
                    any = true;
                    X::commit(MX_BAR(emptyb, s));
                    if (kPair && it.last) X::commit(MX_BAR(emptya, as));
                    if (++s == C::STAGES) { s = 0; ph ^= 1u; }
                    if (++as == NA) { as = 0; aph ^= 1u; }
                }
                if (!ok) break;
                X::commit(MX_BAR(tfull, buf));
                if (it.last) {
                    run_as = as;
                    run_aph = aph;
                }
            }
            if (any) {
                X::commit_here(MX_BAR(drain, 0));
                mbar_wait(&ctl->drain, 0, globaltimer_ns() + kWaitNs);
            }
        }
    } else if (warp < 2 + kScaleWarps) {
        // ---------------------------- scales ----------------------------
        bring_scales<C, kPair, kSilu>(p, ctl, bars, base, tmem_sf, NO, half * kCtaOutputs, kOutputs, nk);
    } else if (warp == kThreads / 32 - 2) {
        // ------------------------- item dealer --------------------------
        for (int c = 0;; ++c) {
            if (c >= 2 && !wait_bar<true>(MX_BAR(taken, c & 1), ((c >> 1) & 1u) ^ 1u, ctl, p.status)) break;
            const int64_t item = begin + (static_cast<int64_t>(c) * kDeal + lane) * (kPair ? 1 : crew);
            int4 it = make_int4(0, 0, 0, 0);
            if (lane < kDeal && item < end)
                it = decode(static_cast<int>(item), begin, end, reuse, NW, mts, offs, E, p.N, kOutputs, C::N_STEP);
            if (lane < kDeal) items[(c & 1) * kDeal + lane] = it;
            __syncwarp();
            if (lane == 0) arrive_bar(MX_BAR(dealt, c & 1));
            if (__any_sync(0xffffffffu, (lane < kDeal && it.w == 0) || aborted(ctl))) break;
        }
    } else {
        // --------------------------- epilogue ---------------------------
        const int q = warp & 3;                   // TMEM lane quarter of this warp
        const int ew = warp - 2 - kScaleWarps;
        const int c_first = (ew >> 2) * 32;       // its 32-column chunks, every second
        const uint32_t stage = smem_u32(stages_out) + ew * Drain<kSilu, T>::kStage;
        T *out = static_cast<T *>(p.out);
        int tile = 0;
        Walk<true> walk(ctl, bars, p.status);
        Item it;
        for (; walk.next(it); ++tile) {
            const int buf = tile & 1;
            const uint32_t use = static_cast<uint32_t>(tile >> 1);
            if (!wait_bar<true>(MX_BAR(tfull, buf), use & 1u, ctl, p.status)) break;
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
                if constexpr (kPair) arrive_leader(MX_BAR(tempty, buf));
                else arrive_bar(MX_BAR(tempty, buf));
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
    // After a time-out a stage's barrier may lack other roles' arrivals, or be in the
    // pair's other CTA, and not tell of a copy; nothing issues any more, and the CTA
    // stays until all have had the time to land.
    if (threadIdx.x == 0 && aborted(ctl)) {
        const uint64_t dl = globaltimer_ns() + kDrainNs;
        while (globaltimer_ns() < dl) __nanosleep(1000);
    }
}

template <int NT, bool kSilu, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    mx_matmul_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmSW,
                     const __grid_constant__ CUtensorMap tmSA, MxKernelParams p) {
    mx_matmul_body<NT, false, kSilu, T>(tmW, tmA, tmSW, tmSA, p);
}

template <int NT, bool kSilu, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_matmul_pair_kernel(const __grid_constant__ CUtensorMap tmW,
                          const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmSW,
                          const __grid_constant__ CUtensorMap tmSA, MxKernelParams p) {
    mx_matmul_body<NT, true, kSilu, T>(tmW, tmA, tmSW, tmSA, p);
}

// Waits that ran out in calls without a context (moe_mx_status). Only counted up, so
// that one thread's reading takes nothing from another's.
__device__ int g_mx_timeouts;

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

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Map of a scale matrix [rows][pitch bytes] in two-byte columns: a box is 16
// bytes of box_rows rows, or, with up_offset, of 4 groups of 16 rows and the 16
// rows up_offset further each (as tc_encode_pair_4d has it for the codes).
int encode_scales(CUtensorMap *m, const void *base, uint64_t rows, uint64_t pitch, uint32_t box_rows,
                  uint64_t up_offset) {
    static std::atomic<void *> found{nullptr};  // any thread may be the first
    void *fn = found.load(std::memory_order_relaxed);
    if (!fn) {
        cudaDriverEntryPointQueryResult q;
        void *ptr = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !ptr)
            return MOE_ERR_CUDA;
        found.store(fn = ptr, std::memory_order_relaxed);
    }
    const bool paired = up_offset != 0;
    const cuuint64_t dims[4] = {pitch / 2, paired ? 16 : rows, 2, paired ? (rows - up_offset) / 16 : 0};
    const cuuint64_t strides[3] = {pitch, pitch * up_offset, pitch * 16};
    const cuuint32_t box[4] = {8, paired ? 16 : box_rows, 2, 4};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    const CUresult r = reinterpret_cast<EncodeTiledFn>(fn)(
        m, CU_TENSOR_MAP_DATA_TYPE_UINT16, paired ? 4 : 2, const_cast<void *>(base), dims, strides, box,
        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
        CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <int NT, bool kPair, bool kSilu, typename T>
int launch(const MxMatmulParams &args, int n_sm, cudaStream_t s) {
    using C = Cfg<NT, kPair>;
    CUtensorMap w, a, sw = {}, sa = {};
    MxKernelParams p;
    static_cast<MxMatmulParams &>(p) = args;
    p.wait_ns = args.wait_us > 0 ? static_cast<uint64_t>(args.wait_us) * 1000u : kWaitNs;
    // TMA wants 16-byte row pitches and addresses
    p.sf_tma = p.K % BK == 0 && aligned(p.ws, 16) && aligned(p.as, 16);
    int rc;
    const uint64_t wrows = static_cast<uint64_t>(p.E) * p.N;
    if (kSilu) rc = tc_encode_pair_4d(&w, p.w, wrows, p.K / 4, p.N / 2);
    else rc = tc_encode_2d(&w, p.w, wrows, p.K / 4, WM);
    if (rc != MOE_OK) return rc;
    if ((rc = tc_encode_2d(&a, p.a, p.rows, p.K / 4, C::B_ROWS)) != MOE_OK) return rc;
    if (p.sf_tma) {
        const uint64_t pitch = p.K / kMxBlock;
        if ((rc = encode_scales(&sw, p.ws, wrows, pitch, WM, kSilu ? p.N / 2 : 0)) != MOE_OK ||
            (rc = encode_scales(&sa, p.as, p.rows, pitch, NT, 0)) != MOE_OK)
            return rc;
    }
    const size_t smem = 1024 + C::SLOTS_BYTES + kEpiWarps * Drain<kSilu, T>::kStage +
                        sizeof(Ctl) + 2 * kDeal * sizeof(int4) + 2 * (p.E + 1) * sizeof(int32_t);
    // no more CTAs than there can be items
    const int64_t items = static_cast<int64_t>(p.rows / NT + p.E) *
                          ((p.N + (kPair ? 2 : 1) * WM - 1) / ((kPair ? 2 : 1) * WM));
    if constexpr (kPair) {
        auto kern = mx_matmul_pair_kernel<NT, kSilu, T>;
        if (ensure_smem(kern, smem) != MOE_OK) return MOE_ERR_CUDA;
        // per kernel, for the device model of the process; any thread may be the first
        static const int resident = resident_pairs(reinterpret_cast<const void *>(kern), smem, n_sm);
        const int pairs = static_cast<int>(items < resident ? items : resident);
        return launch_k(kern, dim3(2 * pairs), dim3(kThreads), smem, s, w, a, sw, sa, p);
    } else {
        auto kern = mx_matmul_kernel<NT, kSilu, T>;
        if (ensure_smem(kern, smem) != MOE_OK) return MOE_ERR_CUDA;
        return launch_k(kern, dim3(static_cast<int>(items < n_sm ? items : n_sm)), dim3(kThreads), smem,
                        s, w, a, sw, sa, p);
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

int timeouts_address(int **out) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(out), g_mx_timeouts) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

}  // namespace

// The tile by the mean rows per expert (the counts themselves are on the
// device). Few rows are bound by the weights' stream: one CTA per 128 weight
// rows, tiles of 32 rows up to 16 per expert (64 experts, K 2048, I 1536: 38.8 us
// at 4 rows each, 39.4 in tiles of 48) and of 48 up to 48 (uneven loads of 32 on
// average: 27.1 us, 28.9 in tiles of 32; even ones of 64: 48.4, pairs 44.0).
// Above, pairs of CTAs with tiles of 192, unless the pairs' tiles would occupy
// less than two thirds of the GPU (one matrix, K 2048, N 6144: 256 rows 8.4 us in
// tiles of 48, 9.5 on pairs; 512 rows 9.2 us on pairs, 14.8 in tiles of 32).
int launch_mx_matmul(const MxMatmulParams &p, int n_sm, cudaStream_t s) {
    const int64_t pair_tiles = static_cast<int64_t>(p.rows / 192 + p.E) * ((p.N + 2 * WM - 1) / (2 * WM));
    if (p.rows <= 16 * p.E) return launch_nt<32, false>(p, n_sm, s);
    if (p.rows <= 48 * p.E || 3 * pair_tiles <= n_sm) return launch_nt<48, false>(p, n_sm, s);
    return launch_nt<192, true>(p, n_sm, s);
}

}  // namespace moe

using namespace moe;

static int matmul(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *w_codes,
                  const uint8_t *w_scales, const int32_t *offsets, int rows, int K, int n_experts,
                  int N, int silu_mul, void *out, int dtype, int wait_us, int withheld, void *stream) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (rows < 0 || (silu_mul != 0 && silu_mul != 1)) return MOE_ERR_INVALID_ARG;
    if (!offsets && n_experts != 1) return MOE_ERR_INVALID_ARG;
    if (K <= 0 || K > kMxMaxK || K % kMxWord != 0 || N <= 0 || N % (silu_mul ? 32 : 16) != 0)
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
    p.dtype = dtype; p.wait_us = wait_us; p.withheld = withheld;
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_NO_DEVICE;
    p.counts = 1;
    if (timeouts_address(&p.status) != MOE_OK) return MOE_ERR_CUDA;
    return launch_mx_matmul(p, n_sm, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_mx_matmul(const uint8_t *a_codes, const uint8_t *a_scales,
                             const uint8_t *w_codes, const uint8_t *w_scales,
                             const int32_t *offsets, int rows, int K, int n_experts, int N,
                             int silu_mul, void *out, int dtype, void *stream) {
    return matmul(a_codes, a_scales, w_codes, w_scales, offsets, rows, K, n_experts, N, silu_mul, out,
                  dtype, 0, 0, stream);
}

extern "C" int moe_mx_selftest_timeout(const uint8_t *a_codes, const uint8_t *a_scales,
                                       const uint8_t *w_codes, const uint8_t *w_scales,
                                       const int32_t *offsets, int rows, int K, int n_experts,
                                       int N, int silu_mul, void *out, int dtype, int timeout_us,
                                       int withheld, void *stream) {
    if (timeout_us <= 0 || timeout_us > 1000000 || withheld < 0 || withheld > kMxTaken)
        return MOE_ERR_INVALID_ARG;
    return matmul(a_codes, a_scales, w_codes, w_scales, offsets, rows, K, n_experts, N, silu_mul, out,
                  dtype, timeout_us, withheld, stream);
}

extern "C" int moe_mx_status(void) {
    constexpr int kMaxDevices = 64;
    static thread_local int seen[kMaxDevices];
    int *timeouts = nullptr, v = 0, dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || timeouts_address(&timeouts) != MOE_OK ||
        cudaDeviceSynchronize() != cudaSuccess ||
        cudaMemcpy(&v, timeouts, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (dev >= kMaxDevices) return MOE_ERR_NO_DEVICE;
    const bool more = v != seen[dev];
    seen[dev] = v;
    return more ? MOE_ERR_DEVICE_TIMEOUT : MOE_OK;
}
