// fp8_linear.cu -- the block's projections in 8 bits: e4m3 activations with a scale per token
// and 128 inputs, e4m3 weights with a scale per 128 x 128 block, on the tcgen05 tensor cores.
//
//   out[t, n] = sum_kb xs[t, kb] ws[n / 128, kb] * (sum_{k in block kb} xq[t, k] wq[n, k])
//
// The inner sums come from tcgen05.mma (kind::f8f6f4, fp32 accumulators in tensor memory),
// 128 inputs at a time: the accumulator is then read back, scaled and added to fp32 sums in
// registers, while the tensor core fills the other half of tensor memory with the next 128
// inputs.  Operand tiles come by TMA with 128-byte swizzle, a ring of stages deep; columns past
// k and rows past the arrays arrive as zeros.
//
// Two kernels:
//   prefill_kernel   256 tokens (the MMA's rows) x 256 outputs per tile, on persistent pairs of
//                    CTAs (cta_group::2): each loads half of either operand, which halves the
//                    weights' share of the shared-memory traffic that a 128 x 256 tile of one CTA is
//                    bound by.  A lane is a token, so its scale is one register a block.
//                    16384 tokens, 2560 -> 10240: 388 us back to back on the device, 2.2 PFLOP/s, the
//                    tensor pipe 52% busy (a pass behind a flush of L2 455-463 us); bound by the
//                    summing warps (without their multiply-adds 334 us, without their reads of
//                    tensor memory alone no less) and the hand-overs to and from them.
//   token_kernel     few tokens: bound by the weights' bytes.  128 outputs are the MMA's rows,
//                    the tokens its columns (16 to 64), and the inputs are cut into pieces over a
//                    cluster whose CTAs add their sums through distributed shared memory in
//                    a fixed order.
//
// Every wait is bounded: one that gives up sets the device error word and the CTA's abort
// flag, and all roles leave their loops.  The role that issued copies or products waits for the last
// of them (bounded too) before the CTA goes on to its end, whichever role gave up and also when none
// did; then tensor memory is freed and the kernel returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "layer_launch.h"
#include "row8.cuh"

namespace s6 {
namespace {

__device__ unsigned int g_linear_error = 0;
constexpr long long kLimit = 2000000000LL;  // SM clocks, about a second
constexpr unsigned kFull = 0xffffffffu;
constexpr int kBK = 128;  // inputs per stage: one scale block, one 128-byte swizzled row
constexpr int kBM = 128;  // rows of the MMA

struct Ctl {
    volatile int abort;
};

// Bounded wait that also leaves when another role of the CTA has given up.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Ctl* ctl) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (ctl->abort) return false;
        if (clock64() - start > kLimit) {
            ctl->abort = 1;
            atomicOr(&g_linear_error, 1u);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}

// ---- tcgen05 ---------------------------------------------------------------------------

// An allocation waits until the SM has the columns.  The waits end: the token kernel frees its
// columns before it waits for other CTAs, and the prefill kernel, whose CTAs hold theirs while they
// work with their pair, leaves no shared memory on its SMs for any CTA of these kernels.
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// The same on a pair of CTAs (ranks 2i and 2i + 1 of a cluster): the leader (even rank) issues
// products of 256 rows, 128 from each CTA's shared memory, and 256 columns, 128 from each; each
// CTA's tensor memory receives its own 128 rows.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// Arrives at the barrier at this offset in both CTAs once the leader's products are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile(
        "{\n .reg .b16 m;\n mov.b16 m, 3;\n"
        " tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::
            "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
        "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Shared-cluster address of a variable in the CTA of `rank`.
__device__ __forceinline__ uint32_t peer_addr(const void* local, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    return a;
}
// A load into this CTA's shared memory that completes on the pair leader's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1,
                                                 uint32_t leader_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(leader_bar)
        : "memory");
}
// An arrival at a barrier of the pair.  What it hands over is tensor memory, ordered by the
// tcgen05 fences; releasing at cluster scope would make the warp wait for all its memory accesses
// (that wait alone took two thirds of the kernel's time).
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
template <int R>
__device__ __forceinline__ void set_registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// 32 lanes x 32 columns; valid after tmem_ld_wait.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Uses of r stay behind this point (the registers pass through it).
__device__ __forceinline__ void pin32(uint32_t (&r)[32]) {
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                   "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                   "+r"(r[31])::"memory");
}
// The registers pass through the wait, so no use of them can be moved before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    pin32(r);
}
// acc += r * scale on 32 columns.  (Packed pairs were 7% slower for 16384 tokens, 2560 ->
// 10240.)
__device__ __forceinline__ void add_scaled(float* acc, const uint32_t (&r)[32], float scale) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(r[j]), scale, acc[j]);
}

// Tiled store shared -> global; what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_addr(src)), "r"(c0), "r"(c1)
                 : "memory");
}

// 32 lanes x 16 columns of fp32 accumulators; the values are valid after tmem_ld_wait(r).
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// The loaded registers pass through the wait, so no use of them can be moved before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// Shared-memory descriptor of a K-major tile of 128-byte rows in 128-byte swizzle (groups of 8
// rows, 1024 bytes apart).  A step of 32 inputs inside the row adds 32 bytes to the address.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Instruction descriptor: e4m3 x e4m3, fp32 accumulators, both operands K-major.
constexpr uint32_t mma_desc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Products of one 128-input stage: four steps of 32 inputs into accumulator columns d.
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint64_t da = tile_desc(a), db = tile_desc(b);
#pragma unroll
    for (int i = 0; i < kBK / 32; ++i) mma_f8(d, da + i * 2, db + i * 2, idesc, i > 0);
}

struct LParams {
    const float* xs;
    const float* ws;
    void* out;
    int64_t tokens, n, seqlen;  // seqlen 0: token-major output
    int kb;                     // blocks of 128 inputs
    int tiles_t, tiles_n;
    int out_tma;  // the output's rows can be described to TMA (16-byte multiples)
};

// Place of (token, output) in a channel-major output.
__device__ __forceinline__ int64_t cm_index(const LParams& p, int64_t t, int64_t n) {
    const int64_t b = t / p.seqlen;
    return (b * p.n + n) * p.seqlen + (t - b * p.seqlen);
}

// (The aligned forms take whole warps, whatever branch some lanes come from.)
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// ---- Many tokens -----------------------------------------------------------------------

constexpr int kPN = 256;                // outputs per tile
constexpr int kPT = 2 * kBM;             // tokens per tile of a pair of CTAs
constexpr int kPStages = 5;              // 5 x 32 KB a CTA
constexpr int kPWarps = 8;               // warps that keep the sums, 32 tokens x 128 outputs each
constexpr int kPCols = 128;
constexpr int kPThreads = 128 + 32 * kPWarps;
constexpr uint32_t kPStageBytes = 2 * kBM * kBK;  // 128 tokens and 128 weight rows
constexpr uint32_t kPStaging = 2 * 4096; // two rounds of output a warp gathers and stores
constexpr uint32_t kPSmem = kPStages * kPStageBytes + kPWarps * kPStaging + 1024;

// Registers: the block starts with 168 a thread; the four warps that hold no sums hand theirs
// over.  What is asked for may not exceed what the block started with.
constexpr int kPRegs = 65536 / kPThreads / 8 * 8, kPRegsLow = 56, kPRegsHigh = 224;
static_assert(128 * kPRegsLow + 32 * kPWarps * kPRegsHigh <= kPThreads * kPRegs, "register split");

struct PBars {
    uint64_t full[kPStages], empty[kPStages];  // operand ring (full: the leader's counts for both)
    uint64_t done[2], free[2];                 // accumulators: filled / read back (free: leader's)
    uint64_t drain;
    uint32_t tmem;
    Ctl ctl;
};

// A place in a ring of N and the parity of its current use.
template <int N>
struct Turn {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) at = 0, phase ^= 1u;
    }
};

// Stores a warp's 32 tokens (a lane each) x 128 outputs from registers.  The output goes through
// the warp's two pieces of 4 KB of shared memory in rounds, and from there by TMA (whole lines,
// tails cut off by the tensor's bounds, and the warp goes on while the copies run); outputs that
// TMA cannot describe, and channel-major pieces that span two sequences, are stored directly.
template <typename Tout>
__device__ __forceinline__ void store_tile(const LParams& p, const CUtensorMap* mo, uint8_t* stage, int64_t t0,
                                           int64_t n0, int lane, const float (&acc)[kPCols]) {
    constexpr int kPer = 16 / sizeof(Tout);   // outputs in 16 bytes
    constexpr int kRound = 128 / sizeof(Tout);  // token-major: outputs of a 128-byte row
    constexpr int kRoundCm = 4096 / 32 / sizeof(Tout);  // channel-major: outputs of a 4 KB round
    const int64_t t = t0 + lane;
    Tout* out = static_cast<Tout*>(p.out);
    if (p.seqlen == 0) {
#pragma unroll
        for (int r = 0; r < kPCols / kRound; ++r) {
            uint8_t* st = stage + (r & 1) * 4096;
            if (p.out_tma && lane == 0) tma_store_wait_read<1>();  // the round before the last has left its piece
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {  // 128-byte swizzle: piece c of row i at c ^ (i % 8)
                alignas(16) Tout v[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j) v[j] = io<Tout>::from_f(acc[r * kRound + c * kPer + j]);
                *reinterpret_cast<uint4*>(st + lane * 128 + ((c ^ (lane & 7)) * 16)) = *reinterpret_cast<uint4*>(v);
            }
            const int64_t col0 = n0 + r * kRound;
            if (p.out_tma) {
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(mo, st, (int)col0, (int)t0);
                    tma_store_commit();
                }
                continue;
            }
            // Rows that begin anywhere: the lanes run along a row, 4 bytes each.  (A lane storing its own
            // token's row touches 32 lines a store: 166 us against 53 for 4096 tokens, 2560 -> 3001.)
            __syncwarp();
            const int rows = (int)min((int64_t)32, p.tokens - t0);
            constexpr int kEach = 4 / sizeof(Tout);
            const int64_t col = col0 + lane * kEach;
#pragma unroll 4
            for (int i = 0; i < rows; ++i) {
                const uint32_t v = *reinterpret_cast<const uint32_t*>(st + i * 128 + (((lane >> 2) ^ (i & 7)) * 16) +
                                                                       (lane & 3) * 4);
                Tout* o = out + (t0 + i) * p.n + col;
                if (col + kEach <= p.n && (reinterpret_cast<uintptr_t>(o) & 3) == 0) {
                    *reinterpret_cast<uint32_t*>(o) = v;
                } else {
                    const Tout* e = reinterpret_cast<const Tout*>(&v);
#pragma unroll
                    for (int j = 0; j < kEach; ++j)
                        if (col + j < p.n) o[j] = e[j];
                }
            }
        }
        return;
    }
    const int64_t b = t0 / p.seqlen, l0 = t0 - b * p.seqlen;
    if (p.out_tma && (l0 + 32 <= p.seqlen || t0 + (p.seqlen - l0) >= p.tokens)) {
#pragma unroll
        for (int r = 0; r < kPCols / kRoundCm; ++r) {
            Tout* st = reinterpret_cast<Tout*>(stage + (r & 1) * 4096);
            if (lane == 0) tma_store_wait_read<1>();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kRoundCm; ++c) st[c * 32 + lane] = io<Tout>::from_f(acc[r * kRoundCm + c]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(mo, st, (int)l0, (int)n0 + r * kRoundCm, (int)b);
                tma_store_commit();
            }
        }
    } else if (t < p.tokens) {
        Tout* o = out + cm_index(p, t, n0);
#pragma unroll
        for (int c = 0; c < kPCols; ++c)
            if (n0 + c < p.n) o[c * p.seqlen] = io<Tout>::from_f(acc[c]);
    }
}

// A pair of CTAs per tile.  In each, warp 0 loads (its 128 tokens and its half of the weight
// rows), warp 1 of the leader issues the products, warp 2 owns tensor memory; warps 4-11 keep the
// sums of the CTA's tokens: warp w holds lanes (w % 4) * 32 .. and columns ((w - 4) / 4) * 128 ..,
// 128 sums a thread.
template <typename Tout>
__global__ void __launch_bounds__(kPThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
               const __grid_constant__ CUtensorMap mo, const LParams p) {
    extern __shared__ uint8_t dyn[];
    __shared__ PBars bars;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.tiles_t * p.tiles_n;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPStages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bars.done[i], 1), mbar_init(&bars.free[i], 2 * kPWarps);
        mbar_init(&bars.drain, 1);
        bars.ctl.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc_pair(&bars.tmem, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp < 4) {
        set_registers_down<kPRegsLow>();
        if (warp == 0) {
            if (elect_one()) {
                Turn<kPStages> s;
                int used = 0;  // stages that have been filled
                bool ok = true;
                for (int tile = pair; tile < tiles && ok; tile += pairs) {
                    const int tt = tile / p.tiles_n, tn = tile - tt * p.tiles_n;
                    for (int k = 0; k < p.kb; ++k, s.next()) {
                        if (!wait_or_abort(&bars.empty[s.at], s.phase ^ 1u, &bars.ctl)) {
                            ok = false;
                            break;
                        }
                        uint8_t* st = ring + s.at * kPStageBytes;
                        const uint32_t full = peer_addr(&bars.full[s.at], 0);
                        if (rank == 0) mbar_arrive_expect_tx(&bars.full[s.at], 2 * kPStageBytes);
                        tma_load_2d_pair(st, &mx, k * kBK, tt * kPT + (int)rank * kBM, full);
                        tma_load_2d_pair(st + kBM * kBK, &mw, k * kBK, tn * kPN + (int)rank * kBM, full);
                        used = max(used, s.at + 1);
                    }
                }
                // The pair does not end before the copies into it have (the last use of each stage): a role
                // that gives up may do so long after the last of them was issued.
                if (rank == 0)
                    for (int j = 0; j < used; ++j)
                        mbar_wait_bounded(&bars.full[j], j < s.at ? s.phase : s.phase ^ 1u, kLimit / 8);
            }
        } else if (warp == 1 && rank == 0) {
            if (elect_one()) {
                constexpr uint32_t idesc = mma_desc(kPT, kPN);
                Turn<kPStages> s;
                Turn<2> d;
                bool ok = true;
                for (int tile = pair; tile < tiles && ok; tile += pairs) {
                    for (int k = 0; k < p.kb; ++k, s.next(), d.next()) {
                        if (!wait_or_abort(&bars.full[s.at], s.phase, &bars.ctl) ||
                            !wait_or_abort(&bars.free[d.at], d.phase ^ 1u, &bars.ctl)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t a = smem_addr(ring + s.at * kPStageBytes);
                        const uint64_t da = tile_desc(a), db = tile_desc(a + kBM * kBK);
#pragma unroll
                        for (int i = 0; i < kBK / 32; ++i)
                            mma_f8_pair(tmem + d.at * kPN, da + i * 2, db + i * 2, idesc, i > 0);
                        tc_commit_pair(&bars.done[d.at]);
                        tc_commit_pair(&bars.empty[s.at]);
                    }
                }
                tc_commit_pair(&bars.drain);
            }
        }
    } else {
        set_registers_up<kPRegsHigh>();
        const int part = (warp - 4) >> 2, quad = warp & 3;
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + part * kPCols;
        uint8_t* stage = ring + kPStages * kPStageBytes + (warp - 4) * kPStaging;
        const uint32_t free0 = peer_addr(&bars.free[0], 0), free1 = peer_addr(&bars.free[1], 0);
        Turn<2> d;
        uint32_t ra[32], rb[32];
        int64_t t0, n0;  // the warp's first token and output of a tile
        const float *xs, *ws;
        float xn, wn;  // the scales of the block to come
        const auto begin = [&](int tile) {
            const int tt = tile / p.tiles_n, tn = tile - tt * p.tiles_n;
            t0 = (int64_t)tt * kPT + rank * kBM + quad * 32;
            n0 = (int64_t)tn * kPN + part * kPCols;
            const bool in = t0 + lane < p.tokens && n0 < p.n;
            xs = p.xs + (in ? t0 + lane : 0) * p.kb;
            ws = p.ws + (in ? n0 / kGroup : 0) * p.kb;
            xn = __ldg(xs), wn = __ldg(ws);
        };
        if (pair < tiles) begin(pair);
        bool ok = __all_sync(kFull, wait_or_abort(&bars.done[0], 0, &bars.ctl));
        tc_fence_after();
        if (ok) tmem_ld32(base, ra);
        for (int tile = pair; tile < tiles && ok; tile += pairs) {
            float acc[kPCols];
#pragma unroll
            for (int i = 0; i < kPCols; ++i) acc[i] = 0.f;
            for (int k = 0; k < p.kb; ++k) {
                const float sc = xn * wn;
                if (k + 1 < p.kb) xn = __ldg(xs + k + 1), wn = __ldg(ws + k + 1);  // used a block later
                // Columns in four pieces of 32: the next piece is on its way while one is added.
                const uint32_t at = base + d.at * kPN;
                tmem_ld_wait(ra);
                tmem_ld32(at + 32, rb);
                add_scaled(acc, ra, sc);
                tmem_ld_wait(rb);
                tmem_ld32(at + 64, ra);
                add_scaled(acc + 32, rb, sc);
                tmem_ld_wait(ra);
                tmem_ld32(at + 96, rb);
                add_scaled(acc + 64, ra, sc);
                tmem_ld_wait(rb);
                // the accumulator is in registers: the next products may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at(d.at ? free1 : free0);
                // the first piece of the next block (this tile's or the next one's)
                d.next();
                if (k + 1 < p.kb || tile + pairs < tiles) {
                    ok = __all_sync(kFull, wait_or_abort(&bars.done[d.at], d.phase, &bars.ctl));
                    if (!ok) break;
                    tc_fence_after();
                    tmem_ld32(base + d.at * kPN, ra);
                }
                add_scaled(acc + 96, rb, sc);
            }
            if (!ok) break;
            const int64_t t_done = t0, n_done = n0;
            if (tile + pairs < tiles) begin(tile + pairs);  // its first scales arrive during the stores
            if (n_done < p.n && t_done < p.tokens) store_tile<Tout>(p, &mo, stage, t_done, n_done, lane, acc);
            __syncwarp();  // the next load of tensor memory takes the whole warp
        }
        if (lane == 0) tma_store_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    // ... nor before the products, which read the pair's shared memory, write its tensor memory and
    // signal both CTAs
    if (warp == 1) {
        if (elect_one()) mbar_wait_bounded(&bars.drain, 0, kLimit / 8);
        __syncwarp();
    }
    cluster_sync();  // neither CTA ends while the other may still signal it or read its memory
    tc_fence_after();
    if (warp == 2) tmem_free_pair(tmem, 512);
}

// ---- Few tokens ------------------------------------------------------------------------

constexpr int kTThreads = 192;  // warps 0-3 keep the sums, warp 4 loads, warp 5 issues products
constexpr int kTStages = 6;     // at most, of the operand ring
constexpr int kTTurns = 8;      // at most, accumulators in tensor memory

struct TBars {
    uint64_t full[kTStages], empty[kTStages];
    uint64_t done[kTTurns], free[kTTurns];
    uint64_t drain;
    uint32_t tmem;
    Ctl ctl;
};

template <int BN>
constexpr uint32_t token_stage_bytes() { return (kBM + BN) * kBK; }
// Accumulators kept at once: as many as fit in half of tensor memory (two CTAs share an SM).
template <int BN>
constexpr int token_turns() { return 256 / BN < kTTurns ? 256 / BN : kTTurns; }
constexpr int kTPitch = kBM + 4;  // floats between the sums of two tokens

__device__ __forceinline__ float4 peer_load4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// Grid (pieces, output tiles, token tiles), a cluster of `pieces` CTAs along x.  Piece q takes
// input blocks [kb q / pieces, kb (q + 1) / pieces); the pieces' sums are added in order of
// piece, each CTA adding and storing its share of the tile's outputs.
template <int BN, typename Tout>
__global__ void __launch_bounds__(kTThreads)
token_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
             const LParams p, int stages) {
    extern __shared__ uint8_t dyn[];
    __shared__ TBars bars;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    constexpr uint32_t kStage = token_stage_bytes<BN>();
    constexpr int kTurns = token_turns<BN>();
    constexpr uint32_t kCols = kTurns * BN;
    float* red = reinterpret_cast<float*>(ring);                        // [BN][kTPitch], after the products
    float* scl = reinterpret_cast<float*>(ring + (size_t)stages * kStage);  // [blocks][BN] scales
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pieces = (int)gridDim.x, piece = (int)cluster_rank();
    const int k0 = (int)((int64_t)p.kb * piece / pieces), k1 = (int)((int64_t)p.kb * (piece + 1) / pieces);
    const int64_t n0 = (int64_t)blockIdx.y * kBM, t0 = (int64_t)blockIdx.z * BN;
    const CUtensorMap *map_x = &mx, *map_w = &mw;
    const auto load = [=](int k, int s) {
        uint8_t* st = ring + (size_t)s * kStage;
        uint64_t* full = &bars.full[s];
        mbar_arrive_expect_tx(full, kStage);
        tma_load_2d(st, map_w, k * kBK, (int)n0, full);
        tma_load_2d(st + kBM * kBK, map_x, k * kBK, (int)t0, full);
    };
    const int ahead = min(stages, k1 - k0);  // blocks that find their stage empty
    if (warp == 4 && elect_one()) {
        for (int i = 0; i < stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < kTurns; ++i) mbar_init(&bars.done[i], 1), mbar_init(&bars.free[i], 4);
        mbar_init(&bars.drain, 1);
        bars.ctl.abort = 0;
        fence_barrier_init();
        // the first loads are on their way while the others set up
        for (int i = 0; i < ahead; ++i) load(k0 + i, i);
    }
    if (warp == 5) tmem_alloc(&bars.tmem, kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    if (warp == 4) {
        if (elect_one()) {
            int s = 0;
            uint32_t phase = 1;
            for (int k = k0 + ahead; k < k1; ++k) {  // ahead == stages here: stage 0 comes next
                if (!wait_or_abort(&bars.empty[s], phase ^ 1u, &bars.ctl)) break;
                load(k, s);
                if (++s == stages) s = 0, phase ^= 1u;
            }
            // the CTA does not end before the copies into it have (see prefill_kernel)
            for (int j = 0; j < ahead; ++j) mbar_wait_bounded(&bars.full[j], j < s ? phase : phase ^ 1u, kLimit / 8);
        }
    } else if (warp == 5) {
        if (elect_one()) {
            constexpr uint32_t idesc = mma_desc(kBM, BN);
            int s = 0;
            uint32_t phase = 0;
            Turn<kTurns> d;
            for (int k = k0; k < k1; ++k, d.next()) {
                if (!wait_or_abort(&bars.free[d.at], d.phase ^ 1u, &bars.ctl) ||
                    !wait_or_abort(&bars.full[s], phase, &bars.ctl))
                    break;
                tc_fence_after();
                const uint32_t a = smem_addr(ring + (size_t)s * kStage);
                mma_stage(tmem + d.at * BN, a, a + kBM * kBK, idesc);
                tc_commit(&bars.done[d.at]);
                tc_commit(&bars.empty[s]);
                if (++s == stages) s = 0, phase ^= 1u;
            }
            tc_commit(&bars.drain);  // ... nor before the products
            mbar_wait_bounded(&bars.drain, 0, kLimit / 8);
        }
    } else {
        // token scales times the tile's weight scales, by block and column, while the tiles load
        const float* ws = p.ws + (n0 / kGroup) * p.kb + k0;
#pragma unroll 4
        for (int i = threadIdx.x; i < (k1 - k0) * BN; i += 128) {
            const int c = i % BN, k = i / BN;
            scl[i] = t0 + c < p.tokens ? __ldg(p.xs + (t0 + c) * p.kb + k0 + k) * __ldg(ws + k) : 0.f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
        float acc[BN];
#pragma unroll
        for (int i = 0; i < BN; ++i) acc[i] = 0.f;
        Turn<kTurns> d;
        for (int k = k0; k < k1; ++k, d.next()) {
            if (!__all_sync(kFull, wait_or_abort(&bars.done[d.at], d.phase, &bars.ctl))) break;
            tc_fence_after();
            const float* sc = scl + (k - k0) * BN;
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
                uint32_t r[16];
                tmem_ld16(base + d.at * BN + c * 16, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(sc + c * 16 + j);
                    acc[c * 16 + j] = fmaf(__uint_as_float(r[j]), s4.x, acc[c * 16 + j]);
                    acc[c * 16 + j + 1] = fmaf(__uint_as_float(r[j + 1]), s4.y, acc[c * 16 + j + 1]);
                    acc[c * 16 + j + 2] = fmaf(__uint_as_float(r[j + 2]), s4.z, acc[c * 16 + j + 2]);
                    acc[c * 16 + j + 3] = fmaf(__uint_as_float(r[j + 3]), s4.w, acc[c * 16 + j + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.free[d.at]);
        }
        // All of this CTA's products are done (each was waited for), and with them its operand
        // tiles: the ring takes the sums.
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!bars.ctl.abort) {
#pragma unroll
            for (int i = 0; i < BN; ++i) red[i * kTPitch + warp * 32 + lane] = acc[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp == 5) tmem_free(tmem, kCols);
    const bool bad = bars.ctl.abort != 0;
    cluster_sync();
    if (!bad) {
        // This CTA's share of the 128 outputs of every token, four at a time.  Channel-major, the
        // lanes run along the tokens, which are the output's inner axis.
        const int quad0 = kBM / 4 * piece / pieces, quads = kBM / 4 * (piece + 1) / pieces - quad0;
        const bool along_tokens = p.seqlen > 1;
        uint32_t peer[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) peer[q] = peer_addr(red, (uint32_t)(q < pieces ? q : 0));
        Tout* out = static_cast<Tout*>(p.out);
        const int64_t b0 = along_tokens ? t0 / p.seqlen : 0;
        for (int i = threadIdx.x; i < quads * BN; i += kTThreads) {
            const int c = along_tokens ? i % BN : i / quads;
            const int row = (quad0 + (along_tokens ? i / BN : i % quads)) * 4;
            const int64_t t = t0 + c, n = n0 + row;
            if (t >= p.tokens || n >= p.n) continue;
            float4 u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < pieces) u[q] = peer_load4(peer[q] + (uint32_t)(c * kTPitch + row) * 4);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < pieces) v[0] += u[q].x, v[1] += u[q].y, v[2] += u[q].z, v[3] += u[q].w;
            if (along_tokens) {
                int64_t b = b0, l = t - b0 * p.seqlen;
                while (l >= p.seqlen) l -= p.seqlen, ++b;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.n) out[(b * p.n + n + j) * p.seqlen + l] = io<Tout>::from_f(v[j]);
            } else if (p.n % 4 == 0) {
                alignas(16) Tout o[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = io<Tout>::from_f(v[j]);
                struct alignas(4 * sizeof(Tout)) Four { Tout o[4]; };
                *reinterpret_cast<Four*>(out + t * p.n + n) = *reinterpret_cast<const Four*>(o);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n + j < p.n) out[t * p.n + n + j] = io<Tout>::from_f(v[j]);
            }
        }
    }
    // A CTA's shared memory outlives its peers' reads.  They are done (their values were used), so the
    // arrival need not wait for the outputs' way to memory as a releasing one does.
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

// ---- host ------------------------------------------------------------------------------

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeFn encoder() {
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(ptr);
    });
    return fn;
}

// (rows, k) bytes in boxes of 128 columns x box_rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, int64_t k, int64_t rows, int box_rows) {
    const EncodeFn enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)k};
    cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Multiprocessors of the current device, asked once per device.
int multiprocessors() {
    static std::atomic<int> known[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) return 148;
    known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// The output for the prefill kernel's stores: 32 tokens x 128 bytes of outputs in 128-byte
// swizzle, or channel-major 32 tokens x 4 KB of outputs.  False where TMA cannot describe it.
template <typename Tout>
bool encode_out(CUtensorMap* m, const LinearArgs& a) {
    const EncodeFn enc = encoder();
    const int64_t inner = a.seqlen ? a.seqlen : a.n;
    if (!enc || inner * (int64_t)sizeof(Tout) % 16 != 0) return false;
    const CUtensorMapDataType dt =
        sizeof(Tout) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    cuuint32_t estr[3] = {1, 1, 1};
    if (!a.seqlen) {
        cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.tokens};
        cuuint64_t strides[1] = {(cuuint64_t)a.n * sizeof(Tout)};
        cuuint32_t box[2] = {128 / sizeof(Tout), 32};
        return enc(m, dt, 2, a.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    cuuint64_t dims[3] = {(cuuint64_t)a.seqlen, (cuuint64_t)a.n, (cuuint64_t)(a.tokens / a.seqlen)};
    cuuint64_t strides[2] = {(cuuint64_t)a.seqlen * sizeof(Tout), (cuuint64_t)a.seqlen * a.n * sizeof(Tout)};
    cuuint32_t box[3] = {32, 4096 / 32 / sizeof(Tout), 1};
    return enc(m, dt, 3, a.out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Tout>
cudaError_t run_prefill(const LinearArgs& a, LParams p, cudaStream_t s) {
    CUtensorMap mx, mw, mo;
    memset(&mo, 0, sizeof(mo));
    if (!encode_rows(&mx, a.xq, a.k, a.tokens, kBM) || !encode_rows(&mw, a.wq, a.k, a.n, kBM))
        return cudaErrorInvalidValue;
    p.out_tma = encode_out<Tout>(&mo, a) ? 1 : 0;
    p.tiles_t = (int)((a.tokens + kPT - 1) / kPT);
    p.tiles_n = (int)((a.n + kPN - 1) / kPN);
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
    if (e != cudaSuccess) return e;
    const int64_t pairs = std::min<int64_t>((int64_t)p.tiles_t * p.tiles_n, std::max(1, multiprocessors() / 2));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kPThreads);
    cfg.dynamicSmemBytes = kPSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_kernel<Tout>, mx, mw, mo, p);
}

// Pieces of the inputs per tile: up to 8 (a portable cluster), while all pieces run at once and
// each has at least two blocks.  Two CTAs fit on an SM; clusters of three and more do not fill
// every SM of a GPC, so they get a ninth fewer places.
int token_pieces(int64_t tiles, int kb) {
    const int64_t slots = 2 * (int64_t)multiprocessors();
    int64_t pieces = 8;
    while (pieces > 1 && (tiles * pieces > (pieces > 2 ? slots * 8 / 9 : slots) || pieces * 2 > kb)) --pieces;
    return (int)pieces;
}

// Which kernel: the token kernel with tiles of 16, 32 or 64 tokens, or (0) the prefill kernel.  Each
// one's time is close to a straight line in the input blocks that a CTA walks one after another,
// times the waves of CTAs; fitted to launches of (16 .. 4096 tokens) x (80 .. 10240 outputs) x
// (1536 .. 10240 inputs), weights in L2:
//   prefill  7 us + 0.39 us a block        token, 64  7 us + 0.60
//   token, 32  6 us + 0.40                 token, 16  5 us + 0.28
// Narrow tiles cut a call into more CTAs, wide ones read the weights fewer times.  Measured, 16, 32, 64
// and prefill: 32 tokens, 5120 -> 2560: 7.1, 8.2, 9.3, 21.6 us; 64 tokens, 2560 -> 5120: 10.5, 8.9,
// 10.1, 13.7; 256 tokens, 5120 -> 2560: -, 21.2, 15.4, 22.6; 128 tokens, 2560 -> 10240: -, 23.8, 19.7,
// 15.1.
int best_columns(const LinearArgs& a, int kb) {
    struct Line { int columns; double fixed, block; };
    constexpr Line kToken[3] = {{16, 5.0, 0.28}, {32, 6.0, 0.40}, {64, 7.0, 0.60}};
    const int64_t sms = multiprocessors();
    const auto ceil_div = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    int best = 0;
    double least = 7.0 + 0.39 * kb * (double)ceil_div(ceil_div(a.tokens, kPT) * ceil_div(a.n, kPN),
                                                      std::max<int64_t>(1, sms / 2));
    for (const Line& l : kToken) {
        const int64_t tiles = ceil_div(a.n, kBM) * ceil_div(a.tokens, l.columns);
        const int pieces = token_pieces(tiles, kb);
        const double time = l.fixed + l.block * (double)ceil_div(kb, pieces) * (double)ceil_div(tiles * pieces, 2 * sms);
        if (time < least) least = time, best = l.columns;
    }
    return best;
}

template <int BN, typename Tout>
cudaError_t run_token(const LinearArgs& a, const LParams& p, cudaStream_t s) {
    CUtensorMap mx, mw;
    if (!encode_rows(&mx, a.xq, a.k, a.tokens, BN) || !encode_rows(&mw, a.wq, a.k, a.n, kBM))
        return cudaErrorInvalidValue;
    const int64_t tn = (a.n + kBM - 1) / kBM, tt = (a.tokens + BN - 1) / BN;
    if (tn > 65535 || tt > 65535) return run_prefill<Tout>(a, p, s);  // beyond a grid's y and z
    const int pieces = token_pieces(tn * tt, p.kb);
    const int blocks = (p.kb + pieces - 1) / pieces;
    constexpr uint32_t kStage = token_stage_bytes<BN>();
    constexpr int kLeast = (BN * kTPitch * 4 + kStage - 1) / kStage;  // the ring also holds the tile's sums
    static_assert(kLeast <= kTStages, "the sums fit in the ring");
    constexpr int64_t kMost = 226 * 1024;
    // a ring that leaves room for a second CTA on the SM
    int stages = std::max(std::min<int>(blocks, std::min<int>(kTStages, 100 * 1024 / kStage)), kLeast);
    const int64_t scales = (int64_t)blocks * BN * 4 + 1024;
    while (stages > kLeast && stages * (int64_t)kStage + scales > kMost) --stages;
    if (stages * (int64_t)kStage + scales > kMost) return run_prefill<Tout>(a, p, s);  // k above 80,000
    const uint32_t smem = (uint32_t)(stages * (int64_t)kStage + scales);
    cudaError_t e = cudaFuncSetAttribute(token_kernel<BN, Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pieces, (unsigned)tn, (unsigned)tt);
    cfg.blockDim = dim3(kTThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)pieces;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, token_kernel<BN, Tout>, mx, mw, p, stages);
}

template <typename Tout>
cudaError_t run_linear(const LinearArgs& a, cudaStream_t s) {
    LParams p;
    p.xs = a.xs;
    p.ws = a.ws;
    p.out = a.out;
    p.tokens = a.tokens;
    p.n = a.n;
    p.seqlen = a.seqlen;
    p.kb = (int)((a.k + kBK - 1) / kBK);
    p.tiles_t = p.tiles_n = p.out_tma = 0;
    switch (best_columns(a, p.kb)) {
        case 16: return run_token<16, Tout>(a, p, s);
        case 32: return run_token<32, Tout>(a, p, s);
        case 64: return run_token<64, Tout>(a, p, s);
        default: return run_prefill<Tout>(a, p, s);
    }
}

// One bounded wait on a barrier that nothing completes, as mamba_diag_wait_timeout_in describes.
__global__ void timeout_probe_kernel(long long limit_cycles) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
        if (!mbar_wait_bounded(&bar, 0, limit_cycles)) atomicOr(&g_linear_error, 1u);
    }
}

}  // namespace

cudaError_t launch_fp8_linear(const LinearArgs& a, cudaStream_t s) {
    if (a.tokens == 0 || a.n == 0) return cudaSuccess;
    return a.out_dtype == DType::BF16 ? run_linear<__nv_bfloat16>(a, s) : run_linear<float>(a, s);
}

cudaError_t launch_linear_timeout_probe(long long limit_cycles, cudaStream_t s) {
    timeout_probe_kernel<<<1, 32, 0, s>>>(limit_cycles);
    return cudaGetLastError();
}

cudaError_t linear_error_word(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_linear_error);
}

}  // namespace s6
