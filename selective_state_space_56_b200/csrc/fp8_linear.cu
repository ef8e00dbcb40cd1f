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
//   prefill_kernel   128 tokens (the MMA's rows) x 256 outputs per tile, persistent CTAs.  A
//                    lane is a token, so its scale is one register a block.
//   token_kernel     few tokens: bound by the weights' bytes.  128 outputs are the MMA's rows,
//                    the tokens its columns (16 to 128), and the inputs are cut into pieces over a
//                    cluster whose CTAs add their sums through distributed shared memory in
//                    a fixed order.
//
// Every wait is bounded: one that gives up sets the device error word and the CTA's abort
// flag, all roles leave their loops, outstanding copies and products are waited for (bounded
// too), tensor memory is freed and the kernel returns.
#include <cudaTypedefs.h>

#include <algorithm>
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
};

template <typename Tout>
__device__ __forceinline__ int64_t out_index(const LParams& p, int64_t t, int64_t n) {
    if (p.seqlen == 0) return t * p.n + n;
    const int64_t b = t / p.seqlen;
    return (b * p.n + n) * p.seqlen + (t - b * p.seqlen);
}

// ---- Many tokens -----------------------------------------------------------------------

constexpr int kPN = 256;      // outputs per tile
constexpr int kPStages = 4;   // 4 x 48 KB
constexpr int kPThreads = 384;
constexpr uint32_t kPStageBytes = (kBM + kPN) * kBK;
constexpr uint32_t kPSmem = kPStages * kPStageBytes + 1024;

struct PBars {
    uint64_t full[kPStages], empty[kPStages];  // operand ring
    uint64_t done[2], free[2];                 // accumulators: filled / read back
    uint64_t drain;
    uint32_t tmem;
    Ctl ctl;
};

// Warp 0 loads, warp 1 issues the products, warp 2 owns tensor memory; warps 4-11 keep the
// sums: warp w holds lanes (w % 4) * 32 .. and columns ((w - 4) / 4) * 128 .., 128 sums a thread.
template <typename Tout>
__global__ void __launch_bounds__(kPThreads, 1)
prefill_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
               const LParams p) {
    extern __shared__ uint8_t dyn[];
    __shared__ PBars bars;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.tiles_t * p.tiles_n;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPStages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bars.done[i], 1), mbar_init(&bars.free[i], 8);
        mbar_init(&bars.drain, 1);
        bars.ctl.abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(&bars.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp == 0) {
        if (elect_one()) {
            int64_t it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                const int tt = tile / p.tiles_n, tn = tile - tt * p.tiles_n;
                for (int k = 0; k < p.kb; ++k, ++it) {
                    const int s = (int)(it % kPStages);
                    if (!wait_or_abort(&bars.empty[s], (uint32_t)((it / kPStages) & 1) ^ 1u, &bars.ctl)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = ring + s * kPStageBytes;
                    mbar_arrive_expect_tx(&bars.full[s], kPStageBytes);
                    tma_load_2d(st, &mx, k * kBK, tt * kBM, &bars.full[s]);
                    tma_load_2d(st + kBM * kBK, &mw, k * kBK, tn * kPN, &bars.full[s]);
                }
            }
            if (!ok)  // copies in flight (the last use of each stage), before the CTA may end
                for (int64_t j = it > kPStages ? it - kPStages : 0; j < it; ++j)
                    mbar_wait_bounded(&bars.full[j % kPStages], (uint32_t)((j / kPStages) & 1), kLimit / 8);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            constexpr uint32_t idesc = mma_desc(kBM, kPN);
            int64_t it = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
                for (int k = 0; k < p.kb; ++k, ++it) {
                    const int s = (int)(it % kPStages), d = (int)(it & 1);
                    if (!wait_or_abort(&bars.free[d], (uint32_t)((it >> 1) & 1) ^ 1u, &bars.ctl) ||
                        !wait_or_abort(&bars.full[s], (uint32_t)((it / kPStages) & 1), &bars.ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_addr(ring + s * kPStageBytes);
                    mma_stage(tmem + d * kPN, a, a + kBM * kBK, idesc);
                    tc_commit(&bars.empty[s]);
                    tc_commit(&bars.done[d]);
                }
            }
            if (!ok) {
                tc_commit(&bars.drain);
                mbar_wait_bounded(&bars.drain, 0, kLimit / 8);
            }
        }
    } else if (warp >= 4) {
        const int half = (warp - 4) >> 2, quad = warp & 3;
        const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + half * 128;
        int64_t it = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
            const int tt = tile / p.tiles_n, tn = tile - tt * p.tiles_n;
            const int64_t t = (int64_t)tt * kBM + quad * 32 + lane;
            const int64_t n0 = (int64_t)tn * kPN + half * 128;
            const bool in = t < p.tokens && n0 < p.n;
            const float* xs = p.xs + (in ? t : 0) * p.kb;
            const float* ws = p.ws + (in ? n0 / kGroup : 0) * p.kb;
            f2 acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = pack2(0.f, 0.f);
            float sc = __ldg(xs) * __ldg(ws);
            for (int k = 0; k < p.kb; ++k, ++it) {
                const int d = (int)(it & 1);
                const int kn = k + 1 < p.kb ? k + 1 : k;
                const float next = __ldg(xs + kn) * __ldg(ws + kn);
                ok = __all_sync(kFull, wait_or_abort(&bars.done[d], (uint32_t)((it >> 1) & 1), &bars.ctl));
                if (!ok) break;
                tc_fence_after();
                const f2 s2 = pack2(sc, sc);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    uint32_t r[16];
                    tmem_ld16(base + d * kPN + c * 16, r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        acc[c * 8 + j] = fma2(pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])),
                                              s2, acc[c * 8 + j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.free[d]);
                sc = next;
            }
            if (!ok) break;
            if (!in) continue;
            Tout* out = static_cast<Tout*>(p.out);
            if (p.seqlen == 0) {
                Tout* o = out + t * p.n + n0;
                if (n0 + 128 <= p.n && p.n % 8 == 0) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float v[kE];
#pragma unroll
                        for (int j = 0; j < 4; ++j) unpack2(acc[c * 4 + j], v[2 * j], v[2 * j + 1]);
                        store_all(o + c * kE, v);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        float v0, v1;
                        unpack2(acc[c], v0, v1);
                        if (n0 + 2 * c < p.n) o[2 * c] = io<Tout>::from_f(v0);
                        if (n0 + 2 * c + 1 < p.n) o[2 * c + 1] = io<Tout>::from_f(v1);
                    }
                }
            } else {
                Tout* o = out + out_index<Tout>(p, t, n0);
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    float v0, v1;
                    unpack2(acc[c], v0, v1);
                    if (n0 + 2 * c < p.n) o[2 * c * p.seqlen] = io<Tout>::from_f(v0);
                    if (n0 + 2 * c + 1 < p.n) o[(2 * c + 1) * p.seqlen] = io<Tout>::from_f(v1);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_free(tmem, 512);
}

// ---- Few tokens ------------------------------------------------------------------------

constexpr int kTThreads = 192;  // warps 0-3 keep the sums, warp 4 loads, warp 5 issues products

struct TBars {
    uint64_t full[6], empty[6];
    uint64_t done[2], free[2];
    uint64_t drain;
    uint32_t tmem;
    Ctl ctl;
};

template <int BN>
constexpr uint32_t token_stage_bytes() { return (kBM + BN) * kBK; }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float peer_load(const float* local, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Grid (pieces, output tiles, token tiles), a cluster of `pieces` CTAs along x.  Piece q takes
// input blocks [kb q / pieces, kb (q + 1) / pieces); the pieces' sums are added in order of
// piece, each CTA adding and storing its share of the tile's columns.
template <int BN, typename Tout>
__global__ void __launch_bounds__(kTThreads)
token_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw,
             const LParams p, int stages) {
    extern __shared__ uint8_t dyn[];
    __shared__ TBars bars;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~(uintptr_t)1023);
    constexpr uint32_t kStage = token_stage_bytes<BN>();
    constexpr uint32_t kCols = 2 * BN < 32 ? 32 : 2 * BN;
    float* red = reinterpret_cast<float*>(ring);                        // [BN][128], after the products
    float* scl = reinterpret_cast<float*>(ring + (size_t)stages * kStage);  // [blocks][BN] scales
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pieces = (int)gridDim.x, piece = (int)cluster_rank();
    const int k0 = (int)((int64_t)p.kb * piece / pieces), k1 = (int)((int64_t)p.kb * (piece + 1) / pieces);
    const int64_t n0 = (int64_t)blockIdx.y * kBM, t0 = (int64_t)blockIdx.z * BN;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&bars.done[i], 1), mbar_init(&bars.free[i], 4);
        mbar_init(&bars.drain, 1);
        bars.ctl.abort = 0;
        fence_barrier_init();
    }
    if (warp == 5) tmem_alloc(&bars.tmem, kCols);
    // token scales times the tile's weight scales, by block and column
    if (warp < 4)
        for (int i = threadIdx.x; i < (k1 - k0) * BN; i += 128) {
            const int c = i % BN, k = i / BN;
            const int64_t t = t0 + c;
            scl[i] = t < p.tokens ? __ldg(p.xs + t * p.kb + k0 + k) * __ldg(p.ws + (n0 / kGroup) * p.kb + k0 + k)
                                  : 0.f;
        }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem;
    bool ok = true;
    if (warp == 4) {
        if (elect_one()) {
            for (int k = k0; k < k1; ++k) {
                const int it = k - k0, s = it % stages;
                if (!wait_or_abort(&bars.empty[s], (uint32_t)((it / stages) & 1) ^ 1u, &bars.ctl)) {
                    for (int j = it > stages ? it - stages : 0; j < it; ++j)
                        mbar_wait_bounded(&bars.full[j % stages], (uint32_t)((j / stages) & 1), kLimit / 8);
                    break;
                }
                uint8_t* st = ring + (size_t)s * kStage;
                mbar_arrive_expect_tx(&bars.full[s], kStage);
                tma_load_2d(st, &mw, k * kBK, (int)n0, &bars.full[s]);
                tma_load_2d(st + kBM * kBK, &mx, k * kBK, (int)t0, &bars.full[s]);
            }
        }
    } else if (warp == 5) {
        if (elect_one()) {
            constexpr uint32_t idesc = mma_desc(kBM, BN);
            for (int k = k0; k < k1; ++k) {
                const int it = k - k0, s = it % stages, d = it & 1;
                if (!wait_or_abort(&bars.free[d], (uint32_t)((it >> 1) & 1) ^ 1u, &bars.ctl) ||
                    !wait_or_abort(&bars.full[s], (uint32_t)((it / stages) & 1), &bars.ctl)) {
                    tc_commit(&bars.drain);
                    mbar_wait_bounded(&bars.drain, 0, kLimit / 8);
                    break;
                }
                tc_fence_after();
                const uint32_t a = smem_addr(ring + (size_t)s * kStage);
                mma_stage(tmem + d * BN, a, a + kBM * kBK, idesc);
                tc_commit(&bars.empty[s]);
                tc_commit(&bars.done[d]);
            }
        }
    } else {
        const uint32_t base = tmem + ((uint32_t)(warp * 32) << 16);
        float acc[BN];
#pragma unroll
        for (int i = 0; i < BN; ++i) acc[i] = 0.f;
        for (int k = k0; k < k1; ++k) {
            const int it = k - k0, d = it & 1;
            ok = __all_sync(kFull, wait_or_abort(&bars.done[d], (uint32_t)((it >> 1) & 1), &bars.ctl));
            if (!ok) break;
            tc_fence_after();
            const float* sc = scl + it * BN;
#pragma unroll
            for (int c = 0; c < BN / 16; ++c) {
                uint32_t r[16];
                tmem_ld16(base + d * BN + c * 16, r);
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
            if (lane == 0) mbar_arrive(&bars.free[d]);
        }
        // All of this CTA's products are done (each was waited for), and with them its operand
        // tiles: the ring takes the sums.
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (!bars.ctl.abort) {
#pragma unroll
            for (int i = 0; i < BN; ++i) red[i * kBM + warp * 32 + lane] = acc[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_free(tmem, kCols);
    const bool bad = bars.ctl.abort != 0;
    __syncwarp();
    cluster_sync();
    if (!bad) {
        // this CTA's columns (tokens) of the tile
        const int c0 = BN * piece / pieces, c1 = BN * (piece + 1) / pieces;
        Tout* out = static_cast<Tout*>(p.out);
        for (int i = threadIdx.x; i < (c1 - c0) * kBM; i += kTThreads) {
            const int c = c0 + i / kBM, row = i % kBM;
            const int64_t t = t0 + c, n = n0 + row;
            if (t >= p.tokens || n >= p.n) continue;
            float v = 0.f;
            for (int q = 0; q < pieces; ++q) v += peer_load(red + c * kBM + row, (uint32_t)q);
            out[out_index<Tout>(p, t, n)] = io<Tout>::from_f(v);
        }
    }
    cluster_sync();  // a CTA's shared memory outlives its peers' reads
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

int multiprocessors() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1)
        return 148;
    return sms;
}

template <typename Tout>
cudaError_t run_prefill(const LinearArgs& a, LParams p, cudaStream_t s) {
    CUtensorMap mx, mw;
    if (!encode_rows(&mx, a.xq, a.k, a.tokens, kBM) || !encode_rows(&mw, a.wq, a.k, a.n, kPN))
        return cudaErrorInvalidValue;
    p.tiles_t = (int)((a.tokens + kBM - 1) / kBM);
    p.tiles_n = (int)((a.n + kPN - 1) / kPN);
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>((int64_t)p.tiles_t * p.tiles_n, multiprocessors());
    prefill_kernel<Tout><<<grid, kPThreads, kPSmem, s>>>(mx, mw, p);
    return cudaGetLastError();
}

template <int BN, typename Tout>
cudaError_t run_token(const LinearArgs& a, const LParams& p, cudaStream_t s) {
    CUtensorMap mx, mw;
    if (!encode_rows(&mx, a.xq, a.k, a.tokens, BN) || !encode_rows(&mw, a.wq, a.k, a.n, kBM))
        return cudaErrorInvalidValue;
    const int64_t tn = (a.n + kBM - 1) / kBM, tt = (a.tokens + BN - 1) / BN;
    // pieces: up to 8 (a portable cluster), while they fill the machine's CTA slots twice over and
    // leave every piece two blocks
    int pieces = 1;
    while (pieces < 8 && pieces * 2 <= BN && tn * tt * pieces < multiprocessors() * 2 && pieces * 4 <= p.kb)
        pieces *= 2;
    const int blocks = (p.kb + pieces - 1) / pieces;
    constexpr uint32_t kStage = token_stage_bytes<BN>();
    constexpr int kLeast = (BN * kBM * 4 + kStage - 1) / kStage;  // the ring also holds the tile's sums
    constexpr int64_t kMost = 226 * 1024;
    int stages = std::max(std::min(blocks, 6), kLeast);
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
    p.tiles_t = p.tiles_n = 0;
    const int64_t big = ((a.tokens + kBM - 1) / kBM) * ((a.n + kPN - 1) / kPN);
    if (big >= multiprocessors()) return run_prefill<Tout>(a, p, s);
    if (a.tokens <= 16) return run_token<16, Tout>(a, p, s);
    if (a.tokens <= 32) return run_token<32, Tout>(a, p, s);
    return run_token<64, Tout>(a, p, s);
}

}  // namespace

cudaError_t launch_fp8_linear(const LinearArgs& a, cudaStream_t s) {
    if (a.tokens == 0 || a.n == 0) return cudaSuccess;
    return a.out_dtype == DType::BF16 ? run_linear<__nv_bfloat16>(a, s) : run_linear<float>(a, s);
}

cudaError_t read_linear_error(unsigned* out, bool clear, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_linear_error, sizeof(unsigned), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && clear && *out) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbolAsync(g_linear_error, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace s6
