// gated_scan.cu -- the gated linear recurrence (forward, backward, one-token update) for
// sm_100a.
//
// Per row (a channel of a batch entry) with h_{-1} = h0:
//
//   sigmoid form   s_t = sigmoid(gate_t + bias), a_t = 1 - s_t, b_t = s_t x_t
//                  (the gated RNN that the selective SSM reduces to with N = 1, A = -1,
//                  B = 1: "Mamba: Linear-Time Sequence Modeling with Selective State
//                  Spaces", Selection mechanism)
//   given decay    a_t = gate_t, b_t = x_t
//   h_t = a_t h_{t-1} + b_t,   y_t = h_t silu(z_t)  (h_t without z)
//
// A step is the transformation (a, b); two in a row compose to (a2 a1, a2 b1 + b2), which is
// associative (page "yongjin360.com/news/29389", derivation steps 1-4), so a row can be cut
// anywhere.  A warp walks a row in chunks of 256 steps: each lane composes its 8 consecutive
// steps in registers, the warp scans the 32 compositions with shuffles, and each lane then
// runs its 8 steps again from the state entering it.  Every array is read once and written
// once; with no B, C and state axis the recurrence is bound by memory (6 to 8 bytes a step
// in bf16), so the layout is that of a stream: 16-byte accesses, the next chunks' loads in
// flight while this one is computed.
//
// Chunks start at multiples of 8 elements of the whole array, not of the row, so rows of any
// length take the same vector accesses; the lanes at a row's two ends mask the steps that
// belong to the neighbouring rows (their transformation is the identity) and store the rest
// element by element.
//
// Few rows leave most of the machine idle with a warp each, so then a row is walked by all warps
// of a CTA, or of a cluster of CTAs, side by side: each takes one of the next chunks, the
// chunks' compositions are scanned over the warps (shared memory) and over the CTAs
// (distributed shared memory), and every array is still read once.  (Cutting rows into segments
// that are first composed and then walked reads x and gate twice: 126 us against 73 for
// (1, 60, 524287) fp32.)
#include <algorithm>

#include "layer_launch.h"
#include "row8.cuh"

namespace s6 {
namespace {

static_assert(kE == kGatedLane, "a lane takes one vector");
constexpr int kWarps = 4;     // per CTA where a warp walks a row by itself
constexpr int kTeamWarps = 8;  // at most, per CTA where warps walk a row together
constexpr int kMaxTeam = 16;    // at most, CTAs of a cluster that walk a row together
constexpr unsigned kFull = 0xffffffffu;
__device__ unsigned int g_gated_error = 0;        // a bounded wait gave up
constexpr long long kLimit = 2000000000LL;  // SM clocks, about a second

// sigmoid of a pair, the arguments given as -v log2(e).
__device__ __forceinline__ f2 sigmoid2(f2 t) {
    float d0, d1;
    unpack2(add2(ex2x2(t), pack2(1.f, 1.f)), d0, d1);
    return pack2(rcp(d0), rcp(d1));
}
__device__ __forceinline__ f2 twice(float v) { return pack2(v, v); }

// A pair of gates: sg = sigmoid(v) and a = 1 - sg, the arguments given as t = -v log2(e).  With e = 2^t,
// sg = 1 / (1 + e), and a is formed from whichever keeps it exact: 1 - sg while sg is the smaller (one
// rounding of a number near one), e sg while a is (1 - sg would leave it the rounding of sg, and
// nothing beyond v = 17).
__device__ __forceinline__ f2 gate2(f2 t, float& a0, float& a1) {
    const f2 e = ex2x2(t);
    float d0, d1, k0, k1, o0, o1;
    unpack2(add2(e, pack2(1.f, 1.f)), d0, d1);
    const float s0 = rcp(d0), s1 = rcp(d1);
    const f2 sg = pack2(s0, s1);
    unpack2(sub2(twice(1.f), sg), k0, k1);
    unpack2(mul2(e, sg), o0, o1);
    a0 = s0 < 0.5f ? k0 : o0;
    a1 = s1 < 0.5f ? k1 : o1;
    return sg;
}

// The lane's 8 decays a_j and (sigmoid form) sigmoids sg_j, two at a time in packed arithmetic;
// nbias = -bias log2(e).
template <bool DECAY, typename T>
__device__ __forceinline__ void decays(const Raw8<T>& g, float nbias, float (&a)[kE], float (&sg)[kE]) {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
        if (DECAY) unpack2(g.pair(i), a[2 * i], a[2 * i + 1]);
        else unpack2(gate2(fma2(g.pair(i), twice(-kLog2e), twice(nbias)), a[2 * i], a[2 * i + 1]),
                     sg[2 * i], sg[2 * i + 1]);
    }
}
// Its inputs b_j.
template <bool DECAY, typename T>
__device__ __forceinline__ void inputs(const Raw8<T>& x, const float (&sg)[kE], float (&b)[kE]) {
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
        const f2 v = DECAY ? x.pair(i) : mul2(pack2(sg[2 * i], sg[2 * i + 1]), x.pair(i));
        unpack2(v, b[2 * i], b[2 * i + 1]);
    }
}
// Steps outside the row become the identity: a = 1, b = 0.
__device__ __forceinline__ void outside(int64_t e, const Row& w, float (&v)[kE], float value) {
#pragma unroll
    for (int j = 0; j < kE; ++j)
        if (e + j < w.lo || e + j >= w.hi) v[j] = value;
}

// Inclusive scan over the lanes of the compositions (P, H), earlier lanes first.  (The shuffle's
// own predicate says which lanes have a partner.)
__device__ __forceinline__ void scan_up(float& P, float& H) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        asm("{\n .reg .f32 q, r;\n .reg .pred p;\n"
            " shfl.sync.up.b32 q|p, %0, %2, 0, 0xffffffff;\n shfl.sync.up.b32 r|p, %1, %2, 0, 0xffffffff;\n"
            " @p fma.rn.f32 %1, %0, r, %1;\n @p mul.rn.f32 %0, %0, q;\n}\n"
            : "+f"(P), "+f"(H)
            : "r"(o));
}
// The same from the last lane down (the adjoint runs backwards in time).
__device__ __forceinline__ void scan_down(float& P, float& H) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        asm("{\n .reg .f32 q, r;\n .reg .pred p;\n"
            " shfl.sync.down.b32 q|p, %0, %2, 31, 0xffffffff;\n shfl.sync.down.b32 r|p, %1, %2, 31, 0xffffffff;\n"
            " @p fma.rn.f32 %1, %0, r, %1;\n @p mul.rn.f32 %0, %0, q;\n}\n"
            : "+f"(P), "+f"(H)
            : "r"(o));
}

// Whether chunk c of row w reaches past an end of the row.
__device__ __forceinline__ bool at_edge(const Row& w, int c, int chunks) {
    return (c == 0 && w.base != w.lo) || (c + 1 >= chunks && w.base + (int64_t)chunks * kGatedChunk != w.hi) ||
           c >= chunks;
}
// A lane's 8 elements from e on: directly, or with the checks of an edge chunk.
template <typename T>
__device__ __forceinline__ void get(Raw8<T>& r, const void* p, int64_t e, const Row& w, bool edge) {
    if (edge) fetch<T>(r, p, e, w);
    else r.load(static_cast<const T*>(p) + e);
}
template <typename T>
__device__ __forceinline__ void set(void* p, int64_t e, const Row& w, bool edge, const float (&v)[kE]) {
    if (edge) put<T>(p, e, w, v);
    else store_all(static_cast<T*>(p) + e, v);
}

// Whether a warp's coming chunks wait in shared memory (a Ring) or, the next one, in registers.
// The ring keeps more bytes in flight in fewer registers: a warp per row, (4, 5120, 4096) bf16 with
// z 113 -> 105 us forward on the device, 326 -> 293 with the backward, (1, 2300, 8192) 44 -> 31 (these
// and the next before gate2 kept both sigmoids whole, which added 2%).  Teams have
// their bytes in flight in many warps, and the way through shared memory lengthens their rounds
// ((1, 60, 524287): fp32 decays 68 -> 75 us, bf16 with z and the backward 197 -> 215), except
// where the registers do not hold a second chunk: fp32 with z (147 -> 91 forward, 352 -> 307 with
// the backward), and the fp32 forward with sigmoids (88 -> 76), the WIDE ones.
template <typename T, bool WIDE, bool TEAM>
constexpr bool in_ring() { return !TEAM || (sizeof(T) == 4 && WIDE); }

// The warp's next kAhead chunks of N arrays (and a value of each chunk) in shared memory, filled by
// asynchronous copies of 512 consecutive bytes.  Depths 2, 3, 4 for a warp per row: 108, 105, 105
// us; 2, 3 for a team: 91, 117.
template <typename T, int N, bool TEAM>
struct Ring {
    static constexpr int kAhead = TEAM ? 2 : 3;
    static constexpr int kPieces = sizeof(Raw8<T>) / 16;  // 16-byte pieces of a lane's 8 elements
    uint4 v[kAhead][N][kPieces * 32];
    float one[kAhead][32];
    // Where the chunk's piece u lies: lanes that read pieces kPieces apart meet no bank twice.
    __device__ __forceinline__ static int place(int u) { return kPieces == 1 ? u : u ^ (u >> 3 & 1); }
    // Whether lanes read what others copied.
    __device__ __forceinline__ static void sync() {
        if (kPieces > 1) __syncwarp();
    }
    // p's chunk whose 8 elements of this lane are at e: zeros for vectors behind the row, nothing
    // from behind the array.
    __device__ __forceinline__ void copy(int stage, int array, const void* p, int64_t e, const Row& w, bool edge) {
        constexpr int kPer = 16 / sizeof(T);
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int u = i * 32 + lane;
            int64_t at = e + (u - lane * kPieces) * kPer;
            int count = kPer;
            if (edge) {
                count = at < w.hi ? (int)min((int64_t)kPer, w.total - at) : 0;
                if (count == 0) at = 0;
            }
            cp_async16(&v[stage][array][place(u)], static_cast<const T*>(p) + at, count * (int)sizeof(T));
        }
    }
    __device__ __forceinline__ void copy_one(int stage, const float* p) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(&one[stage][threadIdx.x & 31])), "l"(p)
                     : "memory");
    }
    // The lane's 8 elements.
    __device__ __forceinline__ void read(int stage, int array, Raw8<T>& r) const {
        uint4* o = reinterpret_cast<uint4*>(&r);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) o[i] = v[stage][array][place((threadIdx.x & 31) * kPieces + i)];
    }
};

template <typename T, int N, bool WIDE, bool TEAM>
constexpr int ring_bytes() { return in_ring<T, WIDE, TEAM>() ? (int)sizeof(Ring<T, N, TEAM>) : 0; }

struct FParams {
    const void* x;
    const void* g;
    const void* z;
    const float* bias;
    const float* h0;
    void* y;
    float* last;
    float* ck;
    int64_t rows, dim, L, maxch;
};

// What the warps that walk a row together hand each other, twice (a round's is read while the
// next one's is written).
struct Team {
    float2 warp[2][kTeamWarps];    // the warps' compositions
    float2 before[2][kTeamWarps];  // of the warps before each in the CTA
    float enter[2];                // the value entering the CTA's chunks
    float2 cta[2][kMaxTeam];       // the CTAs' compositions
    uint64_t here[2];              // ... have arrived
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// (The aligned forms take whole warps, whatever branch some lanes come from.)
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// Sets up a cluster's hand-over; ends with every CTA's shared memory in place.
__device__ __forceinline__ void team_begin(Team& team) {
    if (threadIdx.x == 0) {
        mbar_init(&team.here[0], 1);
        mbar_init(&team.here[1], 1);
        fence_barrier_init();
    }
    __syncthreads();
    cluster_sync();
}
// Stores v into the CTA of `rank` and counts its bytes on that CTA's barrier: what waits there is
// ordered after this store alone (a cluster barrier would wait for the row's stores to global
// memory too).
__device__ __forceinline__ void hand_over(const float2* local, const uint64_t* bar, uint32_t rank, float2 v) {
    uint32_t a, m;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(smem_addr(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(a),
                 "f"(v.x), "f"(v.y), "r"(m)
                 : "memory");
}

// A round of a team: the warp's composition of its chunk, held by lane 31 (FORWARD) or lane 0;
// returns the value entering the chunk.  Warp 0 scans the CTA's compositions, hands its own to
// the cluster, scans the cluster's and moves the row's carry (its alone) past the round.
template <bool FORWARD>
__device__ __forceinline__ float team_round(Team& team, int round, int ctas, int rank, float P, float H, float& carry,
                                            bool& alive) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, buf = round & 1;
    if (lane == (FORWARD ? 31 : 0)) team.warp[buf][warp] = make_float2(P, H);
    __syncthreads();
    if (warp == 0) {
        P = 1.f, H = 0.f;
        if (lane < warps) {
            const float2 v = team.warp[buf][lane];
            P = v.x, H = v.y;
        }
        if (FORWARD) scan_up(P, H);
        else scan_down(P, H);
        const int last = FORWARD ? warps - 1 : 0;
        const float2 all = make_float2(__shfl_sync(kFull, P, last), __shfl_sync(kFull, H, last));
        const float Pb = FORWARD ? __shfl_up_sync(kFull, P, 1) : __shfl_down_sync(kFull, P, 1);
        const float Hb = FORWARD ? __shfl_up_sync(kFull, H, 1) : __shfl_down_sync(kFull, H, 1);
        const bool first = lane == (FORWARD ? 0 : warps - 1);
        if (lane < warps) team.before[buf][lane] = first ? make_float2(1.f, 0.f) : make_float2(Pb, Hb);
        if (ctas == 1) {
            if (lane == 0) team.enter[buf] = carry;
            carry = fmaf(all.x, carry, all.y);
        } else {
            // A CTA that gave up takes no further part: its barrier's phase may be incomplete, and a second
            // arrival in a phase of one is not allowed.  Its peers give up in their turn.
            if (alive) {
                if (lane == 0) mbar_arrive_expect_tx(&team.here[buf], (uint32_t)ctas * 8u);
                if (lane < ctas) hand_over(&team.cta[buf][rank], &team.here[buf], (uint32_t)lane, all);
                __syncwarp();
                if (!__all_sync(kFull, mbar_wait_bounded(&team.here[buf], (uint32_t)(round >> 1) & 1u, kLimit))) {
                    if (lane == 0) atomicOr(&g_gated_error, 1u);
                    alive = false;  // the outputs are void; the rounds end without further waits
                }
            }
            P = 1.f, H = 0.f;
            if (lane < ctas) {
                const float2 v = team.cta[buf][lane];
                P = v.x, H = v.y;
            }
            if (FORWARD) scan_up(P, H);
            else scan_down(P, H);
            const float after = fmaf(P, carry, H);  // this CTA's chunks and those before them
            const float in = __shfl_sync(kFull, after, (FORWARD ? rank - 1 : rank + 1) & 31);
            if (lane == 0) team.enter[buf] = (FORWARD ? rank > 0 : rank + 1 < ctas) ? in : carry;
            carry = __shfl_sync(kFull, after, FORWARD ? ctas - 1 : 0);
        }
    }
    __syncthreads();
    const float2 v = team.before[buf][warp];
    return fmaf(v.x, team.enter[buf], v.y);
}

// TEAM: the row's chunks go round the warps of the CTA (and of its cluster); otherwise a warp
// walks its row alone.  p.y may be null: states (checkpoints, last state) only.
template <typename Tin, typename Tout, bool DECAY, bool GATED, bool TEAM>
__global__ void __launch_bounds__(TEAM ? 32 * kTeamWarps : 32 * kWarps, TEAM ? 4 : 8) gated_fwd_kernel(const FParams p) {
    extern __shared__ uint4 rings[];
    __shared__ Team team;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr bool RING = in_ring<Tin, GATED || !DECAY, TEAM>();
    using Chunks = Ring<Tin, GATED ? 3 : 2, TEAM>;
    constexpr int kAhead = Chunks::kAhead;
    Chunks& ring = reinterpret_cast<Chunks*>(rings)[warp];
    const int ctas = TEAM ? (int)cluster_ctas() : 1, rank = TEAM ? (int)cluster_rank() : 0;
    const int64_t r = TEAM ? blockIdx.x / ctas : (int64_t)blockIdx.x * kWarps + warp;
    if (!TEAM && r >= p.rows) return;
    if (TEAM && ctas > 1) team_begin(team);
    const Row w = row_of(r, p.rows, p.L);
    const int chunks = (int)((w.vectors + 31) / 32);
    const int step = TEAM ? ctas * (int)(blockDim.x >> 5) : 1;  // chunks of a round
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float h = p.h0 ? __ldg(p.h0 + r) : 0.f;  // the state entering the round
    int c = TEAM ? rank * (int)(blockDim.x >> 5) + warp : 0;
    int64_t e = w.base + (int64_t)c * kGatedChunk + lane * kE;
    const auto start = [&](int k, int64_t e0, int stage) {  // the copies of chunk k
        if (k < chunks) {
            const bool edge = at_edge(w, k, chunks);
            ring.copy(stage, 0, p.x, e0, w, edge);
            ring.copy(stage, 1, p.g, e0, w, edge);
            if (GATED) ring.copy(stage, 2, p.z, e0, w, edge);
        }
        cp_async_commit();
    };
    Raw8<Tin> xr, gr, zr, xn, gn, zn;
    bool alive = true, edge, edge_n = at_edge(w, c, chunks);
    if (RING) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) start(c + k * step, e + (int64_t)k * step * kGatedChunk, k);
    } else {
        get<Tin>(xn, p.x, e, w, edge_n);
        get<Tin>(gn, p.g, e, w, edge_n);
        if (GATED) get<Tin>(zn, p.z, e, w, edge_n);
    }
    // every warp of a team makes every round (its chunk may lie past the row: the identity)
    for (int c0 = 0, round = 0, stage = 0; c0 < chunks;
         c0 += step, c += step, e += (int64_t)step * kGatedChunk, ++round) {
        if (RING) {
            cp_async_wait<kAhead - 1>();
            ring.sync();
            ring.read(stage, 0, xr);
            ring.read(stage, 1, gr);
            edge = at_edge(w, c, chunks);
        } else {
            xr = xn, gr = gn, edge = edge_n;
            if (GATED) zr = zn;
            if (c0 + step < chunks) {
                const int64_t en = e + (int64_t)step * kGatedChunk;
                edge_n = at_edge(w, c + step, chunks);
                get<Tin>(xn, p.x, en, w, edge_n);
                get<Tin>(gn, p.g, en, w, edge_n);
                if (GATED) get<Tin>(zn, p.z, en, w, edge_n);
            }
        }
        float a[kE], b[kE];
        decays<DECAY>(gr, nbias, a, b);
        inputs<DECAY>(xr, b, b);
        if (edge) outside(e, w, a, 1.f), outside(e, w, b, 0.f);
        float P = a[0], H = b[0];
#pragma unroll
        for (int j = 1; j < kE; ++j) {
            H = fmaf(a[j], H, b[j]);
            P *= a[j];
        }
        scan_up(P, H);
        float in = h;  // the state entering the warp's chunk
        if (TEAM) in = team_round<true>(team, round, ctas, rank, P, H, h, alive);
        const float after = fmaf(P, in, H);  // ... and leaving the lane's steps
        float hv = __shfl_up_sync(kFull, after, 1);
        if (lane == 0) hv = in;
        if (!TEAM) h = __shfl_sync(kFull, after, 31);
        if (TEAM && c >= chunks) break;  // the last round
        if (p.ck && lane == 0) p.ck[r * p.maxch + c] = in;
        if (p.y) {
            float out[kE];
#pragma unroll
            for (int j = 0; j < kE; ++j) out[j] = hv = fmaf(a[j], hv, b[j]);
            if (GATED) {
                if (RING) ring.read(stage, 2, zr);
#pragma unroll
                for (int i = 0; i < kE / 2; ++i) {
                    const f2 z = zr.pair(i);
                    const f2 zs = mul2(z, sigmoid2(mul2(z, twice(-kLog2e))));
                    unpack2(mul2(pack2(out[2 * i], out[2 * i + 1]), zs), out[2 * i], out[2 * i + 1]);
                }
            }
            set<Tout>(p.y, e, w, edge, out);
        }
        if (RING) {
            ring.sync();  // the stage has been read
            start(c + kAhead * step, e + (int64_t)kAhead * step * kGatedChunk, stage);
            stage = stage + 1 == kAhead ? 0 : stage + 1;
        }
    }
    if (p.last && lane == 0 && (!TEAM || (warp == 0 && rank == 0))) p.last[r] = h;
    if (TEAM && ctas > 1) cluster_sync();  // what the peers hand over has a place until the end
}

struct RParams {
    FParams f;
    const void* dy;
    const float* dlast;
    void* dx;
    void* dg;
    void* dz;
    float* dh0;
    float* bias_part;  // (rows, CTAs of a team)
};

// The backward: with e_t the adjoint handed to h_t from later steps,
//   dh_t = dy_t silu(z_t) + e_t,  e_{t-1} = a_t dh_t,
// the recurrence again, backwards, with the same a.  A chunk's states are formed again from its
// checkpoint, so rounds go from the row's end to its beginning and read every array once.
template <typename T, bool DECAY, bool GATED, bool TEAM>
__global__ void __launch_bounds__(TEAM ? 32 * kTeamWarps : 32 * kWarps, TEAM ? 1 : 6) gated_bwd_kernel(const RParams q) {
    extern __shared__ uint4 rings[];
    __shared__ Team team;
    __shared__ float sums[kTeamWarps];
    const FParams& p = q.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr bool RING = in_ring<T, GATED, TEAM>();
    using Chunks = Ring<T, GATED ? 4 : 3, TEAM>;
    constexpr int kAhead = Chunks::kAhead;
    Chunks& ring = reinterpret_cast<Chunks*>(rings)[warp];
    const int ctas = TEAM ? (int)cluster_ctas() : 1, rank = TEAM ? (int)cluster_rank() : 0;
    const int64_t r = TEAM ? blockIdx.x / ctas : (int64_t)blockIdx.x * kWarps + warp;
    if (!TEAM && r >= p.rows) return;
    if (TEAM && ctas > 1) team_begin(team);
    const Row w = row_of(r, p.rows, p.L);
    const int chunks = (int)((w.vectors + 31) / 32);
    const int step = TEAM ? ctas * (int)(blockDim.x >> 5) : 1;
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float ec = q.dlast ? __ldg(q.dlast + r) : 0.f, bsum = 0.f;
    int c0 = (chunks - 1) / step * step;
    int c = c0 + (TEAM ? rank * (int)(blockDim.x >> 5) + warp : 0);
    const float* ck = p.ck + r * p.maxch;
    int64_t e = w.base + (int64_t)c * kGatedChunk + lane * kE;
    const auto start = [&](int k, int64_t e0, int stage) {  // the copies of chunk k
        if (k >= 0 && k < chunks) {
            const bool edge = at_edge(w, k, chunks);
            ring.copy(stage, 0, p.x, e0, w, edge);
            ring.copy(stage, 1, p.g, e0, w, edge);
            ring.copy(stage, 2, q.dy, e0, w, edge);
            if (GATED) ring.copy(stage, 3, p.z, e0, w, edge);
            ring.copy_one(stage, ck + k);
        }
        cp_async_commit();
    };
    Raw8<T> xr, gr, yr, zr, xn, gn, yn, zn;
    bool alive = true, edge, edge_n = at_edge(w, c, chunks);
    float kn = 0.f;
    if (RING) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) start(c - k * step, e - (int64_t)k * step * kGatedChunk, k);
    } else {
        if (c < chunks) kn = __ldg(ck + c);
        get<T>(xn, p.x, e, w, edge_n);
        get<T>(gn, p.g, e, w, edge_n);
        get<T>(yn, q.dy, e, w, edge_n);
        if (GATED) get<T>(zn, p.z, e, w, edge_n);
    }
    for (int round = 0, stage = 0; c0 >= 0; c0 -= step, c -= step, e -= (int64_t)step * kGatedChunk, ++round) {
        float entering = kn;  // the state entering the chunk
        if (RING) {
            cp_async_wait<kAhead - 1>();
            ring.sync();
            ring.read(stage, 0, xr);
            ring.read(stage, 1, gr);
            ring.read(stage, 2, yr);
            if (GATED) ring.read(stage, 3, zr);
            entering = ring.one[stage][lane];
            edge = at_edge(w, c, chunks);
            ring.sync();  // the stage has been read
            start(c - kAhead * step, e - (int64_t)kAhead * step * kGatedChunk, stage);
            stage = stage + 1 == kAhead ? 0 : stage + 1;
        } else {
            xr = xn, gr = gn, yr = yn, edge = edge_n;
            if (GATED) zr = zn;
            if (c0 > 0) {
                const int64_t en = e - (int64_t)step * kGatedChunk;
                edge_n = at_edge(w, c - step, chunks);
                kn = __ldg(ck + c - step);
                get<T>(xn, p.x, en, w, edge_n);
                get<T>(gn, p.g, en, w, edge_n);
                get<T>(yn, q.dy, en, w, edge_n);
                if (GATED) get<T>(zn, p.z, en, w, edge_n);
            }
        }
        float a[kE], sg[kE], gy[kE], dz[kE];
        decays<DECAY>(gr, nbias, a, sg);
        if (edge) outside(e, w, a, 1.f);
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            f2 g = yr.pair(i);
            if (GATED) {  // dz: dy times the derivative of silu(z), to be multiplied by the state
                const f2 z = zr.pair(i), s = sigmoid2(mul2(z, twice(-kLog2e)));
                const f2 ds = mul2(s, fma2(z, sub2(twice(1.f), s), twice(1.f)));
                unpack2(mul2(g, ds), dz[2 * i], dz[2 * i + 1]);
                g = mul2(g, mul2(z, s));
            }
            unpack2(g, gy[2 * i], gy[2 * i + 1]);
        }
        if (edge) outside(e, w, gy, 0.f);
        float P = 1.f, E = 0.f;
#pragma unroll
        for (int j = kE - 1; j >= 0; --j) {
            E = a[j] * (gy[j] + E);
            P *= a[j];
        }
        float Pd = P;
        scan_down(Pd, E);
        float in = ec;  // the adjoint entering the chunk from its right
        if (TEAM) in = team_round<false>(team, round, ctas, rank, Pd, E, ec, alive);
        const float after = fmaf(Pd, in, E);
        float ev = __shfl_down_sync(kFull, after, 1);
        if (lane == 31) ev = in;
        if (!TEAM) ec = __shfl_sync(kFull, after, 0);
        if (TEAM && c >= chunks) continue;
        // the inputs, formed here so that the sigmoids alone wait for the gradients, and the states before
        // each step
        float b[kE], hv[kE];
        inputs<DECAY>(xr, sg, b);
        if (edge) outside(e, w, b, 0.f);
        {
            float H = b[0];
#pragma unroll
            for (int j = 1; j < kE; ++j) H = fmaf(a[j], H, b[j]);
            scan_up(P, H);
            hv[0] = __shfl_up_sync(kFull, fmaf(P, entering, H), 1);
            if (lane == 0) hv[0] = entering;
#pragma unroll
            for (int j = 1; j < kE; ++j) hv[j] = fmaf(a[j - 1], hv[j - 1], b[j - 1]);
        }
        if (GATED) {
#pragma unroll
            for (int j = 0; j < kE; ++j) dz[j] *= fmaf(a[j], hv[j], b[j]);
            set<T>(q.dz, e, w, edge, dz);
        }
        float dh[kE];
#pragma unroll
        for (int j = kE - 1; j >= 0; --j) {
            dh[j] = gy[j] + ev;
            ev = a[j] * dh[j];
        }
        float dg[kE];
#pragma unroll
        for (int i = 0; i < kE / 2; ++i) {
            const f2 d = pack2(dh[2 * i], dh[2 * i + 1]), hp = pack2(hv[2 * i], hv[2 * i + 1]);
            if (DECAY) {
                unpack2(mul2(d, hp), dg[2 * i], dg[2 * i + 1]);
            } else {
                const f2 av = pack2(a[2 * i], a[2 * i + 1]);
                const f2 dx = mul2(pack2(sg[2 * i], sg[2 * i + 1]), d);
                unpack2(dx, dh[2 * i], dh[2 * i + 1]);
                unpack2(mul2(mul2(dx, sub2(xr.pair(i), hp)), av), dg[2 * i], dg[2 * i + 1]);
            }
        }
        set<T>(q.dx, e, w, edge, dh);
        set<T>(q.dg, e, w, edge, dg);
        if (!DECAY) {
            if (edge) outside(e, w, dg, 0.f);
            bsum += ((dg[0] + dg[1]) + (dg[2] + dg[3])) + ((dg[4] + dg[5]) + (dg[6] + dg[7]));
        }
    }
    if (q.dh0 && lane == 0 && (!TEAM || (warp == 0 && rank == 0))) q.dh0[r] = ec;
    if (q.bias_part) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bsum += __shfl_xor_sync(kFull, bsum, o);
        if (TEAM) {
            if (lane == 0) sums[warp] = bsum;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int i = 1; i < (int)(blockDim.x >> 5); ++i) bsum += sums[i];
                q.bias_part[r * ctas + rank] = bsum;
            }
        } else if (lane == 0) {
            q.bias_part[r] = bsum;
        }
    }
    if (TEAM && ctas > 1) cluster_sync();  // what the peers hand over has a place until the end
}

// dbias[d]: the partial sums of channel d's rows, in a fixed order (a warp per channel).
__global__ void gated_bias_kernel(const float* part, float* dbias, int64_t batch, int64_t dim,
                                  int64_t parts) {
    const int lane = threadIdx.x & 31;
    const int64_t d = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    cudaGridDependencySynchronize();  // launched early: wait for the rows' sums
    if (d >= dim) return;
    float v = 0.f;
    for (int64_t i = lane; i < batch * parts; i += 32)
        v += part[((i / parts) * dim + d) * parts + i % parts];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (lane == 0) dbias[d] = v;
}

// One token: h = a h + b in place, a stream over (batch, dim), four elements per thread.  The
// bias is read as a vector where rows are whole vectors, else element by element, and the last
// thread takes the elements behind the last whole vector: (256, 5121) bf16 with z 6.8 -> 4.4 us
// against one element per thread.
constexpr int kUpdate = 4;
template <typename T, bool DECAY, bool GATED>
__global__ void __launch_bounds__(128) gated_update_kernel(float* state, const T* x, const T* gate,
                                                           const float* bias, const T* z, T* y,
                                                           int64_t n, int64_t dim) {
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * kUpdate;
    if (i >= n) return;
    struct alignas(kUpdate * sizeof(T)) TV { T v[kUpdate]; };
    const int count = (int)min((int64_t)kUpdate, n - i);
    TV xv, gv, zv, yv;
    float4 h4 = make_float4(0.f, 0.f, 0.f, 0.f), b4 = h4;
    float *h = &h4.x, *b = &b4.x;
    if (count == kUpdate) {
        xv = *reinterpret_cast<const TV*>(x + i), gv = *reinterpret_cast<const TV*>(gate + i);
        if (GATED) zv = *reinterpret_cast<const TV*>(z + i);
        h4 = *reinterpret_cast<const float4*>(state + i);
    } else {
#pragma unroll
        for (int j = 0; j < kUpdate; ++j) {
            const int64_t k = i + min(j, count - 1);
            xv.v[j] = x[k], gv.v[j] = gate[k], h[j] = state[k];
            if (GATED) zv.v[j] = z[k];
        }
    }
    if (!DECAY && bias != nullptr) {
        int64_t d = i % dim;
        if (dim % kUpdate == 0) {
            b4 = *reinterpret_cast<const float4*>(bias + d);
        } else {
#pragma unroll
            for (int j = 0; j < kUpdate; ++j) {
                b[j] = __ldg(bias + d);
                if (++d == dim) d = 0;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kUpdate; ++j) {
        const float xf = io<T>::to_f(xv.v[j]), gf = io<T>::to_f(gv.v[j]);
        if (DECAY) {
            h[j] = fmaf(gf, h[j], xf);
        } else {
            const float e = ex2(fmaf(gf, -kLog2e, -kLog2e * b[j])), s = rcp(1.f + e);
            h[j] = fmaf(s < 0.5f ? 1.f - s : e * s, h[j], s * xf);  // as gate2
        }
        yv.v[j] = io<T>::from_f(GATED ? h[j] * silu(io<T>::to_f(zv.v[j])) : h[j]);
    }
    if (count == kUpdate) {
        *reinterpret_cast<float4*>(state + i) = h4;
        *reinterpret_cast<TV*>(y + i) = yv;
    } else {
#pragma unroll
        for (int j = 0; j < kUpdate; ++j)
            if (j < count) state[i + j] = h[j], y[i + j] = yv.v[j];
    }
}

FParams fparams(const GatedArgs& a) {
    FParams p;
    p.x = a.x;
    p.g = a.gate;
    p.z = a.z;
    p.bias = a.given_decay ? nullptr : a.gate_bias;
    p.h0 = a.h0;
    p.y = a.y;
    p.last = a.last_state;
    p.ck = a.ckpt;
    p.rows = a.rows;
    p.dim = a.dim;
    p.L = a.L;
    p.maxch = gated_chunks(a.L);
    return p;
}

constexpr int kPlainShared = 46 * 1024;  // a launch's dynamic shared memory without further permission

// Launches `alone` with a warp per row, or `team` with the plan's warps and CTAs per row, and so many
// bytes of shared memory for each warp's ring.
template <int ALONE_RING, int TEAM_RING, typename Params>
cudaError_t launch_rows(void (*alone)(Params), void (*team)(Params), const Params& p, int64_t rows,
                        const GatedTeam& t, cudaStream_t s) {
    cudaError_t e;
    if (t.warps * t.ctas == 1) {
        constexpr int kBytes = kWarps * ALONE_RING;
        if (kBytes > kPlainShared) {
            e = cudaFuncSetAttribute(alone, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
            if (e != cudaSuccess) return e;
        }
        alone<<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, kBytes, s>>>(p);
        return cudaGetLastError();
    }
    if (kTeamWarps * TEAM_RING > kPlainShared) {
        e = cudaFuncSetAttribute(team, cudaFuncAttributeMaxDynamicSharedMemorySize, kTeamWarps * TEAM_RING);
        if (e != cudaSuccess) return e;
    }
    if (t.ctas > 8) {  // more than every device allows, but within this one's limit of 16
        e = cudaFuncSetAttribute(team, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * t.ctas));
    cfg.blockDim = dim3((unsigned)(32 * t.warps));
    cfg.dynamicSmemBytes = (size_t)(t.warps * TEAM_RING);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)t.ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, team, p);
}

template <typename Tin, typename Tout, bool DECAY, bool GATED>
cudaError_t run_fwd(const FParams& p, cudaStream_t s) {
    constexpr int N = GATED ? 3 : 2;
    constexpr bool WIDE = GATED || !DECAY;
    return launch_rows<ring_bytes<Tin, N, WIDE, false>(), ring_bytes<Tin, N, WIDE, true>()>(
        gated_fwd_kernel<Tin, Tout, DECAY, GATED, false>, gated_fwd_kernel<Tin, Tout, DECAY, GATED, true>, p,
        p.rows, gated_team(p.rows, p.L, false), s);
}
template <typename Tin, typename Tout>
cudaError_t run_fwd_t(const FParams& p, bool decay, cudaStream_t s) {
    const bool gated = p.z != nullptr && p.y != nullptr;
    if (decay) return gated ? run_fwd<Tin, Tout, true, true>(p, s) : run_fwd<Tin, Tout, true, false>(p, s);
    return gated ? run_fwd<Tin, Tout, false, true>(p, s) : run_fwd<Tin, Tout, false, false>(p, s);
}

template <typename T, bool DECAY, bool GATED>
cudaError_t run_bwd(const RParams& q, cudaStream_t s) {
    constexpr int N = GATED ? 4 : 3;
    return launch_rows<ring_bytes<T, N, GATED, false>(), ring_bytes<T, N, GATED, true>()>(
        gated_bwd_kernel<T, DECAY, GATED, false>, gated_bwd_kernel<T, DECAY, GATED, true>, q, q.f.rows,
        gated_team(q.f.rows, q.f.L, true), s);
}
template <typename T>
cudaError_t run_bwd_t(const RParams& q, bool decay, cudaStream_t s) {
    const bool gated = q.f.z != nullptr;
    if (decay) return gated ? run_bwd<T, true, true>(q, s) : run_bwd<T, true, false>(q, s);
    return gated ? run_bwd<T, false, true>(q, s) : run_bwd<T, false, false>(q, s);
}

template <typename T>
cudaError_t run_update(const GatedUpdateArgs& a, cudaStream_t s) {
    const int64_t n = a.batch * a.dim;
    const unsigned blocks = (unsigned)((n + 128 * kUpdate - 1) / (128 * kUpdate));
    const T *x = static_cast<const T*>(a.x), *g = static_cast<const T*>(a.gate), *z = static_cast<const T*>(a.z);
    T* y = static_cast<T*>(a.y);
    const auto kernel = a.given_decay ? (z ? gated_update_kernel<T, true, true> : gated_update_kernel<T, true, false>)
                                      : (z ? gated_update_kernel<T, false, true> : gated_update_kernel<T, false, false>);
    kernel<<<blocks, 128, 0, s>>>(a.state, x, g, a.gate_bias, z, y, n, a.dim);
    return cudaGetLastError();
}

// One bounded wait on a barrier that nothing completes, as mamba_diag_wait_timeout_in describes.
__global__ void timeout_probe_kernel(long long limit_cycles) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
        if (!mbar_wait_bounded(&bar, 0, limit_cycles)) atomicOr(&g_gated_error, 1u);
    }
}

}  // namespace

// Warps that walk a row: one where there are more than 8 rows an SM (1300 rows of 8192 fp32: 31 us
// against 37 with a team; 1184: 28 against 30 in fp32, 22 against 19 in bf16); else as many as give
// an SM `per_sm` warps (32 forward, 16 for the backward's larger register need), in one CTA, or in
// a cluster of up to kMaxTeam where there are fewer rows than CTA places; never more than the row
// has chunks.
GatedTeam gated_team(int64_t rows, int64_t L, bool backward) {
    constexpr int64_t kSms = 148;
    const int64_t per_sm = backward ? 16 : 32, chunks = std::max<int64_t>(1, gated_chunks(L));
    const int64_t ctas_per_sm = (rows + kSms - 1) / kSms;
    GatedTeam t{1, 1};
    const int64_t warps = std::min<int64_t>({kTeamWarps, per_sm / ctas_per_sm, chunks});
    if (ctas_per_sm > 8 || warps <= 1) return t;
    t.warps = (int)warps;
    if (warps == kTeamWarps)
        t.ctas = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxTeam, kSms * per_sm / kTeamWarps / rows,
                                                              (chunks + kTeamWarps - 1) / kTeamWarps}));
    return t;
}

cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t s) {
    if (a.L == 0) {
        if (!a.last_state) return cudaSuccess;
        if (!a.h0) return cudaMemsetAsync(a.last_state, 0, (size_t)a.rows * 4, s);
        return cudaMemcpyAsync(a.last_state, a.h0, (size_t)a.rows * 4, cudaMemcpyDeviceToDevice, s);
    }
    const FParams p = fparams(a);
    if (a.in_dtype == DType::BF16)
        return a.out_dtype == DType::BF16
                   ? run_fwd_t<__nv_bfloat16, __nv_bfloat16>(p, a.given_decay != 0, s)
                   : run_fwd_t<__nv_bfloat16, float>(p, a.given_decay != 0, s);
    return a.out_dtype == DType::BF16 ? run_fwd_t<float, __nv_bfloat16>(p, a.given_decay != 0, s)
                                      : run_fwd_t<float, float>(p, a.given_decay != 0, s);
}

cudaError_t launch_gated_scan_bwd(const GatedArgs& a, const GatedBwdArgs& g, cudaStream_t s) {
    if (a.L == 0) {
        cudaError_t e = cudaSuccess;
        if (g.dh0)
            e = g.dlast ? cudaMemcpyAsync(g.dh0, g.dlast, (size_t)a.rows * 4,
                                          cudaMemcpyDeviceToDevice, s)
                        : cudaMemsetAsync(g.dh0, 0, (size_t)a.rows * 4, s);
        if (e == cudaSuccess && g.dbias) e = cudaMemsetAsync(g.dbias, 0, (size_t)a.dim * 4, s);
        return e;
    }
    RParams q;
    q.f = fparams(a);
    q.dy = g.dy;
    q.dlast = g.dlast;
    q.dx = g.dx;
    q.dg = g.dgate;
    q.dz = g.dz;
    q.dh0 = g.dh0;
    const int64_t batch = a.rows / a.dim, parts = gated_team(a.rows, a.L, true).ctas;
    const bool whole = batch * parts == 1;  // a row's sum is the channel's
    q.bias_part = !g.dbias ? nullptr : whole ? g.dbias : g.bias_part;
    const cudaError_t e = a.in_dtype == DType::BF16 ? run_bwd_t<__nv_bfloat16>(q, a.given_decay != 0, s)
                                                    : run_bwd_t<float>(q, a.given_decay != 0, s);
    if (e != cudaSuccess || !g.dbias || whole) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.dim + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gated_bias_kernel, (const float*)g.bias_part, g.dbias, batch, a.dim, parts);
}

cudaError_t launch_gated_update(const GatedUpdateArgs& a, cudaStream_t s) {
    return a.dtype == DType::BF16 ? run_update<__nv_bfloat16>(a, s) : run_update<float>(a, s);
}

cudaError_t launch_gated_timeout_probe(long long limit_cycles, cudaStream_t s) {
    timeout_probe_kernel<<<1, 32, 0, s>>>(limit_cycles);
    return cudaGetLastError();
}

cudaError_t gated_error_word(unsigned** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_gated_error);
}

}  // namespace s6
