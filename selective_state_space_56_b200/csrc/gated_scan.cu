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
// in bf16), so the layout is that of a stream: 16-byte accesses, the next chunk's loads in
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
// that are first composed and then walked reads x and gate twice: 126 us against FIXME us for
// (1, 60, 524287) fp32.)
#include <algorithm>

#include "layer_launch.h"
#include "row8.cuh"

namespace s6 {
namespace {

static_assert(kE == kGatedLane, "a lane takes one vector");
constexpr int kWarps = 4;     // per CTA where a warp walks a row by itself
constexpr int kTeamWarps = 16;  // at most, per CTA where warps walk a row together
constexpr int kMaxTeam = 8;     // CTAs of a cluster that walk a row together
constexpr unsigned kFull = 0xffffffffu;

// sigmoid(v) with the argument given as -v log2(e).
__device__ __forceinline__ float sigmoid_of(float t) { return rcp(1.f + ex2(t)); }

// The lane's 8 steps (a_j, b_j); steps outside the row become the identity.
template <bool DECAY>
__device__ __forceinline__ void steps(const float (&x)[kE], const float (&g)[kE], float nbias,
                                      int64_t e, const Row& w, float (&a)[kE], float (&b)[kE]) {
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        if (DECAY) {
            a[j] = g[j];
            b[j] = x[j];
        } else {
            const float s = sigmoid_of(fmaf(g[j], -kLog2e, nbias));
            a[j] = 1.f - s;
            b[j] = s * x[j];
        }
    }
    if (e < w.lo || e + kE > w.hi) {
#pragma unroll
        for (int j = 0; j < kE; ++j)
            if (e + j < w.lo || e + j >= w.hi) a[j] = 1.f, b[j] = 0.f;
    }
}

// Inclusive scan over the lanes of the compositions (P, H), earlier lanes first.
__device__ __forceinline__ void scan_up(float& P, float& H, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float Pp = __shfl_up_sync(kFull, P, o), Hp = __shfl_up_sync(kFull, H, o);
        if (lane >= o) {
            H = fmaf(P, Hp, H);
            P *= Pp;
        }
    }
}
// The same from the last lane down (the adjoint runs backwards in time).
__device__ __forceinline__ void scan_down(float& P, float& E, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float Pp = __shfl_down_sync(kFull, P, o), Ep = __shfl_down_sync(kFull, E, o);
        if (lane + o < 32) {
            E = fmaf(P, Ep, E);
            P *= Pp;
        }
    }
}

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
    float2 warp[2][kTeamWarps];
    float2 cta[2][kMaxTeam];
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
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void peer_store(const float2* local, uint32_t rank, float2 v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}

// One level of a team's scan: item `me` of n compositions, in order (FORWARD) or from the last
// one back.  Passes `carry` through the items before `me` into `in`, and through all into carry.
template <bool FORWARD>
__device__ __forceinline__ void through(const float2* items, int n, int me, int lane, float carry_in, float& in,
                                        float& out) {
    float P = 1.f, H = 0.f;
    if (lane < n) {
        const float2 v = items[lane];
        P = v.x, H = v.y;
    }
    if (FORWARD) scan_up(P, H, lane);
    else scan_down(P, H, lane);
    const int before = FORWARD ? me - 1 : me + 1, last = FORWARD ? n - 1 : 0;
    const float Pb = __shfl_sync(kFull, P, before & 31), Hb = __shfl_sync(kFull, H, before & 31);
    const float Pa = __shfl_sync(kFull, P, last), Ha = __shfl_sync(kFull, H, last);
    in = (FORWARD ? me > 0 : me + 1 < n) ? fmaf(Pb, carry_in, Hb) : carry_in;
    out = fmaf(Pa, carry_in, Ha);
}

// A round of a team: this warp's composition (P, H) of its chunk; returns the value entering the
// chunk and moves the row's carry past the round's chunks.
template <bool FORWARD>
__device__ __forceinline__ float team_round(Team& team, int buf, int ctas, int rank, float P, float H, float& carry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0) team.warp[buf][warp] = make_float2(P, H);
    __syncthreads();
    float in, out;
    if (ctas == 1) {
        through<FORWARD>(team.warp[buf], warps, warp, lane, carry, in, out);
        carry = out;
        return in;
    }
    // the CTA's own composition, for its peers; then the carry entering this CTA's chunks
    if (warp == 0) {
        float Pw = 1.f, Hw = 0.f;
        if (lane < warps) {
            const float2 v = team.warp[buf][lane];
            Pw = v.x, Hw = v.y;
        }
        if (FORWARD) scan_up(Pw, Hw, lane);
        else scan_down(Pw, Hw, lane);
        const int last = FORWARD ? warps - 1 : 0;
        const float2 all = make_float2(__shfl_sync(kFull, Pw, last), __shfl_sync(kFull, Hw, last));
        if (lane < ctas) peer_store(&team.cta[buf][rank], (uint32_t)lane, all);
    }
    __syncwarp();
    cluster_sync();
    float cta_in;
    through<FORWARD>(team.cta[buf], ctas, rank, lane, carry, cta_in, out);
    carry = out;
    through<FORWARD>(team.warp[buf], warps, warp, lane, cta_in, in, out);
    return in;
}

// TEAM: the row's chunks go round the warps of the CTA (and of its cluster); otherwise a warp
// walks its row alone.  p.y may be null: states (checkpoints, last state) only.
template <typename Tin, typename Tout, bool DECAY, bool GATED, bool TEAM>
__global__ void __launch_bounds__(TEAM ? 32 * kTeamWarps : 32 * kWarps, TEAM ? 2 : 1) gated_fwd_kernel(const FParams p) {
    __shared__ Team team;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = TEAM ? (int)cluster_ctas() : 1, rank = TEAM ? (int)cluster_rank() : 0;
    const int64_t r = TEAM ? blockIdx.x / ctas : (int64_t)blockIdx.x * kWarps + warp;
    if (!TEAM && r >= p.rows) return;
    if (TEAM && ctas > 1) cluster_sync();  // every CTA's shared memory exists
    const Row w = row_of(r, p.rows, p.L);
    const int64_t chunks = (w.vectors + 31) / 32;
    const int64_t step = TEAM ? (int64_t)ctas * (blockDim.x >> 5) : 1;  // chunks of a round
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float h = p.h0 ? __ldg(p.h0 + r) : 0.f;  // the state entering the round
    int64_t c = TEAM ? (int64_t)rank * (blockDim.x >> 5) + warp : 0;
    int64_t e = w.base + c * kGatedChunk + lane * kE;
    Raw8<Tin> xr, gr, zr, xn, gn, zn;
    fetch<Tin>(xn, p.x, e, w);
    fetch<Tin>(gn, p.g, e, w);
    if (GATED) fetch<Tin>(zn, p.z, e, w);
    int buf = 0;
    // every warp of a team makes every round (its chunk may lie past the row: the identity)
    for (int64_t c_round = 0; c_round < chunks; c_round += step, c += step, e += step * kGatedChunk, buf ^= 1) {
        xr = xn, gr = gn;
        if (GATED) zr = zn;
        if (c_round + step < chunks) {
            fetch<Tin>(xn, p.x, e + step * kGatedChunk, w);
            fetch<Tin>(gn, p.g, e + step * kGatedChunk, w);
            if (GATED) fetch<Tin>(zn, p.z, e + step * kGatedChunk, w);
        }
        float x[kE], g[kE], a[kE], b[kE];
        xr.to_f(x);
        gr.to_f(g);
        steps<DECAY>(x, g, nbias, e, w, a, b);
        float P = a[0], H = b[0];
#pragma unroll
        for (int j = 1; j < kE; ++j) {
            H = fmaf(a[j], H, b[j]);
            P *= a[j];
        }
        scan_up(P, H, lane);
        const float P31 = __shfl_sync(kFull, P, 31), H31 = __shfl_sync(kFull, H, 31);
        float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
        if (lane == 0) Pe = 1.f, He = 0.f;
        float in;  // the state entering the warp's chunk
        if (TEAM) {
            in = team_round<true>(team, buf, ctas, rank, P31, H31, h);
        } else {
            in = h;
            h = fmaf(P31, h, H31);
        }
        if (c < chunks) {
            if (p.ck && lane == 0) p.ck[r * p.maxch + c] = in;
            if (p.y) {
                float hv = fmaf(Pe, in, He);
                float out[kE], z[kE];
                if (GATED) zr.to_f(z);
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    hv = fmaf(a[j], hv, b[j]);
                    out[j] = GATED ? hv * silu(z[j]) : hv;
                }
                put<Tout>(p.y, e, w, out);
            }
        }
    }
    if (p.last && lane == 0 && (!TEAM || (warp == 0 && rank == 0))) p.last[r] = h;
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
__global__ void __launch_bounds__(TEAM ? 32 * kTeamWarps : 32 * kWarps) gated_bwd_kernel(const RParams q) {
    __shared__ Team team;
    __shared__ float sums[kTeamWarps];
    const FParams& p = q.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = TEAM ? (int)cluster_ctas() : 1, rank = TEAM ? (int)cluster_rank() : 0;
    const int64_t r = TEAM ? blockIdx.x / ctas : (int64_t)blockIdx.x * kWarps + warp;
    if (!TEAM && r >= p.rows) return;
    if (TEAM && ctas > 1) cluster_sync();  // every CTA's shared memory exists
    const Row w = row_of(r, p.rows, p.L);
    const int64_t chunks = (w.vectors + 31) / 32;
    const int64_t step = TEAM ? (int64_t)ctas * (blockDim.x >> 5) : 1;
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float ec = q.dlast ? __ldg(q.dlast + r) : 0.f, bsum = 0.f;
    int64_t c_round = (chunks - 1) / step * step;
    int64_t c = c_round + (TEAM ? (int64_t)rank * (blockDim.x >> 5) + warp : 0);
    int64_t e = w.base + c * kGatedChunk + lane * kE;
    Raw8<T> xr, gr, yr, zr, xn, gn, yn, zn;
    float kn = c < chunks ? __ldg(p.ck + r * p.maxch + c) : 0.f;
    fetch<T>(xn, p.x, e, w);
    fetch<T>(gn, p.g, e, w);
    fetch<T>(yn, q.dy, e, w);
    if (GATED) fetch<T>(zn, p.z, e, w);
    int buf = 0;
    for (; c_round >= 0; c_round -= step, c -= step, e -= step * kGatedChunk, buf ^= 1) {
        xr = xn, gr = gn, yr = yn;
        if (GATED) zr = zn;
        const float entering = kn;
        if (c_round > 0) {
            const int64_t en = e - step * kGatedChunk;
            kn = __ldg(p.ck + r * p.maxch + c - step);
            fetch<T>(xn, p.x, en, w);
            fetch<T>(gn, p.g, en, w);
            fetch<T>(yn, q.dy, en, w);
            if (GATED) fetch<T>(zn, p.z, en, w);
        }
        float x[kE], g[kE], gy[kE], a[kE], b[kE], z[kE];
        xr.to_f(x);
        gr.to_f(g);
        yr.to_f(gy);
        steps<DECAY>(x, g, nbias, e, w, a, b);
        float dz[kE];  // dy times the derivative of silu(z), to be multiplied by the state
        if (GATED) {
            zr.to_f(z);
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const float sg = sigmoid_of(z[j] * -kLog2e);
                dz[j] = gy[j] * (sg * fmaf(z[j], 1.f - sg, 1.f));
                gy[j] *= z[j] * sg;
            }
        }
        const bool edge = e < w.lo || e + kE > w.hi;
        if (edge) {
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (e + j < w.lo || e + j >= w.hi) gy[j] = 0.f;
        }
        float P = 1.f, E = 0.f;
#pragma unroll
        for (int j = kE - 1; j >= 0; --j) {
            E = a[j] * (gy[j] + E);
            P *= a[j];
        }
        float Pd = P;
        scan_down(Pd, E, lane);
        const float P0 = __shfl_sync(kFull, Pd, 0), E0 = __shfl_sync(kFull, E, 0);
        float in;  // the adjoint entering the chunk from its right
        if (TEAM) {
            in = team_round<false>(team, buf, ctas, rank, P0, E0, ec);
            if (c >= chunks) continue;
        } else {
            in = ec;
            ec = fmaf(P0, ec, E0);
        }
        float hv[kE];  // the state before each step
        {
            float H = b[0];
#pragma unroll
            for (int j = 1; j < kE; ++j) H = fmaf(a[j], H, b[j]);
            scan_up(P, H, lane);
            float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
            if (lane == 0) Pe = 1.f, He = 0.f;
            hv[0] = fmaf(Pe, entering, He);
#pragma unroll
            for (int j = 1; j < kE; ++j) hv[j] = fmaf(a[j - 1], hv[j - 1], b[j - 1]);
        }
        if (GATED) {
#pragma unroll
            for (int j = 0; j < kE; ++j) dz[j] *= fmaf(a[j], hv[j], b[j]);
            put<T>(q.dz, e, w, dz);
        }
        float Pe = __shfl_down_sync(kFull, Pd, 1), Ee = __shfl_down_sync(kFull, E, 1);
        if (lane == 31) Pe = 1.f, Ee = 0.f;
        float ev = fmaf(Pe, in, Ee);
        float dx[kE], dg[kE];
#pragma unroll
        for (int j = kE - 1; j >= 0; --j) {
            const float dh = gy[j] + ev;
            ev = a[j] * dh;
            if (DECAY) {
                dx[j] = dh;
                dg[j] = dh * hv[j];
            } else {
                const float s = 1.f - a[j];
                dx[j] = s * dh;
                dg[j] = dx[j] * (x[j] - hv[j]) * a[j];
            }
        }
        put<T>(q.dx, e, w, dx);
        put<T>(q.dg, e, w, dg);
        if (!DECAY) {
            if (edge) {
#pragma unroll
                for (int j = 0; j < kE; ++j)
                    if (e + j < w.lo || e + j >= w.hi) dg[j] = 0.f;
            }
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
}

// dbias[d]: the partial sums of channel d's rows, in a fixed order (a warp per channel).
__global__ void gated_bias_kernel(const float* part, float* dbias, int64_t batch, int64_t dim,
                                  int64_t parts) {
    const int lane = threadIdx.x & 31;
    const int64_t d = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (d >= dim) return;
    float v = 0.f;
    for (int64_t i = lane; i < batch * parts; i += 32)
        v += part[((i / parts) * dim + d) * parts + i % parts];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    if (lane == 0) dbias[d] = v;
}

// One token: h = a h + b in place, a stream over (batch, dim).  V elements per thread.
template <typename T, bool DECAY, bool GATED, int V>
__global__ void __launch_bounds__(128) gated_update_kernel(float* state, const T* x, const T* gate,
                                                           const float* bias, const T* z, T* y,
                                                           int64_t n, int64_t dim) {
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V;
    if (i >= n) return;
    struct alignas(V * sizeof(T)) TV { T v[V]; };
    struct alignas(V * 4) FV { float v[V]; };
    const TV xv = *reinterpret_cast<const TV*>(x + i), gv = *reinterpret_cast<const TV*>(gate + i);
    TV zv, yv;
    if (GATED) zv = *reinterpret_cast<const TV*>(z + i);
    FV h = *reinterpret_cast<const FV*>(state + i), bv;
    const bool biased = !DECAY && bias != nullptr;
    if (biased) bv = *reinterpret_cast<const FV*>(bias + i % dim);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float xf = io<T>::to_f(xv.v[j]), gf = io<T>::to_f(gv.v[j]);
        if (DECAY) {
            h.v[j] = fmaf(gf, h.v[j], xf);
        } else {
            const float s = sigmoid_of(fmaf(gf, -kLog2e, biased ? -kLog2e * bv.v[j] : 0.f));
            h.v[j] = fmaf(1.f - s, h.v[j], s * xf);
        }
        yv.v[j] = io<T>::from_f(GATED ? h.v[j] * silu(io<T>::to_f(zv.v[j])) : h.v[j]);
    }
    *reinterpret_cast<FV*>(state + i) = h;
    *reinterpret_cast<TV*>(y + i) = yv;
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

// Launches `alone` with a warp per row, or `team` with the plan's warps and CTAs per row.
template <typename Params>
cudaError_t launch_rows(void (*alone)(Params), void (*team)(Params), const Params& p, int64_t rows,
                        const GatedTeam& t, cudaStream_t s) {
    if (t.warps * t.ctas == 1) {
        alone<<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, s>>>(p);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * t.ctas));
    cfg.blockDim = dim3((unsigned)(32 * t.warps));
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
    return launch_rows(gated_fwd_kernel<Tin, Tout, DECAY, GATED, false>,
                       gated_fwd_kernel<Tin, Tout, DECAY, GATED, true>, p, p.rows,
                       gated_team(p.rows, p.L, false), s);
}
template <typename Tin, typename Tout>
cudaError_t run_fwd_t(const FParams& p, bool decay, cudaStream_t s) {
    const bool gated = p.z != nullptr && p.y != nullptr;
    if (decay) return gated ? run_fwd<Tin, Tout, true, true>(p, s) : run_fwd<Tin, Tout, true, false>(p, s);
    return gated ? run_fwd<Tin, Tout, false, true>(p, s) : run_fwd<Tin, Tout, false, false>(p, s);
}

template <typename T, bool DECAY, bool GATED>
cudaError_t run_bwd(const RParams& q, cudaStream_t s) {
    return launch_rows(gated_bwd_kernel<T, DECAY, GATED, false>, gated_bwd_kernel<T, DECAY, GATED, true>, q,
                       q.f.rows, gated_team(q.f.rows, q.f.L, true), s);
}
template <typename T>
cudaError_t run_bwd_t(const RParams& q, bool decay, cudaStream_t s) {
    const bool gated = q.f.z != nullptr;
    if (decay) return gated ? run_bwd<T, true, true>(q, s) : run_bwd<T, true, false>(q, s);
    return gated ? run_bwd<T, false, true>(q, s) : run_bwd<T, false, false>(q, s);
}

template <typename T, int V>
cudaError_t run_update(const GatedUpdateArgs& a, cudaStream_t s) {
    const int64_t n = a.batch * a.dim;
    const unsigned blocks = (unsigned)((n / V + 127) / 128);
    const T *x = static_cast<const T*>(a.x), *g = static_cast<const T*>(a.gate),
            *z = static_cast<const T*>(a.z);
    T* y = static_cast<T*>(a.y);
    if (a.given_decay) {
        if (z) gated_update_kernel<T, true, true, V><<<blocks, 128, 0, s>>>(a.state, x, g, a.gate_bias, z, y, n, a.dim);
        else gated_update_kernel<T, true, false, V><<<blocks, 128, 0, s>>>(a.state, x, g, a.gate_bias, z, y, n, a.dim);
    } else {
        if (z) gated_update_kernel<T, false, true, V><<<blocks, 128, 0, s>>>(a.state, x, g, a.gate_bias, z, y, n, a.dim);
        else gated_update_kernel<T, false, false, V><<<blocks, 128, 0, s>>>(a.state, x, g, a.gate_bias, z, y, n, a.dim);
    }
    return cudaGetLastError();
}

}  // namespace

// Warps that walk a row: one while the rows alone give every SM `per_sm` of them (32 forward, 16
// for the backward's larger register need); else as many as bring it there, in one CTA, or in a
// cluster of up to 8 where there are fewer rows than CTA places; never more than the row has chunks.
GatedTeam gated_team(int64_t rows, int64_t L, bool backward) {
    constexpr int64_t kSms = 148;
    const int64_t per_sm = backward ? 16 : 32, chunks = std::max<int64_t>(1, gated_chunks(L));
    const int64_t ctas_per_sm = (rows + kSms - 1) / kSms;
    GatedTeam t{1, 1};
    const int64_t warps = std::min<int64_t>({kTeamWarps, per_sm / std::min(ctas_per_sm, per_sm), chunks});
    if (warps <= 1) return t;
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
    q.bias_part = g.dbias ? g.bias_part : nullptr;
    cudaError_t e = a.in_dtype == DType::BF16 ? run_bwd_t<__nv_bfloat16>(q, a.given_decay != 0, s)
                                              : run_bwd_t<float>(q, a.given_decay != 0, s);
    if (e == cudaSuccess && g.dbias) {
        gated_bias_kernel<<<(unsigned)((a.dim + 3) / 4), 128, 0, s>>>(g.bias_part, g.dbias,
                                                                     a.rows / a.dim, a.dim,
                                                                     gated_team(a.rows, a.L, true).ctas);
        e = cudaGetLastError();
    }
    return e;
}

cudaError_t launch_gated_update(const GatedUpdateArgs& a, cudaStream_t s) {
    // Vectors of 4 where a row is a whole number of them (the bias is read as a vector too).
    if (a.dtype == DType::BF16)
        return a.dim % 4 == 0 ? run_update<__nv_bfloat16, 4>(a, s) : run_update<__nv_bfloat16, 1>(a, s);
    return a.dim % 4 == 0 ? run_update<float, 4>(a, s) : run_update<float, 1>(a, s);
}

}  // namespace s6
