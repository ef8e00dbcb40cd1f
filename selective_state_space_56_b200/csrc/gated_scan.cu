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
// Few rows leave most of the machine idle, so then each row is cut into segments, a warp
// each: one launch composes every segment, a second walks them from their true starts, which
// each warp forms itself from the compositions before its own.
#include <algorithm>

#include "layer_launch.h"
#include "row8.cuh"

namespace s6 {
namespace {

static_assert(kE == kGatedLane, "a lane takes one vector");
constexpr int kWarps = 4;  // per CTA
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
    const float2* agg;
    float2* agg_out;
    int64_t rows, dim, L, maxch, nseg, seg_chunks;
};

// The state entering segment `seg` of row r: h0 through the compositions of the segments
// before it, 32 at a time.
__device__ __forceinline__ float enter_forward(const float2* agg, float h, int64_t seg, int lane) {
    for (int64_t s0 = 0; s0 < seg; s0 += 32) {
        float P = 1.f, H = 0.f;
        if (s0 + lane < seg) {
            const float2 v = agg[s0 + lane];
            P = v.x, H = v.y;
        }
        scan_up(P, H, lane);
        h = fmaf(__shfl_sync(kFull, P, 31), h, __shfl_sync(kFull, H, 31));
    }
    return h;
}

// MODE 0: outputs (y unless null, last state, checkpoints).  MODE 1: the composition of the
// warp's segment only.
template <typename Tin, typename Tout, bool DECAY, bool GATED, int MODE>
__global__ void __launch_bounds__(32 * kWarps) gated_fwd_kernel(const FParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= p.rows * p.nseg) return;
    const int64_t r = unit / p.nseg, seg = unit - r * p.nseg;
    const Row w = row_of(r, p.rows, p.L);
    const int64_t c0 = seg * p.seg_chunks;
    const int64_t c1 = min((w.vectors + 31) / 32, c0 + p.seg_chunks);
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float h = 0.f, Pall = 1.f;
    if (MODE == 0) {
        h = p.h0 ? __ldg(p.h0 + r) : 0.f;
        if (seg > 0) h = enter_forward(p.agg + r * p.nseg, h, seg, lane);
    }
    Raw8<Tin> xr, gr, zr, xn, gn, zn;
    int64_t e = w.base + c0 * kGatedChunk + lane * kE;
    if (c0 < c1) {
        fetch<Tin>(xn, p.x, e, w);
        fetch<Tin>(gn, p.g, e, w);
        if (GATED) fetch<Tin>(zn, p.z, e, w);
    }
    for (int64_t c = c0; c < c1; ++c, e += kGatedChunk) {
        xr = xn, gr = gn;
        if (GATED) zr = zn;
        if (c + 1 < c1) {
            fetch<Tin>(xn, p.x, e + kGatedChunk, w);
            fetch<Tin>(gn, p.g, e + kGatedChunk, w);
            if (GATED) fetch<Tin>(zn, p.z, e + kGatedChunk, w);
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
        if (MODE == 0) {
            if (p.ck && lane == 0) p.ck[r * p.maxch + c] = h;
            float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
            if (lane == 0) Pe = 1.f, He = 0.f;
            if (p.y) {
                float hv = fmaf(Pe, h, He);
                float out[kE], z[kE];
                if (GATED) zr.to_f(z);
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    hv = fmaf(a[j], hv, b[j]);
                    out[j] = GATED ? hv * silu(z[j]) : hv;
                }
                put<Tout>(p.y, e, w, out);
            }
        } else {
            Pall *= P31;
        }
        h = fmaf(P31, h, H31);
    }
    if (MODE == 1) {
        if (lane == 0) p.agg_out[r * p.nseg + seg] = make_float2(Pall, h);
    } else if (p.last && seg == p.nseg - 1 && lane == 0) {
        p.last[r] = h;
    }
}

struct RParams {
    FParams f;
    const void* dy;
    const float* dlast;
    void* dx;
    void* dg;
    void* dz;
    float* dh0;
    float* bias_part;
};

// The adjoint entering segment `seg` of row r from its right: dlast through the
// compositions of the segments after it.
__device__ __forceinline__ float enter_backward(const float2* agg, float e, int64_t seg,
                                                int64_t nseg, int lane) {
    for (int64_t s1 = nseg; s1 > seg + 1; s1 -= 32) {  // lane l holds segment s1 - 32 + l
        float P = 1.f, E = 0.f;
        const int64_t s = s1 - 32 + lane;
        if (s > seg) {
            const float2 v = agg[s];
            P = v.x, E = v.y;
        }
        scan_down(P, E, lane);
        e = fmaf(__shfl_sync(kFull, P, 0), e, __shfl_sync(kFull, E, 0));
    }
    return e;
}

// The backward: with e_t the adjoint handed to h_t from later steps,
//   dh_t = dy_t silu(z_t) + e_t,  e_{t-1} = a_t dh_t,
// the recurrence again, backwards, with the same a.  MODE 0: the gradients; a chunk's states
// are formed again from its checkpoint.  MODE 1: the segment's composition only.
template <typename T, bool DECAY, bool GATED, int MODE>
__global__ void __launch_bounds__(32 * kWarps) gated_bwd_kernel(const RParams q) {
    const FParams& p = q.f;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= p.rows * p.nseg) return;
    const int64_t r = unit / p.nseg, seg = unit - r * p.nseg;
    const Row w = row_of(r, p.rows, p.L);
    const int64_t c0 = seg * p.seg_chunks;
    const int64_t c1 = min((w.vectors + 31) / 32, c0 + p.seg_chunks);
    const float nbias = p.bias ? -kLog2e * __ldg(p.bias + r % p.dim) : 0.f;
    float ec = 0.f, Pall = 1.f, bsum = 0.f;
    if (MODE == 0) {
        ec = q.dlast ? __ldg(q.dlast + r) : 0.f;
        if (seg + 1 < p.nseg) ec = enter_backward(p.agg + r * p.nseg, ec, seg, p.nseg, lane);
    }
    Raw8<T> xr, gr, yr, zr, xn, gn, yn, zn;
    int64_t e = w.base + (c1 - 1) * kGatedChunk + lane * kE;
    if (c0 < c1) {
        if (MODE == 0) fetch<T>(xn, p.x, e, w);
        fetch<T>(gn, p.g, e, w);
        fetch<T>(yn, q.dy, e, w);
        if (GATED) fetch<T>(zn, p.z, e, w);
    }
    for (int64_t c = c1 - 1; c >= c0; --c, e -= kGatedChunk) {
        if (MODE == 0) xr = xn;
        gr = gn, yr = yn;
        if (GATED) zr = zn;
        if (c > c0) {
            if (MODE == 0) fetch<T>(xn, p.x, e - kGatedChunk, w);
            fetch<T>(gn, p.g, e - kGatedChunk, w);
            fetch<T>(yn, q.dy, e - kGatedChunk, w);
            if (GATED) fetch<T>(zn, p.z, e - kGatedChunk, w);
        }
        float x[kE], g[kE], gy[kE], a[kE], b[kE], z[kE];
        if (MODE == 0) xr.to_f(x);
        else
#pragma unroll
            for (int j = 0; j < kE; ++j) x[j] = 0.f;
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
        if (MODE == 0) {
            float hv[kE];  // the state before each step
            {
                float H = b[0];
#pragma unroll
                for (int j = 1; j < kE; ++j) H = fmaf(a[j], H, b[j]);
                scan_up(P, H, lane);
                float Pe = __shfl_up_sync(kFull, P, 1), He = __shfl_up_sync(kFull, H, 1);
                if (lane == 0) Pe = 1.f, He = 0.f;
                hv[0] = fmaf(Pe, __ldg(p.ck + r * p.maxch + c), He);
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
            float ev = fmaf(Pe, ec, Ee);
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
        } else {
            Pall *= P0;
        }
        ec = fmaf(P0, ec, E0);
    }
    if (MODE == 1) {
        if (lane == 0) const_cast<float2*>(p.agg)[r * p.nseg + seg] = make_float2(Pall, ec);
        return;
    }
    if (q.dh0 && seg == 0 && lane == 0) q.dh0[r] = ec;
    if (q.bias_part) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) bsum += __shfl_xor_sync(kFull, bsum, o);
        if (lane == 0) q.bias_part[r * p.nseg + seg] = bsum;
    }
}

// dbias[d]: the partial sums of channel d's rows, in a fixed order (a warp per channel).
__global__ void gated_bias_kernel(const float* part, float* dbias, int64_t batch, int64_t dim,
                                  int64_t nseg) {
    const int lane = threadIdx.x & 31;
    const int64_t d = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (d >= dim) return;
    float v = 0.f;
    for (int64_t i = lane; i < batch * nseg; i += 32)
        v += part[((i / nseg) * dim + d) * nseg + i % nseg];
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

unsigned warp_blocks(int64_t units) { return (unsigned)((units + kWarps - 1) / kWarps); }

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
    p.agg = a.agg;
    p.agg_out = a.agg;
    p.rows = a.rows;
    p.dim = a.dim;
    p.L = a.L;
    p.maxch = gated_chunks(a.L);
    gated_plan(a.rows, a.L, &p.nseg, &p.seg_chunks);
    return p;
}

template <typename Tin, typename Tout, bool DECAY, bool GATED>
cudaError_t run_fwd(const FParams& p, cudaStream_t s) {
    const unsigned blocks = warp_blocks(p.rows * p.nseg);
    if (p.nseg > 1) {
        gated_fwd_kernel<Tin, Tin, DECAY, false, 1><<<blocks, 32 * kWarps, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    gated_fwd_kernel<Tin, Tout, DECAY, GATED, 0><<<blocks, 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename Tin, typename Tout>
cudaError_t run_fwd_t(const FParams& p, bool decay, cudaStream_t s) {
    const bool gated = p.z != nullptr && p.y != nullptr;
    if (decay) return gated ? run_fwd<Tin, Tout, true, true>(p, s) : run_fwd<Tin, Tout, true, false>(p, s);
    return gated ? run_fwd<Tin, Tout, false, true>(p, s) : run_fwd<Tin, Tout, false, false>(p, s);
}

template <typename T, bool DECAY, bool GATED>
cudaError_t run_bwd(const RParams& q, cudaStream_t s) {
    const unsigned blocks = warp_blocks(q.f.rows * q.f.nseg);
    if (q.f.nseg > 1) {
        gated_bwd_kernel<T, DECAY, GATED, 1><<<blocks, 32 * kWarps, 0, s>>>(q);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    gated_bwd_kernel<T, DECAY, GATED, 0><<<blocks, 32 * kWarps, 0, s>>>(q);
    return cudaGetLastError();
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

void gated_plan(int64_t rows, int64_t L, int64_t* nseg, int64_t* seg_chunks) {
    const int64_t chunks = std::max<int64_t>(1, gated_chunks(L));
    int64_t n = 1;
    constexpr int64_t kEnough = 148 * 16, kTarget = 148 * 32, kLeast = 4;
    if (rows < kEnough) n = std::min((kTarget + rows - 1) / rows, (chunks + kLeast - 1) / kLeast);
    *seg_chunks = (chunks + n - 1) / n;
    *nseg = (chunks + *seg_chunks - 1) / *seg_chunks;
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
                                                                     a.rows / a.dim, a.dim, q.f.nseg);
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
