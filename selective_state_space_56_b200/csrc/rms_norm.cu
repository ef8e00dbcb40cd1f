// rms_norm.cu -- the residual addition with RMS norm that opens a block (forward to fp32,
// bf16 or e4m3 with scales; backward), and the quantisation to e4m3, for sm_100a.
//
//   v = residual + x (kept in the residual stream's type),  rstd = 1 / sqrt(mean v^2 + eps)
//   out = v rstd weight
// and with xhat = v rstd, g = dout weight, dv the gradient arriving at the stream:
//   dx = dresidual = dv + rstd (g - xhat mean(g xhat)),   dweight = sum over rows dout xhat.
//
// All of it is bound by memory (11 bytes an element for the fp32 stream with e4m3 output), so
// a row is read once, kept in registers between the sum and the scaling, and written once.
// The sums are fp32: per thread, then over the warp, then over the CTA.
#include <algorithm>

#include "layer_launch.h"
#include "row8.cuh"

namespace s6 {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxThreads = 512;

// A row belongs to one CTA, or (ALONE: up to 768 columns) to one of the eight warps of a CTA,
// which then needs no barrier: a thread's place in the row and the row's threads.
constexpr int kAloneWarps = 8;
template <bool ALONE>
__device__ __forceinline__ int place() { return ALONE ? threadIdx.x & 31 : threadIdx.x; }
template <bool ALONE>
__device__ __forceinline__ int threads() { return ALONE ? 32 : blockDim.x; }

// Sum of two values over the row's threads, the same bits in every one.
template <bool ALONE>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(kFull, v.x, o);
        v.y += __shfl_xor_sync(kFull, v.y, o);
    }
    const int warps = blockDim.x >> 5;
    if (ALONE || warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 t = red[0];
    for (int i = 1; i < warps; ++i) t.x += red[i].x, t.y += red[i].y;
    return t;
}

struct NParams {
    const void* x;
    const void* res;
    const float* w;
    void* out;
    float* scales;
    void* res_out;
    int64_t rows, dim;
    float eps;
};

// Weights of the 8 columns from column c (c = e - row start, possibly negative at the edge).
template <bool ALIGNED>
__device__ __forceinline__ void weights8(const float* w, int64_t c, int64_t dim, float (&o)[kE]) {
    if (ALIGNED) {
        Raw8<float> r;
        r.load(w + c);
        r.to_f(o);
    } else if (c >= 0 && c + kE <= dim) {
#pragma unroll
        for (int j = 0; j < kE; ++j) o[j] = __ldg(w + c + j);
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) o[j] = (c + j >= 0 && c + j < dim) ? __ldg(w + c + j) : 0.f;
    }
}

// V vectors of 8 per thread.  ALIGNED: dim is a multiple of 8.  OUT: the
// output's type; FP8 writes e4m3 and a scale per 128 columns (dim is a multiple of 16 then):
// 16 lanes hold the 128 columns of a group, and its largest magnitude is their shuffled maximum.
template <typename Tx, typename Tr, typename Tout, int V, bool ALIGNED, bool FP8, bool ALONE>
__global__ void __launch_bounds__(ALONE ? 32 * kAloneWarps : kMaxThreads) norm_kernel(const NParams p) {
    __shared__ float2 red[kMaxThreads / 32];
    const int64_t row = ALONE ? (int64_t)blockIdx.x * kAloneWarps + (threadIdx.x >> 5) : blockIdx.x;
    if (ALONE && row >= p.rows) return;
    const Row w = row_of(row, p.rows, p.dim);
    float v[V][kE];
    Raw8<Tx> xr[V];
    Raw8<Tr> rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + (i * threads<ALONE>() + place<ALONE>()) * kE;
        fetch<Tx>(xr[i], p.x, e, w);
        if (p.res) fetch<Tr>(rr[i], p.res, e, w);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + (i * threads<ALONE>() + place<ALONE>()) * kE;
        xr[i].to_f(v[i]);
        if (p.res) {
            float r[kE];
            rr[i].to_f(r);
#pragma unroll
            for (int j = 0; j < kE; ++j) v[i][j] = io<Tr>::to_f(io<Tr>::from_f(v[i][j] + r[j]));
        }
        if (!ALIGNED && (e < w.lo || e + kE > w.hi)) {
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (e + j < w.lo || e + j >= w.hi) v[i][j] = 0.f;
        }
        if (p.res_out) put<Tr>(p.res_out, e, w, v[i]);
#pragma unroll
        for (int j = 0; j < kE; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    const float2 t = row_sum2<ALONE>(make_float2(ss, 0.f), red);
    const float rstd = rsqrtf(t.x / (float)p.dim + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + (i * threads<ALONE>() + place<ALONE>()) * kE;
        const bool in = e < w.hi;
        float o[kE] = {};
        if (in) {
            float wt[kE];
            weights8<ALIGNED>(p.w, e - w.lo, p.dim, wt);
            // e4m3: rstd goes into the scale alone, since it cancels in out / scale
#pragma unroll
            for (int j = 0; j < kE; ++j) o[j] = FP8 ? v[i][j] * wt[j] : v[i][j] * rstd * wt[j];
        }
        if (FP8) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < kE; ++j) m = fmaxf(m, fabsf(o[j]));
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
            if (in) {
                const float top = m * rstd;  // the group's largest output
                float largest = m;
                // rstd goes into the values where without it they, or with it the outputs, are so small
                // that the quotient's factors would leave fp32's range (groups of zeros; small eps)
                if (!(m >= kAmaxFloor && top >= kAmaxFloor)) {
                    largest = fmaxf(top, kAmaxFloor);
#pragma unroll
                    for (int j = 0; j < kE; ++j) o[j] *= rstd;
                }
                const Quotient by(largest);
                by(o);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + e) = to_e4m3(o);
                const int64_t c = e - w.lo, groups = (p.dim + kGroup - 1) / kGroup;
                if (c % kGroup == 0)
                    p.scales[row * groups + c / kGroup] = fmaxf(top, kAmaxFloor) / kE4m3Max;
            }
        } else if (in) {
            put<Tout>(p.out, e, w, o);
        }
    }
}

struct BNParams {
    const void* dout;
    const void* s;
    const float* w;
    const void* ds;
    void* dx;
    void* dres;
    float* part;
    int64_t rows, dim;
    float eps;
};

// CTAs (or warps: ALONE) walk rows with the grid's stride and keep their share of dweight in
// registers; the shares are summed by dweight_kernel in a fixed order (no atomics: the same call
// gives the same bits).  A thread's columns are the same in every row only when rows begin at
// vector boundaries (dim a multiple of 8); others go to norm_bwd_elem_kernel.  The next row's
// loads are in flight while this one is computed, which the weights make room for by staying in
// shared memory.
template <typename Tx, typename Tr, int V, bool ALONE>
__global__ void __launch_bounds__(ALONE ? 32 * kAloneWarps : kMaxThreads, ALONE ? 2 : 1) norm_bwd_kernel(const BNParams p) {
    __shared__ float2 red[2][kMaxThreads / 32];
    __shared__ alignas(16) float sums[ALONE ? kAloneWarps * V * 32 * kE : 4];
    extern __shared__ float4 weight4[];
    const int64_t first = ALONE ? (int64_t)blockIdx.x * kAloneWarps + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t stride = ALONE ? (int64_t)gridDim.x * kAloneWarps : gridDim.x;
    const int dim = (int)p.dim;
    const auto column = [](int i) { return (i * threads<ALONE>() + place<ALONE>()) * kE; };
    Raw8<Tx> gn[V];
    Raw8<Tr> sn[V], dn[V];
    const auto load = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t e = r * dim + column(i);
            sn[i].zero(), gn[i].zero();
            if (p.ds) dn[i].zero();
            if (column(i) < dim) {
                sn[i].load(static_cast<const Tr*>(p.s) + e);
                gn[i].load(static_cast<const Tx*>(p.dout) + e);
                if (p.ds) dn[i].load(static_cast<const Tr*>(p.ds) + e);
            }
        }
    };
    if (first < p.rows) load(first);
    for (int c = threadIdx.x; c < dim / 4; c += blockDim.x) weight4[c] = reinterpret_cast<const float4*>(p.w)[c];
    __syncthreads();
    float dw[V][kE];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < kE; ++j) dw[i][j] = 0.f;
    const auto weights = [&](int i, float (&o)[kE]) {
        const float4 a = weight4[column(i) / 4], b = weight4[column(i) / 4 + 1];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w, o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    };
    int flip = 0;
    for (int64_t r = first; r < p.rows; r += stride, flip ^= 1) {
        Raw8<Tx> gr[V];
        Raw8<Tr> sr[V], dr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sr[i] = sn[i], gr[i] = gn[i];
            if (p.ds) dr[i] = dn[i];
        }
        if (r + stride < p.rows) load(r + stride);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (column(i) >= dim) continue;
            float v[kE], g[kE], wt[kE];
            sr[i].to_f(v);
            gr[i].to_f(g);
            weights(i, wt);
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                sum.x = fmaf(v[j], v[j], sum.x);
                sum.y = fmaf(g[j] * wt[j], v[j], sum.y);
            }
        }
        sum = row_sum2<ALONE>(sum, red[flip]);
        const float rstd = rsqrtf(sum.x / (float)dim + p.eps);
        const float k = sum.y / (float)dim * rstd * rstd;  // mean(g xhat) rstd
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (column(i) >= dim) continue;
            const int64_t e = r * dim + column(i);
            float v[kE], g[kE], d[kE], wt[kE];
            sr[i].to_f(v);
            gr[i].to_f(g);
            weights(i, wt);
            if (p.ds) {
                dr[i].to_f(d);
            } else {
#pragma unroll
                for (int j = 0; j < kE; ++j) d[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                dw[i][j] = fmaf(g[j], v[j] * rstd, dw[i][j]);
                d[j] = fmaf(rstd, fmaf(-k, v[j], g[j] * wt[j]), d[j]);
            }
            store_all(static_cast<Tx*>(p.dx) + e, d);
            if (p.dres) store_all(static_cast<Tr*>(p.dres) + e, d);
        }
    }
    float* part = p.part + (int64_t)blockIdx.x * dim;
    if (ALONE) {  // the warps' shares, in order
#pragma unroll
        for (int i = 0; i < V; ++i) store_all(sums + (threadIdx.x >> 5) * V * 32 * kE + column(i), dw[i]);
        __syncthreads();
        for (int c = threadIdx.x; c < dim; c += 32 * kAloneWarps) {
            float t = sums[c];
#pragma unroll
            for (int w = 1; w < kAloneWarps; ++w) t += sums[w * V * 32 * kE + c];
            part[c] = t;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (column(i) < dim) store_all(part + column(i), dw[i]);
}

// The same for any dim: a thread takes C single columns, threadIdx.x + i blockDim.x, of every
// row, so that its share of dweight is its own there too (in registers up to C = 8; the instance of 32,
// for widths above 4096, keeps its arrays in local memory, 1 KB a thread); the next row's values are
// on their way while this one is computed.  (16384, 1023) bf16: 122 us with two passes over a row
// and shares in memory, 57 so.
template <typename Tx, typename Tr, int C>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_elem_kernel(const BNParams p) {
    __shared__ float2 red[2][kMaxThreads / 32];
    const int dim = (int)p.dim;
    const auto column = [](int i) { return (int)(threadIdx.x + i * blockDim.x); };
    Tr sn[C], dn[C];
    Tx gn[C];
    const auto load = [&](int64_t r) {
        const int64_t at = r * dim;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = column(i);
            sn[i] = dn[i] = io<Tr>::from_f(0.f), gn[i] = io<Tx>::from_f(0.f);
            if (c < dim) {
                sn[i] = static_cast<const Tr*>(p.s)[at + c];
                gn[i] = static_cast<const Tx*>(p.dout)[at + c];
                if (p.ds) dn[i] = static_cast<const Tr*>(p.ds)[at + c];
            }
        }
    };
    load(blockIdx.x);  // no more CTAs than rows
    float wt[C], dw[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        wt[i] = column(i) < dim ? __ldg(p.w + column(i)) : 0.f;
        dw[i] = 0.f;
    }
    int flip = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1) {
        float v[C], g[C], d[C];
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] = io<Tr>::to_f(sn[i]), g[i] = io<Tx>::to_f(gn[i]), d[i] = io<Tr>::to_f(dn[i]);
        if (r + gridDim.x < p.rows) load(r + gridDim.x);
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < C; ++i) {
            sum.x = fmaf(v[i], v[i], sum.x);
            sum.y = fmaf(g[i] * wt[i], v[i], sum.y);
        }
        sum = row_sum2<false>(sum, red[flip]);
        const float rstd = rsqrtf(sum.x / (float)dim + p.eps);
        const float k = sum.y / (float)dim * rstd * rstd;
        const int64_t at = r * dim;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            dw[i] = fmaf(g[i], v[i] * rstd, dw[i]);
            d[i] = fmaf(rstd, fmaf(-k, v[i], g[i] * wt[i]), d[i]);
            if (column(i) < dim) {
                static_cast<Tx*>(p.dx)[at + column(i)] = io<Tx>::from_f(d[i]);
                if (p.dres) static_cast<Tr*>(p.dres)[at + column(i)] = io<Tr>::from_f(d[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (column(i) < dim) p.part[(int64_t)blockIdx.x * dim + column(i)] = dw[i];
}

// Columns' sums of part (blocks, dim): 8 columns per CTA, 32 rows side by side.
__global__ void __launch_bounds__(256) dweight_kernel(const float* part, float* dw, int64_t blocks,
                                                      int64_t dim) {
    __shared__ float red[32][9];
    const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 8 + cx;
    float v = 0.f;
    cudaGridDependencySynchronize();  // launched early: wait for the shares, which no read-only
                                      // load may fetch: they are written while this kernel runs
    if (c < dim)
#pragma unroll 8
        for (int64_t r = ry; r < blocks; r += 32) v += part[r * dim + c];
    red[ry][cx] = v;
    __syncthreads();
    if (ry == 0 && c < dim) {
        float t = red[0][cx];
        for (int i = 1; i < 32; ++i) t += red[i][cx];
        dw[c] = t;
    }
}

// ---- Quantisation --------------------------------------------------------------------

// Row-major: 16 lanes take a group of 128, 8 values each, and kBatch groups one after another
// whose loads are issued together.  Groups are numbered over rows padded to whole ones; WHOLE
// (dim a multiple of 128): group g lies at 128 g.  (16384, 2560) bf16: 29.2 us with one
// group a thread, 21.0 with four; 21.8 us (5.8 TB/s) since the quotients are rounded once.
constexpr int kBatch = 4;
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(256) quantize_kernel(const T* x, uint8_t* q, float* scales,
                                                       int64_t rows, int64_t dim) {
    const int64_t groups = (dim + kGroup - 1) / kGroup, all = rows * groups;
    const int64_t g0 = (int64_t)blockIdx.x * (16 * kBatch) + (threadIdx.x >> 4);
    const int lane = threadIdx.x & 15;
    int64_t at[kBatch];
    Raw8<T> raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int64_t g = g0 + i * 16;
        at[i] = -1;
        if (WHOLE) {
            if (g < all) at[i] = g * kGroup + lane * kE;
        } else {
            const int64_t r = g / groups, c = (g - r * groups) * kGroup + lane * kE;
            if (r < rows && c < dim) at[i] = r * dim + c;
        }
        raw[i].zero();
        if (at[i] >= 0) raw[i].load(x + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        float v[kE], m = 0.f;
        raw[i].to_f(v);
#pragma unroll
        for (int j = 0; j < kE; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
        for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
        m = fmaxf(m, kAmaxFloor);
        if (at[i] < 0) continue;
        const Quotient by(m);
        by(v);
        *reinterpret_cast<uint2*>(q + at[i]) = to_e4m3(v);
        if (lane == 0) scales[g0 + i * 16] = m / kE4m3Max;
    }
}

// Channel-major (batch, dim, L) to token rows (batch * L, dim): a CTA takes 128 channels of 64
// tokens through shared memory, read along the tokens and written along the channels.  The
// channels' rows are copied in 16-byte vectors of the whole array (asynchronously, so that
// six CTAs keep 110 KB an SM on the way), which a row may enter at any element: a row's first
// token lies `shift` elements into its copy.  A thread holds 16 channels of
// two tokens; the e4m3 values go back through shared memory, so that a token's 128 bytes are
// stored as one line.
// Two neighbouring elements, and the running maximum of such pairs' magnitudes.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    __nv_bfloat162 v;
    __device__ __forceinline__ static Pair of(__nv_bfloat16 a, __nv_bfloat16 b) { return {__nv_bfloat162(a, b)}; }
    __device__ __forceinline__ static Pair zero() { return {__floats2bfloat162_rn(0.f, 0.f)}; }
    __device__ __forceinline__ void max_abs(Pair w) { v = __hmax2(v, __habs2(w.v)); }
    __device__ __forceinline__ float2 f() const { return __bfloat1622float2(v); }
    __device__ __forceinline__ f2 packed() const { return bf16pair(*reinterpret_cast<const uint32_t*>(&v)); }
};
template <> struct Pair<float> {
    float2 v;
    __device__ __forceinline__ static Pair of(float a, float b) { return {make_float2(a, b)}; }
    __device__ __forceinline__ static Pair zero() { return {make_float2(0.f, 0.f)}; }
    __device__ __forceinline__ void max_abs(Pair w) { v = make_float2(fmaxf(v.x, fabsf(w.v.x)), fmaxf(v.y, fabsf(w.v.y))); }
    __device__ __forceinline__ float2 f() const { return v; }
    __device__ __forceinline__ f2 packed() const { return pack2(v.x, v.y); }
};

// ALIGNED: rows begin at vector boundaries (L a multiple of the vector), so all shifts are zero
// and a thread reads its two tokens of a channel at once.
constexpr int kTok = 64;
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 6 : 4) quantize_cm_kernel(const T* x, uint8_t* q, float* scales,
                                                          int64_t dim, int64_t L, int64_t total) {
    constexpr int kVec = 16 / sizeof(T);       // elements of a copy
    constexpr int kVecs = kTok / kVec + (ALIGNED ? 0 : 1);  // copies of a row's 64 tokens
    constexpr int kPitch = (kTok / kVec + 1) * kVec;
    __shared__ alignas(16) T tile[kGroup * kPitch];
    __shared__ float2 mx[8][kTok / 2];
    static_assert(kTok * kGroup <= (int)sizeof(tile), "the output goes where the input was");
    const int64_t t0 = (int64_t)blockIdx.x * kTok, c0 = (int64_t)blockIdx.y * kGroup, b = blockIdx.z;
    const int nc = (int)min((int64_t)kGroup, dim - c0), nt = (int)min((int64_t)kTok, L - t0);
    const int64_t first = (b * dim + c0) * L + t0;  // the tile's first element
    if (ALIGNED) {
        const int v = threadIdx.x % kVecs;
        const T* src = x + first + v * kVec;
        if (v * kVec < nt)
#pragma unroll
            for (int c = threadIdx.x / kVecs; c < kGroup; c += 256 / kVecs)
                if (c < nc) cp_async16(tile + c * kPitch + v * kVec, src + c * L, 16);
    } else {
        for (int i = threadIdx.x; i < nc * kVecs; i += 256) {
            const int c = i / kVecs, v = i - c * kVecs;
            const int64_t e = ((first + c * L) & ~(int64_t)(kVec - 1)) + v * kVec;
            const int64_t left = total - e;  // elements up to the array's end
            if (left > 0)
                cp_async16(tile + c * kPitch + v * kVec, x + e, left < kVec ? (int)left * (int)sizeof(T) : 16);
        }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    // two tokens of 16 channels
    const int t = (threadIdx.x % (kTok / 2)) * 2, part = threadIdx.x / (kTok / 2);
    Pair<T> w[16], m = Pair<T>::zero();
    if (part * 16 < nc) {
        const T* at = tile + part * 16 * kPitch + t;
        const int step = (int)(L & (kVec - 1));
        int shift = (int)((first + part * 16 * L) & (kVec - 1));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (ALIGNED) {
                w[i] = *reinterpret_cast<const Pair<T>*>(at + i * kPitch);
            } else {
                w[i] = Pair<T>::of(at[i * kPitch + shift], at[i * kPitch + shift + 1]);
                shift = (shift + step) & (kVec - 1);
            }
            m.max_abs(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = Pair<T>::zero();
    }
    mx[part][t / 2] = m.f();
    __syncthreads();
    float m0 = kAmaxFloor, m1 = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < 8; ++i) m0 = fmaxf(m0, mx[i][t / 2].x), m1 = fmaxf(m1, mx[i][t / 2].y);
    // piece `part` of token r at place part ^ (r / 2 % 8) of its 128 bytes: no bank conflicts
    // where it is written (every second token) and none where it is read (whole tokens)
    uint8_t* staged = reinterpret_cast<uint8_t*>(tile);
    {
        const Quotient by(m0, m1);
        uint8_t* at = staged + t * kGroup + ((part ^ (t / 2 & 7)) * 16);
#pragma unroll
        for (int i = 0; i < 16; i += kE) {
            float v0[kE], v1[kE];
#pragma unroll
            for (int j = 0; j < kE; ++j) unpack2(by(w[i + j].packed()), v0[j], v1[j]);
            *reinterpret_cast<uint2*>(at + i) = to_e4m3(v0);
            *reinterpret_cast<uint2*>(at + kGroup + i) = to_e4m3(v1);
        }
    }
    if (part == 0) {
        const int64_t groups = (dim + kGroup - 1) / kGroup;
        float* sc = scales + (b * L + t0 + t) * groups + blockIdx.y;
        if (t < nt) sc[0] = m0 / kE4m3Max;
        if (t + 1 < nt) sc[groups] = m1 / kE4m3Max;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (threadIdx.x >> 3) + i * 32, c = threadIdx.x & 7;
        if (r < nt && c * 16 < nc)
            *reinterpret_cast<uint4*>(q + (b * L + t0 + r) * dim + c0 + c * 16) =
                *reinterpret_cast<const uint4*>(staged + r * kGroup + ((c ^ (r / 2 & 7)) * 16));
    }
}

// Weights: a CTA per block of 128 x 128; thread (row, half) holds 64 columns of its row.
template <typename T>
__global__ void __launch_bounds__(256) quantize_weight_kernel(const T* w, uint8_t* q, float* scales,
                                                              int64_t n, int64_t k) {
    __shared__ float mx[8];
    const int64_t r = (int64_t)blockIdx.y * kGroup + (threadIdx.x >> 1);
    const int64_t c = (int64_t)blockIdx.x * kGroup + (threadIdx.x & 1) * 64;
    float m = 0.f;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        raw[i].zero();
        if (r < n && c + i * kE < k) raw[i].load(w + r * k + c + i * kE);
        float v[kE];
        raw[i].to_f(v);
#pragma unroll
        for (int j = 0; j < kE; ++j) m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
    if ((threadIdx.x & 31) == 0) mx[threadIdx.x >> 5] = m;
    __syncthreads();
    m = mx[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, mx[i]);
    m = fmaxf(m, kAmaxFloor);
    const Quotient by(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r >= n || c + i * kE >= k) continue;
        float v[kE];
        raw[i].to_f(v);
        by(v);
        *reinterpret_cast<uint2*>(q + r * k + c + i * kE) = to_e4m3(v);
    }
    if (threadIdx.x == 0) scales[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = m / kE4m3Max;
}

// Threads of a CTA for `vectors` vectors at V a thread (whole warps).
int threads_for(int64_t vectors, int V) {
    return (int)std::max<int64_t>(32, ((vectors + V - 1) / V + 31) / 32 * 32);
}

template <typename Tx, typename Tr, typename Tout, bool ALIGNED, bool FP8>
cudaError_t norm_v(const NParams& p, cudaStream_t s) {
    // a row's vectors: one more where it may begin inside a vector
    const int64_t vectors = ALIGNED ? p.dim / kE : p.dim / kE + 2;
    const unsigned grid = (unsigned)p.rows;
    const unsigned alone = (unsigned)((p.rows + kAloneWarps - 1) / kAloneWarps);
    // A warp per row up to three vectors a lane, a CTA per row beyond: the training step (16001,
    // 768) bf16 takes 49.5 us with warps, 56.6 with CTAs of 64 threads.
    if (vectors <= 32)
        norm_kernel<Tx, Tr, Tout, 1, ALIGNED, FP8, true><<<alone, 32 * kAloneWarps, 0, s>>>(p);
    else if (vectors <= 64)
        norm_kernel<Tx, Tr, Tout, 2, ALIGNED, FP8, true><<<alone, 32 * kAloneWarps, 0, s>>>(p);
    else if (vectors <= 96)
        norm_kernel<Tx, Tr, Tout, 3, ALIGNED, FP8, true><<<alone, 32 * kAloneWarps, 0, s>>>(p);
    else if (vectors <= 2 * kMaxThreads)
        norm_kernel<Tx, Tr, Tout, 2, ALIGNED, FP8, false><<<grid, threads_for(vectors, 2), 0, s>>>(p);
    else {
        constexpr int V = ALIGNED ? 4 : 5;
        norm_kernel<Tx, Tr, Tout, V, ALIGNED, FP8, false><<<grid, threads_for(vectors, V), 0, s>>>(p);
    }
    return cudaGetLastError();
}
template <typename Tx, typename Tr>
cudaError_t norm_t(const NParams& p, DType out, cudaStream_t s) {
    if (p.scales) return norm_v<Tx, Tr, float, true, true>(p, s);
    if (p.dim % kE == 0)
        return out == DType::BF16 ? norm_v<Tx, Tr, __nv_bfloat16, true, false>(p, s)
                                  : norm_v<Tx, Tr, float, true, false>(p, s);
    return out == DType::BF16 ? norm_v<Tx, Tr, __nv_bfloat16, false, false>(p, s)
                              : norm_v<Tx, Tr, float, false, false>(p, s);
}

template <typename Tx, typename Tr>
cudaError_t norm_bwd_t(const BNParams& p, cudaStream_t s) {
    const unsigned grid = (unsigned)norm_bwd_blocks(p.rows, p.dim);
    const int64_t vectors = p.dim / kE;
    const size_t weights = (size_t)p.dim * 4;
    if (p.dim % kE != 0) {
        const auto threads = [&](int C) { return (unsigned)(((p.dim + C - 1) / C + 31) / 32 * 32); };
        if (p.dim <= 4 * kMaxThreads) norm_bwd_elem_kernel<Tx, Tr, 4><<<grid, threads(4), 0, s>>>(p);
        else if (p.dim <= 8 * kMaxThreads) norm_bwd_elem_kernel<Tx, Tr, 8><<<grid, threads(8), 0, s>>>(p);
        else norm_bwd_elem_kernel<Tx, Tr, 32><<<grid, threads(32), 0, s>>>(p);
    } else if (vectors <= 32)
        norm_bwd_kernel<Tx, Tr, 1, true><<<grid, 32 * kAloneWarps, weights, s>>>(p);
    else if (vectors <= 64)
        norm_bwd_kernel<Tx, Tr, 2, true><<<grid, 32 * kAloneWarps, weights, s>>>(p);
    else if (vectors <= 96)
        norm_bwd_kernel<Tx, Tr, 3, true><<<grid, 32 * kAloneWarps, weights, s>>>(p);
    else if (vectors <= kMaxThreads)
        norm_bwd_kernel<Tx, Tr, 1, false><<<grid, threads_for(vectors, 1), weights, s>>>(p);
    else if (vectors <= 2 * kMaxThreads)
        norm_bwd_kernel<Tx, Tr, 2, false><<<grid, threads_for(vectors, 2), weights, s>>>(p);
    else {
        const cudaError_t e = cudaFuncSetAttribute(norm_bwd_kernel<Tx, Tr, 4, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxDim * 4);
        if (e != cudaSuccess) return e;
        norm_bwd_kernel<Tx, Tr, 4, false><<<grid, threads_for(vectors, 4), weights, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename T>
void quantize_rows(const QuantArgs& a, int64_t rows, cudaStream_t s) {
    const T* x = static_cast<const T*>(a.x);
    uint8_t* q = static_cast<uint8_t*>(a.q);
    const unsigned grid = (unsigned)((rows * ((a.dim + kGroup - 1) / kGroup) + 16 * kBatch - 1) / (16 * kBatch));
    if (a.dim % kGroup == 0) quantize_kernel<T, true><<<grid, 256, 0, s>>>(x, q, a.scales, rows, a.dim);
    else quantize_kernel<T, false><<<grid, 256, 0, s>>>(x, q, a.scales, rows, a.dim);
}

template <typename T>
void quantize_cm(const QuantArgs& a, dim3 grid, cudaStream_t s) {
    const T* x = static_cast<const T*>(a.x);
    uint8_t* q = static_cast<uint8_t*>(a.q);
    const int64_t total = a.batch * a.dim * a.seqlen;
    if (a.seqlen % (16 / (int64_t)sizeof(T)) == 0)
        quantize_cm_kernel<T, true><<<grid, 256, 0, s>>>(x, q, a.scales, a.dim, a.seqlen, total);
    else
        quantize_cm_kernel<T, false><<<grid, 256, 0, s>>>(x, q, a.scales, a.dim, a.seqlen, total);
}

}  // namespace

int64_t norm_bwd_blocks(int64_t rows, int64_t dim) {
    if (dim % kE == 0 && dim <= 96 * kE)  // a warp per row
        return std::max<int64_t>(1, std::min<int64_t>((rows + kAloneWarps - 1) / kAloneWarps, 148 * 2));
    return std::max<int64_t>(1, std::min<int64_t>(rows, 148 * (dim <= 4096 ? 4 : 2)));
}

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    const NParams p{a.x, a.residual, a.weight, a.out, a.scales, a.residual_out, a.rows, a.dim, a.eps};
    if (a.x_dtype == DType::BF16)
        return a.res_dtype == DType::BF16 ? norm_t<__nv_bfloat16, __nv_bfloat16>(p, a.out_dtype, s)
                                          : norm_t<__nv_bfloat16, float>(p, a.out_dtype, s);
    return a.res_dtype == DType::BF16 ? norm_t<float, __nv_bfloat16>(p, a.out_dtype, s)
                                      : norm_t<float, float>(p, a.out_dtype, s);
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    if (a.rows == 0) return cudaMemsetAsync(a.dweight, 0, (size_t)a.dim * 4, s);
    const BNParams p{a.dout, a.stream_in, a.weight, a.dstream, a.dx, a.dresidual, a.part,
                     a.rows, a.dim, a.eps};
    cudaError_t e;
    if (a.x_dtype == DType::BF16)
        e = a.res_dtype == DType::BF16 ? norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, s)
                                       : norm_bwd_t<__nv_bfloat16, float>(p, s);
    else
        e = a.res_dtype == DType::BF16 ? norm_bwd_t<float, __nv_bfloat16>(p, s)
                                       : norm_bwd_t<float, float>(p, s);
    if (e != cudaSuccess) return e;
    // Launched while the backward's last CTAs run (it waits for them before it reads): the training step
    // (16001, 768) bf16 43.0 -> 41.1 us.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.dim + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, dweight_kernel, (const float*)a.part, a.dweight,
                              norm_bwd_blocks(a.rows, a.dim), a.dim);
}

cudaError_t launch_fp8_quantize(const QuantArgs& a, cudaStream_t s) {
    const int64_t rows = a.batch * a.seqlen;
    if (rows == 0) return cudaSuccess;
    const int64_t groups = (a.dim + kGroup - 1) / kGroup;
    if (!a.channel_major) {
        if (a.dtype == DType::BF16) quantize_rows<__nv_bfloat16>(a, rows, s);
        else quantize_rows<float>(a, rows, s);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)((a.seqlen + kTok - 1) / kTok), (unsigned)groups, (unsigned)a.batch);
    if (a.dtype == DType::BF16) quantize_cm<__nv_bfloat16>(a, grid, s);
    else quantize_cm<float>(a, grid, s);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_weight(const QuantWeightArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)((a.k + kGroup - 1) / kGroup), (unsigned)((a.n + kGroup - 1) / kGroup));
    uint8_t* q = static_cast<uint8_t*>(a.q);
    if (a.dtype == DType::BF16)
        quantize_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(a.w), q, a.scales, a.n, a.k);
    else
        quantize_weight_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(a.w), q, a.scales, a.n, a.k);
    return cudaGetLastError();
}

}  // namespace s6
