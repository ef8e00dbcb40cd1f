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

// Sum of one value (or two) over the CTA, the same bits in every thread.
__device__ __forceinline__ float2 cta_sum2(float2 v, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(kFull, v.x, o);
        v.y += __shfl_xor_sync(kFull, v.y, o);
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
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
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) o[j] = (c + j >= 0 && c + j < dim) ? __ldg(w + c + j) : 0.f;
    }
}

// One CTA per row, V vectors of 8 per thread.  ALIGNED: dim is a multiple of 8.  OUT: the
// output's type; FP8 writes e4m3 and a scale per 128 columns (dim is a multiple of 16 then):
// 16 lanes hold the 128 columns of a group, and its largest magnitude is their shuffled maximum.
template <typename Tx, typename Tr, typename Tout, int V, bool ALIGNED, bool FP8>
__global__ void __launch_bounds__(kMaxThreads) norm_kernel(const NParams p) {
    __shared__ float2 red[kMaxThreads / 32];
    const Row w = row_of(blockIdx.x, p.rows, p.dim);
    float v[V][kE];
    Raw8<Tx> xr[V];
    Raw8<Tr> rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + ((int64_t)i * blockDim.x + threadIdx.x) * kE;
        fetch<Tx>(xr[i], p.x, e, w);
        if (p.res) fetch<Tr>(rr[i], p.res, e, w);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + ((int64_t)i * blockDim.x + threadIdx.x) * kE;
        xr[i].to_f(v[i]);
        if (p.res) {
            float r[kE];
            rr[i].to_f(r);
#pragma unroll
            for (int j = 0; j < kE; ++j) v[i][j] = io<Tr>::to_f(io<Tr>::from_f(v[i][j] + r[j]));
        }
        if (!ALIGNED) {
#pragma unroll
            for (int j = 0; j < kE; ++j)
                if (e + j < w.lo || e + j >= w.hi) v[i][j] = 0.f;
        }
        if (p.res_out) put<Tr>(p.res_out, e, w, v[i]);
#pragma unroll
        for (int j = 0; j < kE; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    const float2 t = cta_sum2(make_float2(ss, 0.f), red);
    const float rstd = rsqrtf(t.x / (float)p.dim + p.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t e = w.base + ((int64_t)i * blockDim.x + threadIdx.x) * kE;
        const bool in = e < w.hi;
        float o[kE] = {};
        if (in) {
            float wt[kE];
            weights8<ALIGNED>(p.w, e - w.lo, p.dim, wt);
#pragma unroll
            for (int j = 0; j < kE; ++j) o[j] = v[i][j] * rstd * wt[j];
        }
        if (FP8) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < kE; ++j) m = fmaxf(m, fabsf(o[j]));
#pragma unroll
            for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
            m = fmaxf(m, kAmaxFloor);
            if (in) {
                const float inv = kE4m3Max / m;
#pragma unroll
                for (int j = 0; j < kE; ++j) o[j] *= inv;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + e) = to_e4m3(o);
                const int64_t c = e - w.lo, groups = (p.dim + kGroup - 1) / kGroup;
                if (c % kGroup == 0)
                    p.scales[blockIdx.x * groups + c / kGroup] = m / kE4m3Max;
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

// CTAs walk rows with the grid's stride and keep their share of dweight in registers; the
// shares are summed by dweight_kernel in a fixed order (no atomics: the same call gives the
// same bits).  A thread's columns are the same in every row only when rows begin at vector
// boundaries; otherwise (dim not a multiple of 8) a thread takes single columns.
template <typename Tx, typename Tr, int V>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_kernel(const BNParams p) {
    __shared__ float2 red[2][kMaxThreads / 32];
    float dw[V][kE], wt[V][kE];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * kE;
#pragma unroll
        for (int j = 0; j < kE; ++j) dw[i][j] = 0.f, wt[i][j] = 0.f;
        if (c < p.dim) weights8<true>(p.w, c, p.dim, wt[i]);
    }
    int flip = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1) {
        const Row w = row_of(r, p.rows, p.dim);
        Raw8<Tx> gr[V];
        Raw8<Tr> sr[V], dr[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t e = w.base + ((int64_t)i * blockDim.x + threadIdx.x) * kE;
            fetch<Tr>(sr[i], p.s, e, w);
            fetch<Tx>(gr[i], p.dout, e, w);
            if (p.ds) fetch<Tr>(dr[i], p.ds, e, w);
        }
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float v[kE], g[kE];
            sr[i].to_f(v);
            gr[i].to_f(g);
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                sum.x = fmaf(v[j], v[j], sum.x);
                sum.y = fmaf(g[j] * wt[i][j], v[j], sum.y);
            }
        }
        sum = cta_sum2(sum, red[flip]);
        const float rstd = rsqrtf(sum.x / (float)p.dim + p.eps);
        const float k = sum.y / (float)p.dim * rstd * rstd;  // mean(g xhat) rstd
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int64_t e = w.base + ((int64_t)i * blockDim.x + threadIdx.x) * kE;
            if (e >= w.hi) continue;
            float v[kE], g[kE], d[kE];
            sr[i].to_f(v);
            gr[i].to_f(g);
            if (p.ds) {
                dr[i].to_f(d);
            } else {
#pragma unroll
                for (int j = 0; j < kE; ++j) d[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                dw[i][j] = fmaf(g[j], v[j] * rstd, dw[i][j]);
                d[j] = fmaf(rstd, fmaf(-k, v[j], g[j] * wt[i][j]), d[j]);
            }
            put<Tx>(p.dx, e, w, d);
            if (p.dres) put<Tr>(p.dres, e, w, d);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t c = ((int64_t)i * blockDim.x + threadIdx.x) * kE;
        if (c < p.dim) store_all(p.part + (int64_t)blockIdx.x * p.dim + c, dw[i]);
    }
}

// The same for any dim: a thread takes columns threadIdx.x + i blockDim.x, and dweight's share
// goes through its row of `part` in memory.
template <typename Tx, typename Tr>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_elem_kernel(const BNParams p) {
    __shared__ float2 red[2][kMaxThreads / 32];
    float* part = p.part + (int64_t)blockIdx.x * p.dim;
    const Tx* dout = static_cast<const Tx*>(p.dout);
    const Tr *st = static_cast<const Tr*>(p.s), *ds = static_cast<const Tr*>(p.ds);
    int flip = 0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x, flip ^= 1) {
        float2 sum = make_float2(0.f, 0.f);
        for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) {
            const float v = io<Tr>::to_f(st[r * p.dim + c]);
            const float g = io<Tx>::to_f(dout[r * p.dim + c]) * __ldg(p.w + c);
            sum.x = fmaf(v, v, sum.x);
            sum.y = fmaf(g, v, sum.y);
        }
        sum = cta_sum2(sum, red[flip]);
        const float rstd = rsqrtf(sum.x / (float)p.dim + p.eps);
        const float k = sum.y / (float)p.dim * rstd * rstd;
        for (int64_t c = threadIdx.x; c < p.dim; c += blockDim.x) {
            const float v = io<Tr>::to_f(st[r * p.dim + c]), g = io<Tx>::to_f(dout[r * p.dim + c]);
            const float d = fmaf(rstd, fmaf(-k, v, g * __ldg(p.w + c)),
                                 ds ? io<Tr>::to_f(ds[r * p.dim + c]) : 0.f);
            const float dw = g * (v * rstd);
            part[c] = r == blockIdx.x ? dw : part[c] + dw;
            static_cast<Tx*>(p.dx)[r * p.dim + c] = io<Tx>::from_f(d);
            if (p.dres) static_cast<Tr*>(p.dres)[r * p.dim + c] = io<Tr>::from_f(d);
        }
    }
}

// Columns' sums of part (blocks, dim): 8 columns per CTA, 32 rows side by side.
__global__ void __launch_bounds__(256) dweight_kernel(const float* part, float* dw, int64_t blocks,
                                                      int64_t dim) {
    __shared__ float red[32][9];
    const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
    const int64_t c = (int64_t)blockIdx.x * 8 + cx;
    float v = 0.f;
    if (c < dim)
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

// Row-major: a thread takes 8 values, 16 lanes a group of 128; rows are padded to whole groups
// in the thread numbering only.
template <typename T>
__global__ void __launch_bounds__(256) quantize_kernel(const T* x, uint8_t* q, float* scales,
                                                       int64_t rows, int64_t dim) {
    const int64_t groups = (dim + kGroup - 1) / kGroup;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t gi = i >> 4;  // (row, group)
    const int64_t r = gi / groups, c = (gi - r * groups) * kGroup + (i & 15) * kE;
    const bool in = r < rows && c < dim;
    float v[kE] = {};
    if (in) {
        Raw8<T> raw;
        raw.load(x + r * dim + c);
        raw.to_f(v);
    }
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < kE; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
    m = fmaxf(m, kAmaxFloor);
    if (!in) return;
    const float inv = kE4m3Max / m;
#pragma unroll
    for (int j = 0; j < kE; ++j) v[j] *= inv;
    *reinterpret_cast<uint2*>(q + r * dim + c) = to_e4m3(v);
    if ((i & 15) == 0) scales[gi] = m / kE4m3Max;
}

// Channel-major (batch, dim, L) to token rows (batch * L, dim): a CTA takes 128 channels of 64
// tokens through shared memory, read along the tokens and written along the channels.  Thread
// (token, quarter) holds 32 channels of its token, so a token's 128 values are 4 threads'.
constexpr int kTok = 64;
template <typename T>
__global__ void __launch_bounds__(256) quantize_cm_kernel(const T* x, uint8_t* q, float* scales,
                                                          int64_t dim, int64_t L) {
    constexpr int kPad = 16 / sizeof(T);  // rows stay 16-byte aligned
    __shared__ alignas(16) T tile[kGroup][kTok + kPad];
    __shared__ float mx[4][kTok];
    const int64_t t0 = (int64_t)blockIdx.x * kTok, c0 = (int64_t)blockIdx.y * kGroup,
                  b = blockIdx.z;
    const int nc = (int)min((int64_t)kGroup, dim - c0), nt = (int)min((int64_t)kTok, L - t0);
    const T* src = x + (b * dim + c0) * L + t0;
    if (L % kPad == 0) {
        constexpr int kVecs = kTok / kPad;
        for (int i = threadIdx.x; i < kGroup * kVecs; i += 256) {
            const int c = i / kVecs, t = (i % kVecs) * kPad;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (c < nc && t < nt) v = *reinterpret_cast<const uint4*>(src + (int64_t)c * L + t);
            *reinterpret_cast<uint4*>(&tile[c][t]) = v;
        }
    } else {
        for (int i = threadIdx.x; i < kGroup * kTok; i += 256) {
            const int c = i / kTok, t = i % kTok;
            tile[c][t] = (c < nc && t < nt) ? src[(int64_t)c * L + t] : io<T>::from_f(0.f);
        }
    }
    __syncthreads();
    const int t = threadIdx.x % kTok, part = threadIdx.x / kTok;
    float v[4][kE], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            v[i][j] = io<T>::to_f(tile[part * 32 + i * kE + j][t]);
            m = fmaxf(m, fabsf(v[i][j]));
        }
    mx[part][t] = m;
    __syncthreads();
    if (t >= nt) return;
    m = fmaxf(fmaxf(fmaxf(mx[0][t], mx[1][t]), fmaxf(mx[2][t], mx[3][t])), kAmaxFloor);
    const float inv = kE4m3Max / m;
    const int64_t row = b * L + t0 + t;
    uint8_t* dst = q + row * dim + c0 + part * 32;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        if (part * 32 + i * kE >= nc) break;
#pragma unroll
        for (int j = 0; j < kE; ++j) v[i][j] *= inv, v[i + 1][j] *= inv;
        const uint2 lo = to_e4m3(v[i]), hi = to_e4m3(v[i + 1]);
        *reinterpret_cast<uint4*>(dst + i * kE) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
    if (part == 0) scales[row * ((dim + kGroup - 1) / kGroup) + blockIdx.y] = m / kE4m3Max;
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
    const float inv = kE4m3Max / m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r >= n || c + i * kE >= k) continue;
        float v[kE];
        raw[i].to_f(v);
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] *= inv;
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
    if (vectors <= 2 * kMaxThreads)
        norm_kernel<Tx, Tr, Tout, 2, ALIGNED, FP8><<<grid, threads_for(vectors, 2), 0, s>>>(p);
    else {
        constexpr int V = ALIGNED ? 4 : 5;
        norm_kernel<Tx, Tr, Tout, V, ALIGNED, FP8><<<grid, threads_for(vectors, V), 0, s>>>(p);
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
    if (p.dim % kE != 0)
        norm_bwd_elem_kernel<Tx, Tr><<<grid, 256, 0, s>>>(p);
    else if (vectors <= 2 * kMaxThreads)
        norm_bwd_kernel<Tx, Tr, 2><<<grid, threads_for(vectors, 2), 0, s>>>(p);
    else
        norm_bwd_kernel<Tx, Tr, 4><<<grid, threads_for(vectors, 4), 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int64_t norm_bwd_blocks(int64_t rows, int64_t dim) {
    return std::max<int64_t>(1, std::min<int64_t>(rows, 148 * (dim <= 1024 ? 8 : dim <= 4096 ? 4 : 2)));
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
    dweight_kernel<<<(unsigned)((a.dim + 7) / 8), 256, 0, s>>>(a.part, a.dweight,
                                                              norm_bwd_blocks(a.rows, a.dim), a.dim);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quantize(const QuantArgs& a, cudaStream_t s) {
    const int64_t rows = a.batch * a.seqlen;
    if (rows == 0) return cudaSuccess;
    const int64_t groups = (a.dim + kGroup - 1) / kGroup;
    uint8_t* q = static_cast<uint8_t*>(a.q);
    if (!a.channel_major) {
        const unsigned grid = (unsigned)((rows * groups * 16 + 255) / 256);
        if (a.dtype == DType::BF16)
            quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(a.x), q, a.scales, rows, a.dim);
        else
            quantize_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(a.x), q, a.scales, rows, a.dim);
        return cudaGetLastError();
    }
    const dim3 grid((unsigned)((a.seqlen + kTok - 1) / kTok), (unsigned)groups, (unsigned)a.batch);
    if (a.dtype == DType::BF16)
        quantize_cm_kernel<<<grid, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(a.x), q, a.scales, a.dim, a.seqlen);
    else
        quantize_cm_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(a.x), q, a.scales, a.dim, a.seqlen);
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
