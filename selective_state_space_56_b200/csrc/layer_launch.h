// layer_launch.h -- internal (C++) launch interface of the layer operators around the scan:
// the gated linear recurrence, the residual addition with RMS norm, the quantisation to
// e4m3 and the 8-bit projection.  Arguments are already validated by the ABI layer.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "s6_launch.h"

namespace s6 {

// Elements one lane takes at a time, and one warp per step of its walk along a row.
constexpr int kGatedLane = 8;
constexpr int kGatedChunk = 32 * kGatedLane;

// Chunks a row of L elements can touch: chunks start at multiples of kGatedLane elements
// of the whole array, so a row may begin up to kGatedLane - 1 elements into its first one.
inline int64_t gated_chunks(int64_t L) {
    return L > 0 ? (L + (kGatedLane - 1) + (kGatedChunk - 1)) / kGatedChunk : 0;
}

// Warps of a CTA and CTAs of a cluster that walk a row together (1, 1: a warp by itself).
// Depends on the sizes alone.
struct GatedTeam {
    int warps, ctas;
};
GatedTeam gated_team(int64_t rows, int64_t L, bool backward);

struct GatedArgs {
    const void* x;     // (rows, L) in_dtype
    const void* gate;  // (rows, L) in_dtype
    const float* gate_bias;  // (dim) or null
    const void* z;           // (rows, L) in_dtype or null
    const float* h0;         // (rows) or null (zero)
    void* y;                 // (rows, L) out_dtype, or null (states only)
    float* last_state;       // (rows) or null
    float* ckpt;             // (rows, gated_chunks(L)) or null: the state entering each chunk
    int64_t rows, dim, L;
    int given_decay;
    DType in_dtype, out_dtype;
};

struct GatedBwdArgs {
    const void* dy;       // (rows, L) in_dtype
    const float* dlast;   // (rows) or null
    void* dx;             // (rows, L) in_dtype
    void* dgate;          // (rows, L) in_dtype
    void* dz;             // (rows, L) in_dtype, null without z
    float* dbias;         // (dim), null without a bias
    float* dh0;           // (rows) or null
    float* bias_part;     // (rows, CTAs of the backward's team) partial sums of dgate, when dbias
};

cudaError_t launch_gated_scan(const GatedArgs& a, cudaStream_t stream);
// a.ckpt holds the checkpoints already.
cudaError_t launch_gated_scan_bwd(const GatedArgs& a, const GatedBwdArgs& g, cudaStream_t stream);

// The recurrence's error word, as device_error_word.
cudaError_t gated_error_word(unsigned** word);
// One wait of limit_cycles on a barrier that nothing completes; sets that word.
cudaError_t launch_gated_timeout_probe(long long limit_cycles, cudaStream_t stream);

struct GatedUpdateArgs {
    float* state;  // (batch, dim), updated in place
    const void* x;
    const void* gate;
    const float* gate_bias;
    const void* z;
    void* y;
    int64_t batch, dim;
    int given_decay;
    DType dtype;
};
cudaError_t launch_gated_update(const GatedUpdateArgs& a, cudaStream_t stream);

struct NormArgs {
    const void* x;         // (rows, dim) x_dtype
    const void* residual;  // (rows, dim) res_dtype or null
    const float* weight;   // (dim)
    void* out;             // (rows, dim) out_dtype, or e4m3 when scales is given
    float* scales;         // (rows, ceil(dim / 128)) or null
    void* residual_out;    // (rows, dim) res_dtype or null
    int64_t rows, dim;
    float eps;
    DType x_dtype, res_dtype, out_dtype;
};
cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t stream);

struct NormBwdArgs {
    const void* dout;          // (rows, dim) x_dtype
    const void* stream_in;     // (rows, dim) res_dtype: what the forward normalised
    const float* weight;       // (dim)
    const void* dstream;       // (rows, dim) res_dtype or null: gradient of residual_out
    void* dx;                  // (rows, dim) x_dtype
    void* dresidual;           // (rows, dim) res_dtype or null
    float* dweight;            // (dim)
    float* part;               // workspace: (norm_bwd_blocks, dim)
    int64_t rows, dim;
    float eps;
    DType x_dtype, res_dtype;
};
// Rows of partial sums of dweight (one per CTA of the backward) for these sizes.
int64_t norm_bwd_blocks(int64_t rows, int64_t dim);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, cudaStream_t stream);
constexpr int64_t kNormMaxDim = 16384;  // a CTA keeps a row in registers

struct QuantArgs {
    const void* x;   // (batch * seqlen, dim), or (batch, dim, seqlen) when channel_major
    void* q;         // (batch * seqlen, dim) e4m3
    float* scales;   // (batch * seqlen, ceil(dim / 128))
    int64_t batch, dim, seqlen;
    int channel_major;
    DType dtype;
};
cudaError_t launch_fp8_quantize(const QuantArgs& a, cudaStream_t stream);

struct QuantWeightArgs {
    const void* w;   // (n, k)
    void* q;         // (n, k) e4m3
    float* scales;   // (ceil(n / 128), ceil(k / 128))
    int64_t n, k;
    DType dtype;
};
cudaError_t launch_fp8_quantize_weight(const QuantWeightArgs& a, cudaStream_t stream);

struct LinearArgs {
    const void* xq;    // (tokens, k) e4m3
    const float* xs;   // (tokens, ceil(k / 128))
    const void* wq;    // (n, k) e4m3
    const float* ws;   // (ceil(n / 128), ceil(k / 128))
    void* out;         // (tokens, n), or (tokens / seqlen, n, seqlen) when seqlen > 0
    int64_t tokens, n, k;
    int64_t seqlen;    // 0: token-major output
    DType out_dtype;
};
cudaError_t launch_fp8_linear(const LinearArgs& a, cudaStream_t stream);
// The projection's error word, as device_error_word.
cudaError_t linear_error_word(unsigned** word);
cudaError_t launch_linear_timeout_probe(long long limit_cycles, cudaStream_t stream);  // as for the recurrence

}  // namespace s6
