// api_layer.cu -- the extern "C" boundary of the operators around the scan (gated linear
// recurrence, residual addition with RMS norm, e4m3 quantisation, 8-bit projection), as
// declared in include/mamba_s6.h.  Host-side only: every argument is checked before anything
// is enqueued; no allocation, no synchronisation, no state kept between calls.
#include <initializer_list>
#include <stdint.h>

#include "../../include/mamba_s6.h"
#include "layer_launch.h"

namespace {

constexpr int64_t kGroup = 128;

bool dtype_ok(int dt) { return dt == MAMBA_F32 || dt == MAMBA_BF16; }
s6::DType to_dtype(int dt) { return dt == MAMBA_BF16 ? s6::DType::BF16 : s6::DType::F32; }
int cuda_status(cudaError_t e) { return s6::taken(e) == cudaSuccess ? MAMBA_OK : MAMBA_ERR_CUDA; }

bool all_aligned(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
    return true;
}

// a * b * c elements of up to 8 bytes are addressable (all sizes non-negative).
bool fits(int64_t a, int64_t b, int64_t c) {
    constexpr int64_t kMost = INT64_MAX / 16;
    if (a < 0 || b < 0 || c < 0) return false;
    if (a == 0 || b == 0 || c == 0) return true;
    return b <= kMost / a && c <= kMost / a / b;
}

constexpr int64_t kMaxBlocks = 0x7fffffff;

constexpr int64_t kMaxSteps = (int64_t)1 << 38;  // a row's chunks are counted in 32 bits

bool gated_dims_ok(const mamba_gated_dims& d) {
    if (d.batch < 1 || d.dim < 1 || d.seqlen < 0 || d.seqlen > kMaxSteps || !fits(d.batch, d.dim, d.seqlen + 512)) return false;
    return d.batch * d.dim <= kMaxBlocks / 8;  // CTAs of a launch
}

int64_t round256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

// Partial sums of the bias' gradient: one per row and CTA of the team that walks it.
int64_t bias_bytes(const mamba_gated_dims& d) {
    const int64_t rows = d.batch * d.dim;
    return round256(rows * s6::gated_team(rows, d.seqlen, true).ctas * 4);
}

}  // namespace

extern "C" {

size_t mamba_gated_scan_checkpoints_size(mamba_gated_dims dims) {
    if (!gated_dims_ok(dims)) return 0;
    return (size_t)round256(dims.batch * dims.dim * s6::gated_chunks(dims.seqlen) * 4);
}

size_t mamba_gated_scan_bwd_workspace_size(mamba_gated_dims dims) {
    if (!gated_dims_ok(dims) || dims.seqlen == 0) return 0;
    return (size_t)bias_bytes(dims) + mamba_gated_scan_checkpoints_size(dims);
}

int mamba_diag_gated_team(mamba_gated_dims dims, int backward, int* warps, int* ctas) {
    if (!warps || !ctas) return MAMBA_ERR_NULL;
    if (!gated_dims_ok(dims)) return MAMBA_ERR_DIMS;
    const s6::GatedTeam t = s6::gated_team(dims.batch * dims.dim, dims.seqlen, backward != 0);
    *warps = t.warps;
    *ctas = t.ctas;
    return MAMBA_OK;
}

int mamba_gated_scan_fwd(const void* x, const void* gate, const float* gate_bias, const void* z,
                         const float* initial_state, void* y, float* last_state,
                         float* checkpoints, size_t checkpoint_bytes, mamba_gated_dims dims,
                         mamba_dtype in_dtype, mamba_dtype out_dtype, unsigned flags, void* stream) {
    if (flags & ~MAMBA_FLAG_GIVEN_DECAY) return MAMBA_ERR_FLAGS;
    if (dims.seqlen != 0 && (!x || !gate || !y)) return MAMBA_ERR_NULL;
    if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
    if (!gated_dims_ok(dims)) return MAMBA_ERR_DIMS;
    if (!all_aligned({x, gate, gate_bias, z, initial_state, y, last_state, checkpoints}))
        return MAMBA_ERR_ALIGN;
    if (checkpoints && checkpoint_bytes < mamba_gated_scan_checkpoints_size(dims))
        return MAMBA_ERR_WORKSPACE;
    s6::GatedArgs a{};
    a.x = x;
    a.gate = gate;
    a.gate_bias = gate_bias;
    a.z = z;
    a.h0 = initial_state;
    a.y = y;
    a.last_state = last_state;
    a.ckpt = checkpoints;
    a.rows = dims.batch * dims.dim;
    a.dim = dims.dim;
    a.L = dims.seqlen;
    a.given_decay = (flags & MAMBA_FLAG_GIVEN_DECAY) ? 1 : 0;
    a.in_dtype = to_dtype(in_dtype);
    a.out_dtype = to_dtype(out_dtype);
    return cuda_status(s6::launch_gated_scan(a, static_cast<cudaStream_t>(stream)));
}

int mamba_gated_scan_bwd(const void* x, const void* gate, const float* gate_bias, const void* z,
                         const float* initial_state, const void* dy, const float* dlast_state,
                         void* dx, void* dgate, void* dz, float* dgate_bias,
                         float* dinitial_state, const float* checkpoints, size_t checkpoint_bytes,
                         mamba_gated_dims dims, mamba_dtype dtype, void* workspace,
                         size_t workspace_bytes, unsigned flags, void* stream) {
    if (flags & ~MAMBA_FLAG_GIVEN_DECAY) return MAMBA_ERR_FLAGS;
    const bool decay = (flags & MAMBA_FLAG_GIVEN_DECAY) != 0, empty = dims.seqlen == 0;
    if (!empty && (!x || !gate || !dy || !dx || !dgate)) return MAMBA_ERR_NULL;
    if (!empty && (z == nullptr) != (dz == nullptr)) return MAMBA_ERR_NULL;
    // the gradient of the bias is present exactly when the bias is, and it has one in the
    // sigmoid form alone
    if ((gate_bias == nullptr || decay) != (dgate_bias == nullptr)) return MAMBA_ERR_NULL;
    if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
    if (!gated_dims_ok(dims)) return MAMBA_ERR_DIMS;
    if (!all_aligned({x, gate, gate_bias, z, initial_state, dy, dlast_state, dx, dgate, dz, dgate_bias,
                      dinitial_state, checkpoints, workspace}))
        return MAMBA_ERR_ALIGN;
    const size_t ck_bytes = mamba_gated_scan_checkpoints_size(dims);
    if (checkpoints && checkpoint_bytes < ck_bytes) return MAMBA_ERR_WORKSPACE;
    const size_t need = mamba_gated_scan_bwd_workspace_size(dims);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    s6::GatedArgs a{};
    a.x = x;
    a.gate = gate;
    a.gate_bias = gate_bias;
    a.h0 = initial_state;
    a.rows = dims.batch * dims.dim;
    a.dim = dims.dim;
    a.L = dims.seqlen;
    a.given_decay = decay ? 1 : 0;
    a.in_dtype = a.out_dtype = to_dtype(dtype);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (checkpoints || empty) {
        a.ckpt = const_cast<float*>(checkpoints);
    } else {  // the states entering every chunk, by a forward pass without outputs
        a.ckpt = reinterpret_cast<float*>(ws + bias_bytes(dims));
        const cudaError_t e = s6::launch_gated_scan(a, st);
        if (e != cudaSuccess) return cuda_status(e);
    }
    a.z = z;
    s6::GatedBwdArgs g{};
    g.dy = dy;
    g.dlast = dlast_state;
    g.dx = dx;
    g.dgate = dgate;
    g.dz = dz;
    g.dbias = dgate_bias;
    g.dh0 = dinitial_state;
    g.bias_part = reinterpret_cast<float*>(ws);
    return cuda_status(s6::launch_gated_scan_bwd(a, g, st));
}

int mamba_gated_state_update(float* state, const void* x, const void* gate, const float* gate_bias,
                             const void* z, void* y, int64_t batch, int64_t dim,
                             mamba_dtype dtype, unsigned flags, void* stream) {
    if (flags & ~MAMBA_FLAG_GIVEN_DECAY) return MAMBA_ERR_FLAGS;
    if (!state || !x || !gate || !y) return MAMBA_ERR_NULL;
    if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
    if (batch < 1 || dim < 1 || !fits(batch, dim, 1) || batch * dim / 128 >= kMaxBlocks)
        return MAMBA_ERR_DIMS;
    if (!all_aligned({state, x, gate, gate_bias, z, y})) return MAMBA_ERR_ALIGN;
    s6::GatedUpdateArgs a{state, x, gate, gate_bias, z, y, batch, dim,
                          (flags & MAMBA_FLAG_GIVEN_DECAY) ? 1 : 0, to_dtype(dtype)};
    return cuda_status(s6::launch_gated_update(a, static_cast<cudaStream_t>(stream)));
}

static int norm_check(int64_t rows, int64_t dim, bool fp8) {
    if (rows < 0 || rows > kMaxBlocks || dim < 1 || dim > s6::kNormMaxDim || !fits(rows, dim, 1))
        return MAMBA_ERR_DIMS;
    return fp8 && dim % 16 != 0 ? MAMBA_ERR_DIMS : MAMBA_OK;
}

int mamba_add_rms_norm_fwd(const void* x, const void* residual, const float* weight, float eps,
                           void* out, void* residual_out, int64_t rows, int64_t dim,
                           mamba_dtype x_dtype, mamba_dtype residual_dtype, mamba_dtype out_dtype,
                           void* stream) {
    if (!weight || (rows > 0 && (!x || !out || (residual && !residual_out)))) return MAMBA_ERR_NULL;
    if (!dtype_ok(x_dtype) || !dtype_ok(residual_dtype) || !dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
    const int rc = norm_check(rows, dim, false);
    if (rc != MAMBA_OK) return rc;
    if (!all_aligned({x, residual, weight, out, residual_out})) return MAMBA_ERR_ALIGN;
    s6::NormArgs a{x, residual, weight, out, nullptr, residual_out, rows, dim, eps,
                   to_dtype(x_dtype), to_dtype(residual ? residual_dtype : x_dtype), to_dtype(out_dtype)};
    return cuda_status(s6::launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

int mamba_add_rms_norm_fp8(const void* x, const void* residual, const float* weight, float eps,
                           void* q, float* scales, void* residual_out, int64_t rows, int64_t dim,
                           mamba_dtype x_dtype, mamba_dtype residual_dtype, void* stream) {
    if (!weight || (rows > 0 && (!x || !q || !scales || (residual && !residual_out))))
        return MAMBA_ERR_NULL;
    if (!dtype_ok(x_dtype) || !dtype_ok(residual_dtype)) return MAMBA_ERR_DTYPE;
    const int rc = norm_check(rows, dim, true);
    if (rc != MAMBA_OK) return rc;
    if (!all_aligned({x, residual, weight, q, scales, residual_out})) return MAMBA_ERR_ALIGN;
    s6::NormArgs a{x, residual, weight, q, scales, residual_out, rows, dim, eps,
                   to_dtype(x_dtype), to_dtype(residual ? residual_dtype : x_dtype), s6::DType::F32};
    return cuda_status(s6::launch_rms_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t mamba_add_rms_norm_bwd_workspace_size(int64_t rows, int64_t dim) {
    if (norm_check(rows, dim, false) != MAMBA_OK || rows == 0) return 0;
    return (size_t)round256(s6::norm_bwd_blocks(rows, dim) * dim * 4);
}

int mamba_add_rms_norm_bwd(const void* dout, const void* residual_out, const float* weight,
                           const void* dresidual_out, float eps, void* dx, void* dresidual,
                           float* dweight, int64_t rows, int64_t dim, mamba_dtype x_dtype,
                           mamba_dtype residual_dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
    if (!weight || !dweight || (rows > 0 && (!dout || !residual_out || !dx))) return MAMBA_ERR_NULL;
    if (!dtype_ok(x_dtype) || !dtype_ok(residual_dtype)) return MAMBA_ERR_DTYPE;
    const int rc = norm_check(rows, dim, false);
    if (rc != MAMBA_OK) return rc;
    if (!all_aligned({dout, residual_out, weight, dresidual_out, dx, dresidual, dweight, workspace}))
        return MAMBA_ERR_ALIGN;
    const size_t need = mamba_add_rms_norm_bwd_workspace_size(rows, dim);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
    s6::NormBwdArgs a{dout, residual_out, weight, dresidual_out, dx, dresidual, dweight,
                      static_cast<float*>(workspace), rows, dim, eps, to_dtype(x_dtype),
                      to_dtype(residual_dtype)};
    return cuda_status(s6::launch_rms_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

int mamba_fp8_quantize(const void* x, void* q, float* scales, int64_t batch, int64_t dim,
                       int64_t seqlen, int channel_major, mamba_dtype dtype, void* stream) {
    if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
    if (dim < 16 || dim % 16 != 0 || !fits(batch, dim, seqlen) || !fits(batch, dim + kGroup, seqlen) ||
        batch * seqlen * (dim + kGroup) / 2048 >= kMaxBlocks)
        return MAMBA_ERR_DIMS;
    if (batch * seqlen != 0 && (!x || !q || !scales)) return MAMBA_ERR_NULL;
    if (channel_major && (batch > 65535 || dim / kGroup >= 65535)) return MAMBA_ERR_DIMS;
    if (!all_aligned({x, q, scales})) return MAMBA_ERR_ALIGN;
    s6::QuantArgs a{x, q, scales, batch, dim, seqlen, channel_major ? 1 : 0, to_dtype(dtype)};
    return cuda_status(s6::launch_fp8_quantize(a, static_cast<cudaStream_t>(stream)));
}

int mamba_fp8_quantize_weight(const void* w, void* q, float* scales, int64_t n, int64_t k,
                              mamba_dtype dtype, void* stream) {
    if (!w || !q || !scales) return MAMBA_ERR_NULL;
    if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
    if (n < 1 || k < 16 || k % 16 != 0 || !fits(n, k, 1) || n / kGroup >= 65535 || k / kGroup >= kMaxBlocks)
        return MAMBA_ERR_DIMS;
    if (!all_aligned({w, q, scales})) return MAMBA_ERR_ALIGN;
    s6::QuantWeightArgs a{w, q, scales, n, k, to_dtype(dtype)};
    return cuda_status(s6::launch_fp8_quantize_weight(a, static_cast<cudaStream_t>(stream)));
}

int mamba_fp8_linear(const void* xq, const float* x_scales, const void* wq, const float* w_scales,
                     void* out, int64_t tokens, int64_t n, int64_t k, int64_t seqlen,
                     mamba_dtype out_dtype, void* stream) {
    if (!wq || !w_scales || (tokens > 0 && (!xq || !x_scales || !out))) return MAMBA_ERR_NULL;
    if (!dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
    constexpr int64_t kMost = 0x7fffff00;  // rows and inputs are 32-bit tile coordinates
    if (tokens < 0 || n < 1 || k < 16 || k % 16 != 0 || seqlen < 0 || tokens > kMost || n > kMost ||
        k > kMost || !fits(tokens, n, 4) || !fits(tokens, k, 1) || !fits(n, k, 1) ||
        (seqlen > 0 && tokens % seqlen != 0) ||
        ((tokens + 127) / 128) * ((n + 255) / 256) > kMost)
        return MAMBA_ERR_DIMS;
    if (!all_aligned({xq, x_scales, wq, w_scales, out})) return MAMBA_ERR_ALIGN;
    s6::LinearArgs a{xq, x_scales, wq, w_scales, out, tokens, n, k, seqlen, to_dtype(out_dtype)};
    return cuda_status(s6::launch_fp8_linear(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
