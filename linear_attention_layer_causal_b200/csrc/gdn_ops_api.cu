// gdn_ops_api.cu -- the C ABI of the state-space mixer, the norm with an 8-bit
// output and the 8-bit matrix product: host-side argument checks and launches.
// Every check runs before the first CUDA call.
#include <limits.h>
#include <math.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

gdn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

bool dtype_ok(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
int dtype_bytes(int32_t t) { return t == GDN_BF16 ? 2 : 4; }

gdn_status check_ssm_config(const gdn_ssm_config *c) {
    if (c == nullptr || c->num_groups < 1 || c->num_heads < 1 || c->head_dim < 1 || c->state_dim < 1 ||
        c->conv_kernel < 1 || c->num_heads % c->num_groups != 0 || !dtype_ok(c->act_dtype))
        return GDN_ERR_INVALID_ARG;
    if (!(c->dt_min >= 0.f) || !isfinite(c->dt_min) || !(c->dt_max >= c->dt_min))
        return GDN_ERR_INVALID_ARG;
    if (c->segments < 0 || c->segments > kMaxSegments)
        return GDN_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128) || (c->state_dim != 64 && c->state_dim != 128) ||
        c->conv_kernel != 4)
        return GDN_ERR_UNSUPPORTED;
    if (c->num_heads > 16384 || c->num_groups > 8192) // channels and grids index in int
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_ssm_params(const gdn_ssm_params *p) {
    if (p == nullptr || p->conv_w == nullptr || p->A_log == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned(p->conv_w, 16) || !aligned(p->conv_b, 16) || !aligned(p->A_log, 4) ||
        !aligned(p->dt_bias, 4) || !aligned(p->D, 4))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// The row inputs of prefill (rows = tokens) and decode (rows = sequences).
gdn_status check_ssm_rows(const gdn_ssm_config *c, const void *xbc, int64_t xbc_stride, const void *dt,
                          int64_t dt_stride, const void *z, int64_t z_stride, const void *y, int64_t rows) {
    if (rows == 0)
        return GDN_OK;
    const int el = dtype_bytes(c->act_dtype);
    const int64_t hp = (int64_t)c->num_heads * c->head_dim;
    const int64_t conv_dim = hp + 2 * (int64_t)c->num_groups * c->state_dim;
    if (xbc == nullptr || dt == nullptr || y == nullptr)
        return GDN_ERR_INVALID_ARG;
    if (!aligned(xbc, 16) || !aligned(z, 16) || !aligned(y, 16) || !aligned(dt, el))
        return GDN_ERR_INVALID_ARG;
    // rows < 2^31 and strides <= 2^31 keep every element offset within 62 bits
    if (xbc_stride < conv_dim || dt_stride < c->num_heads || (xbc_stride * el) % 16 != 0 ||
        xbc_stride > INT32_MAX || dt_stride > INT32_MAX)
        return GDN_ERR_INVALID_ARG;
    if (z != nullptr && (z_stride < hp || (z_stride * el) % 16 != 0 || z_stride > INT32_MAX))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

SsmArgs ssm_args(const gdn_ssm_config *c, const gdn_ssm_params *par, const void *xbc, int64_t xbc_stride,
                 const void *dt, int64_t dt_stride, const void *z, int64_t z_stride, int32_t batch, void *y) {
    SsmArgs p{};
    p.H = c->num_heads;
    p.G = c->num_groups;
    p.P = c->head_dim;
    p.S = c->state_dim;
    p.bf16 = c->act_dtype == GDN_BF16;
    p.dt_min = c->dt_min;
    p.dt_max = c->dt_max;
    p.xbc = xbc; p.dt = dt; p.z = z;
    p.xbc_stride = xbc_stride; p.dt_stride = dt_stride; p.z_stride = z_stride;
    p.batch = batch;
    p.y = y;
    p.conv_w = par->conv_w;
    p.conv_b = par->conv_b;
    p.A_log = par->A_log;
    p.dt_bias = par->dt_bias;
    p.D = par->D;
    return p;
}

} // namespace
} // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_ssm_prefill_workspace_size(const gdn_ssm_config *cfg, int32_t batch, int64_t total_tokens,
                                          size_t *bytes) {
    const gdn_status st = check_ssm_config(cfg);
    if (st != GDN_OK)
        return st;
    if (bytes == nullptr || batch < 0 || total_tokens < 0 || (batch == 0 && total_tokens > 0))
        return GDN_ERR_INVALID_ARG;
    if (batch > 65535 || total_tokens > INT32_MAX || !ssm_addressable(cfg, batch, total_tokens)) // cu_seqlens is int32
        return GDN_ERR_UNSUPPORTED;
    *bytes = ssm_workspace_bytes(cfg, batch, total_tokens);
    return GDN_OK;
}

gdn_status gdn_ssm_prefill(const gdn_ssm_config *cfg, const gdn_ssm_params *params, const void *xbc,
                           int64_t xbc_stride, const void *dt, int64_t dt_stride, const void *z,
                           int64_t z_stride, const int32_t *cu_seqlens, int32_t batch, int64_t total_tokens,
                           const float *initial_state, const void *initial_conv, void *y, float *final_state,
                           void *final_conv, void *workspace, size_t workspace_bytes, void *stream) {
    gdn_status st = check_ssm_config(cfg);
    if (st != GDN_OK)
        return st;
    if ((st = check_ssm_params(params)) != GDN_OK)
        return st;
    if (batch < 0 || total_tokens < 0 || (batch == 0 && total_tokens > 0) ||
        (batch > 0 && cu_seqlens == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (batch > 65535 || total_tokens > INT32_MAX || !ssm_addressable(cfg, batch, total_tokens))
        return GDN_ERR_UNSUPPORTED;
    if ((st = check_ssm_rows(cfg, xbc, xbc_stride, dt, dt_stride, z, z_stride, y, total_tokens)) != GDN_OK)
        return st;
    if (!aligned(cu_seqlens, 4) || !aligned(initial_state, 16) || !aligned(initial_conv, 16) ||
        !aligned(final_state, 16) || !aligned(final_conv, 16))
        return GDN_ERR_INVALID_ARG;
    const size_t need = ssm_workspace_bytes(cfg, batch, total_tokens);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256)))
        return GDN_ERR_WORKSPACE;
    const ProfileHook hook = take_profile_hook();
    const long long wait_limit = take_wait_limit();
    if (batch == 0)
        return GDN_OK;
    SsmArgs p = ssm_args(cfg, params, xbc, xbc_stride, dt, dt_stride, z, z_stride, batch, y);
    p.cu = cu_seqlens;
    p.N = total_tokens;
    p.init_state = initial_state;
    p.init_conv = initial_conv;
    p.final_state = final_state;
    p.final_conv = final_conv;
    p.ws = workspace;
    p.wait_limit = wait_limit;
    ssm_cut(cfg, batch, total_tokens, &p.segments, &p.fine);
    return cuda_status(launch_ssm_prefill(p, hook.begin, hook.end, (cudaStream_t)stream));
}

gdn_status gdn_ssm_decode(const gdn_ssm_config *cfg, const gdn_ssm_params *params, const void *xbc,
                          int64_t xbc_stride, const void *dt, int64_t dt_stride, const void *z,
                          int64_t z_stride, float *state, void *conv_cache, int32_t batch, void *y,
                          void *stream) {
    gdn_status st = check_ssm_config(cfg);
    if (st != GDN_OK)
        return st;
    if ((st = check_ssm_params(params)) != GDN_OK)
        return st;
    if (batch < 0)
        return GDN_ERR_INVALID_ARG;
    if (batch > 65535)
        return GDN_ERR_UNSUPPORTED;
    if ((st = check_ssm_rows(cfg, xbc, xbc_stride, dt, dt_stride, z, z_stride, y, batch)) != GDN_OK)
        return st;
    if (batch > 0 && (state == nullptr || conv_cache == nullptr || !aligned(state, 16) || !aligned(conv_cache, 16)))
        return GDN_ERR_INVALID_ARG;
    const ProfileHook hook = take_profile_hook();
    if (batch == 0)
        return GDN_OK;
    SsmArgs p = ssm_args(cfg, params, xbc, xbc_stride, dt, dt_stride, z, z_stride, batch, y);
    p.N = batch;
    p.state = state;
    p.conv_cache = conv_cache;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = record_if(hook.begin, s);
    if (e == cudaSuccess)
        e = launch_ssm_decode(p, s);
    if (e == cudaSuccess)
        e = record_if(hook.end, s);
    return cuda_status(e);
}

gdn_status gdn_rmsnorm_fp8(const gdn_norm_config *cfg, const void *x, int64_t x_stride, const void *residual,
                           const float *weight, void *residual_out, void *y, void *q, float *scale,
                           void *stream) {
    if (cfg == nullptr || cfg->rows < 0 || cfg->dim < 1 || cfg->dim % 8 != 0 || cfg->groups < 1 ||
        cfg->dim % cfg->groups != 0 || !dtype_ok(cfg->act_dtype) || !(cfg->eps >= 0.f) || !isfinite(cfg->eps) ||
        !isfinite(cfg->weight_offset))
        return GDN_ERR_INVALID_ARG;
    if (cfg->groups > 1 && (cfg->dim / cfg->groups) % 128 != 0)
        return GDN_ERR_UNSUPPORTED;
    if (cfg->dim > 1 << 24 || cfg->rows > INT32_MAX / cfg->groups) // the grid is one dimension
        return GDN_ERR_UNSUPPORTED;
    if ((q == nullptr) != (scale == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (cfg->rows == 0)
        return GDN_OK;
    if (x == nullptr || (residual_out == nullptr && y == nullptr && q == nullptr))
        return GDN_ERR_INVALID_ARG;
    if (x_stride < cfg->dim || (x_stride * dtype_bytes(cfg->act_dtype)) % 16 != 0 || x_stride > INT32_MAX)
        return GDN_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
        !aligned(y, 16) || !aligned(q, 16) || !aligned(scale, 4))
        return GDN_ERR_INVALID_ARG;
    if (residual_out != nullptr && residual_out == x && x_stride != cfg->dim)
        return GDN_ERR_INVALID_ARG;
    NormArgs p{cfg->rows, cfg->dim, cfg->groups, cfg->act_dtype == GDN_BF16, cfg->eps, cfg->weight_offset,
               x, x_stride, residual, weight, residual_out, y, q, scale};
    return cuda_status(launch_norm(p, (cudaStream_t)stream));
}

static gdn_status check_matmul_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 1 || K % 16 != 0)
        return GDN_ERR_INVALID_ARG;
    if (M > 1 << 30 || N > 1 << 30 || K > 1 << 30) // TMA coordinates are 32-bit
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status gdn_matmul_fp8_workspace_size(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    const gdn_status st = check_matmul_shape(M, N, K);
    if (st != GDN_OK)
        return st;
    if (bytes == nullptr)
        return GDN_ERR_INVALID_ARG;
    *bytes = M == 0 || N == 0 ? 0 : matmul_workspace_bytes(M, N, K);
    return GDN_OK;
}

gdn_status gdn_matmul_fp8(const void *a, const float *a_scale, const void *w, const float *w_scale, int64_t M,
                          int64_t N, int64_t K, void *out, int64_t out_stride, int32_t out_dtype,
                          void *workspace, size_t workspace_bytes, void *stream) {
    const gdn_status st = check_matmul_shape(M, N, K);
    if (st != GDN_OK)
        return st;
    if (!dtype_ok(out_dtype))
        return GDN_ERR_INVALID_ARG;
    if (M == 0 || N == 0) {
        take_wait_limit(); // the armed bound was for this call
        return GDN_OK;
    }
    if (a == nullptr || a_scale == nullptr || w == nullptr || w_scale == nullptr || out == nullptr ||
        out_stride < N || out_stride > INT32_MAX)
        return GDN_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4))
        return GDN_ERR_INVALID_ARG;
    const size_t need = matmul_workspace_bytes(M, N, K);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
        return GDN_ERR_WORKSPACE;
    MatmulArgs p{a, w, a_scale, w_scale, M, N, K, out, out_stride, out_dtype == GDN_BF16, workspace, take_wait_limit()};
    return cuda_status(launch_matmul(p, (cudaStream_t)stream));
}

} // extern "C"
