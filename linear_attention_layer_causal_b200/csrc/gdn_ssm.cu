// gdn_ssm.cu -- prefill of the selective state-space mixer: token by token.
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// One channel and token: convolution and SiLU into ws_u [N, C] float32.
template <typename T> __global__ void __launch_bounds__(kThreads) ssm_conv_kernel(const SsmArgs p, float *u) {
    const int C = p.conv_dim();
    const int c = blockIdx.y * kThreads + threadIdx.x;
    const int64_t t = blockIdx.x;
    if (c >= C)
        return;
    const int n = seq_of_token(p.cu, p.batch, t);
    int64_t s, e;
    seq_bounds(p.cu, n, p.N, s, e);
    if (t < s || t >= e)
        return;
    float acc = p.conv_b ? p.conv_b[c] : 0.f;
    for (int i = 0; i < 4; ++i) {
        const int64_t src = t - 3 + i;
        float v = 0.f;
        if (src >= s)
            v = to_f(reinterpret_cast<const T *>(p.xbc)[src * p.xbc_stride + c]);
        else if (p.init_conv)
            v = to_f(reinterpret_cast<const T *>(p.init_conv)[((int64_t)n * 3 + 3 + (src - s)) * C + c]);
        acc = fmaf(p.conv_w[c * 4 + i], v, acc);
    }
    u[t * C + c] = siluf_(acc);
}

// One sequence and head: the recurrence, a warp per state row at a time.
template <typename T, int P, int S>
__global__ void __launch_bounds__(kThreads) ssm_serial_kernel(const SsmArgs p, const float *u) {
    constexpr int R = P / 8, E = S / 32;
    const int h = blockIdx.x, n = blockIdx.y, j = h / (p.H / p.G), C = p.conv_dim();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t s, e;
    seq_bounds(p.cu, n, p.N, s, e);
    float st[R][E];
    const int64_t at = (((int64_t)n * p.H + h) * P + warp * R) * S + lane * E;
    for (int r = 0; r < R; ++r)
        for (int k = 0; k < E; ++k)
            st[r][k] = p.init_state ? p.init_state[at + r * S + k] : 0.f;
    const float A = -expf(p.A_log[h]), bias = p.dt_bias ? p.dt_bias[h] : 0.f, D = p.D ? p.D[h] : 0.f;
    for (int64_t t = s; t < e; ++t) {
        const float d = ssm_delta(to_f(reinterpret_cast<const T *>(p.dt)[t * p.dt_stride + h]), bias, p.dt_min, p.dt_max);
        const float a = expf(A * d);
        const float *row = u + t * C;
        float b[E], c[E];
        for (int k = 0; k < E; ++k) {
            b[k] = row[p.H * P + j * S + lane * E + k];
            c[k] = row[p.H * P + p.G * S + j * S + lane * E + k];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float x = row[h * P + warp * R + r];
            float acc = 0.f;
            for (int k = 0; k < E; ++k) {
                st[r][k] = fmaf(d * x, b[k], a * st[r][k]);
                acc = fmaf(st[r][k], c[k], acc);
            }
            acc = group_sum<32>(acc);
            if (lane == 0) {
                const int col = h * P + warp * R + r;
                float y = fmaf(D, x, acc);
                if (p.z)
                    y *= siluf_(to_f(reinterpret_cast<const T *>(p.z)[t * p.z_stride + col]));
                reinterpret_cast<T *>(p.y)[t * p.H * P + col] = from_f<T>(y);
            }
        }
    }
    if (p.final_state)
        for (int r = 0; r < R; ++r)
            for (int k = 0; k < E; ++k)
                p.final_state[at + r * S + k] = st[r][k];
}

// The last three pre-conv rows of [initial window; sequence].
template <typename T> __global__ void __launch_bounds__(kThreads) ssm_final_conv_kernel(const SsmArgs p) {
    const int C = p.conv_dim(), c = blockIdx.x * kThreads + threadIdx.x, n = blockIdx.y;
    if (c >= C)
        return;
    int64_t s, e;
    seq_bounds(p.cu, n, p.N, s, e);
    T v[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t src = e - 3 + i;
        if (src >= s)
            v[i] = reinterpret_cast<const T *>(p.xbc)[src * p.xbc_stride + c];
        else
            v[i] = p.init_conv ? reinterpret_cast<const T *>(p.init_conv)[((int64_t)n * 3 + 3 + (src - s)) * C + c]
                               : from_f<T>(0.f);
    }
    for (int i = 0; i < 3; ++i)
        reinterpret_cast<T *>(p.final_conv)[((int64_t)n * 3 + i) * C + c] = v[i];
}

template <typename T> cudaError_t launch_t(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    const int C = p.conv_dim();
    float *u = reinterpret_cast<float *>(p.ws);
    if (p.N > 0)
        ssm_conv_kernel<T><<<dim3((unsigned)p.N, (C + kThreads - 1) / kThreads), kThreads, 0, s>>>(p, u);
    cudaError_t e = record_if(begin, s);
    if (e != cudaSuccess)
        return e;
    const dim3 grid(p.H, p.batch);
    if (p.P == 64 && p.S == 64)
        ssm_serial_kernel<T, 64, 64><<<grid, kThreads, 0, s>>>(p, u);
    else if (p.P == 64)
        ssm_serial_kernel<T, 64, 128><<<grid, kThreads, 0, s>>>(p, u);
    else if (p.S == 64)
        ssm_serial_kernel<T, 128, 64><<<grid, kThreads, 0, s>>>(p, u);
    else
        ssm_serial_kernel<T, 128, 128><<<grid, kThreads, 0, s>>>(p, u);
    e = record_if(end, s);
    if (e == cudaSuccess && p.final_conv)
        ssm_final_conv_kernel<T><<<dim3((C + kThreads - 1) / kThreads, p.batch), kThreads, 0, s>>>(p);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

} // namespace

size_t ssm_workspace_bytes(const gdn_ssm_config *c, int, int64_t N) {
    return round_up((size_t)N * ((size_t)c->num_heads * c->head_dim + 2 * (size_t)c->num_groups * c->state_dim) * 4);
}

cudaError_t launch_ssm_prefill(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    return p.bf16 ? launch_t<__nv_bfloat16>(p, begin, end, s) : launch_t<float>(p, begin, end, s);
}

} // namespace gdn
