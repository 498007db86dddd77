// gdn_norm.cu -- root-mean-square norm with the residual's addition and an
// e4m3 output with one float32 scale for each 128 elements, and the plain
// quantisation (no weight: v = r).
//
//     r = x + residual,  v = r / sqrt(mean r^2 + eps) * (offset + weight),
//     scale = max(max|v| / 448, 2^-126),  q = e4m3(v / scale)
//
// Bound by HBM: each input is read once and each output written once, with the
// row held in registers between the sum of squares and the output.
// A thread's unit is 8 consecutive elements, so that 16 neighbouring lanes
// hold one block of 128 and the block's maximum is four shuffles.
#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

template <typename T> __device__ __forceinline__ void load8(const T *p, float (&v)[8]);
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&v)[8]) {
    const Vec16<__nv_bfloat16> x = ld16(p);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = x.get(i);
}
template <> __device__ __forceinline__ void load8<float>(const float *p, float (&v)[8]) {
    const Vec16<float> x = ld16(p), y = ld16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = x.get(i);
        v[i + 4] = y.get(i);
    }
}
template <typename T> __device__ __forceinline__ void store8(T *p, const float (&v)[8]);
template <> __device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float (&v)[8]) {
    Vec16<__nv_bfloat16> x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x.set(i, v[i]);
    st16(p, x);
}
template <> __device__ __forceinline__ void store8<float>(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

// Two floats to two e4m3 bytes (the first in the low byte), to nearest even,
// saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// r of unit u of a row: x + residual in float32.
template <typename T>
__device__ __forceinline__ void load_unit(const T *x, const T *res, int u, float (&v)[8]) {
    load8(x + 8 * u, v);
    if (res != nullptr) {
        float w[8];
        load8(res + 8 * u, w);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += w[i];
    }
}

// The outputs of unit u (active), and its share of the block's maximum.  The
// maximum is taken over the bit patterns of |v|, which order like the values
// and put infinity and NaN above all of them, so that neither is lost.
template <typename T>
__device__ __forceinline__ void emit_unit(const NormArgs &p, bool active, int64_t row, int first, int u,
                                          float rs, float (&v)[8]) {
    const int col = first + 8 * u; // column in the whole row
    const int64_t at = row * p.dim + col;
    if (active) {
        if (p.residual_out != nullptr)
            store8(reinterpret_cast<T *>(p.residual_out) + at, v);
        if (p.weight != nullptr) {
            float w[8];
            load8(p.weight + col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = v[i] * rs * (p.weight_offset + w[i]);
        }
        if (p.y != nullptr)
            store8(reinterpret_cast<T *>(p.y) + at, v);
    }
    if (p.q == nullptr)
        return;
    uint32_t m = 0u;
    if (active) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!active)
        return;
    const float amax = __uint_as_float(m);
    // fmaxf would drop a NaN maximum
    const float scale = m > 0x7f800000u ? amax : fmaxf(amax / 448.0f, 1.17549435e-38f);
    const float inv = 1.0f / scale;
    uint2 b;
    b.x = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
    b.y = e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16);
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(p.q) + at) = b;
    if ((col & 127) == 0)
        p.scale[row * ((p.dim + 127) / 128) + col / 128] = scale;
}

// One row part (a norm group) per `TPR` threads, NU units per thread in
// registers; NU = 0: parts of any length, read a second time for the output.
template <typename T, int TPR, int NU>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) norm_kernel(const NormArgs p) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    __shared__ float red[kThreads / 32];
    const int tid = threadIdx.x % TPR;
    const int64_t part = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (part >= p.rows * p.groups)
        return; // whole warps: TPR is a multiple of 32
    const int64_t row = part / p.groups;
    const int len = p.dim / p.groups, first = (int)(part % p.groups) * len, units = len / 8;
    const T *x = reinterpret_cast<const T *>(p.x) + row * p.x_stride + first;
    const T *res = p.residual == nullptr ? nullptr
                                         : reinterpret_cast<const T *>(p.residual) + row * p.dim + first;
    float v[NU > 0 ? NU : 1][8];
    float ss = 0.f;
    if (NU > 0) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            const int u = tid + i * TPR;
            if (u < units) {
                load_unit(x, res, u, v[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    ss = fmaf(v[i][k], v[i][k], ss);
            }
        }
    } else if (p.weight != nullptr) {
        for (int u = tid; u < units; u += TPR) {
            load_unit(x, res, u, v[0]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                ss = fmaf(v[0][k], v[0][k], ss);
        }
    }
    float rs = 1.f;
    if (p.weight != nullptr) {
        ss = group_sum<32>(ss);
        if (TPR > 32) {
            if ((tid & 31) == 0)
                red[tid >> 5] = ss;
            __syncthreads();
            ss = (tid & 31) < TPR / 32 ? red[tid & 31] : 0.f;
            ss = group_sum<32>(ss);
        }
        rs = rsqrtf(ss / (float)len + p.eps);
    }
    if (NU > 0) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
            if (TPR == 32 ? i * 32 < units : i * TPR + (tid & ~31) < units) // uniform over the warp
                emit_unit<T>(p, tid + i * TPR < units, row, first, tid + i * TPR, rs, v[i]);
        }
    } else {
        for (int u = tid; (u & ~31) < units; u += TPR) {
            if (u < units)
                load_unit(x, res, u, v[0]);
            emit_unit<T>(p, u < units, row, first, u, rs, v[0]);
        }
    }
}

template <typename T, int TPR, int NU> cudaError_t go(const NormArgs &p, cudaStream_t s) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR;
    const int64_t parts = p.rows * p.groups;
    norm_kernel<T, TPR, NU><<<(unsigned)((parts + kThreads / TPR - 1) / (kThreads / TPR)), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const NormArgs &p, cudaStream_t s) {
    const int units = p.dim / p.groups / 8;
    if (units <= 32)
        return go<T, 32, 1>(p, s);
    if (units <= 128)
        return go<T, 32, 4>(p, s);
    if (units <= 256)
        return go<T, 256, 1>(p, s);
    if (units <= 512)
        return go<T, 256, 2>(p, s);
    if (units <= 1024)
        return go<T, 256, 4>(p, s);
    return go<T, 256, 0>(p, s);
}

} // namespace

cudaError_t launch_norm(const NormArgs &p, cudaStream_t s) {
    return p.bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

} // namespace gdn
