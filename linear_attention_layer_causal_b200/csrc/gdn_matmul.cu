// gdn_matmul.cu -- product of e4m3 operands with one float32 scale for each
// 1 x 128 block of a and each 128 x 128 block of w:
//     out[m][n] = sum_b sa[m][b] sw[n / 128][b] sum_{k in block b} a[m][k] w[n][k].
#include <cuda_fp8.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kT = 64, kKT = 16;

template <typename O> __global__ void __launch_bounds__(256) matmul_kernel(const MatmulArgs p) {
    __shared__ float as[kKT][kT + 1], ws[kKT][kT + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
    const int64_t KB = (p.K + 127) / 128;
    float acc[4][4] = {}, part[4][4] = {};
    const __nv_fp8_e4m3 *a = reinterpret_cast<const __nv_fp8_e4m3 *>(p.a);
    const __nv_fp8_e4m3 *w = reinterpret_cast<const __nv_fp8_e4m3 *>(p.w);
    for (int64_t k0 = 0; k0 < p.K; k0 += kKT) {
        for (int i = tid; i < kT * kKT; i += 256) {
            const int r = i / kKT, c = i % kKT;
            as[c][r] = m0 + r < p.M ? float(a[(m0 + r) * p.K + k0 + c]) : 0.f;
            ws[c][r] = n0 + r < p.N ? float(w[(n0 + r) * p.K + k0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < kKT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[i][j] = fmaf(as[c][ty + 16 * i], ws[c][tx + 16 * j], part[i][j]);
        __syncthreads();
        if ((k0 + kKT) % 128 == 0 || k0 + kKT == p.K) {
            const int64_t b = k0 / 128;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                    if (m < p.M && n < p.N)
                        acc[i][j] = fmaf(p.a_scale[m * KB + b] * p.w_scale[n / 128 * KB + b], part[i][j], acc[i][j]);
                    part[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N)
                reinterpret_cast<O *>(p.out)[m * p.out_stride + n] = from_f<O>(acc[i][j]);
        }
}

} // namespace

size_t matmul_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

cudaError_t launch_matmul(const MatmulArgs &p, cudaStream_t s) {
    const dim3 grid((unsigned)((p.N + kT - 1) / kT), (unsigned)((p.M + kT - 1) / kT));
    if (p.out_bf16)
        matmul_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
    else
        matmul_kernel<float><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace gdn
