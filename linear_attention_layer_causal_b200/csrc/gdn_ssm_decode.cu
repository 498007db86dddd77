// gdn_ssm_decode.cu -- one token of the selective state-space mixer per
// sequence against its resident states.
//
//     u = SiLU(conv_b + sum_i conv_w[.][i] xbc_{t-3+i}),  x | B | C = u
//     S <- exp(-exp(A_log) delta) S + delta x B^T,  y = (S C + D x) SiLU(z)
//
// Bound by HBM: every state is read once and written once (4 P S bytes each
// way per head); everything else is a few kilobytes per sequence.
// A block takes units of 64 state rows of one group.  Its first unit's states
// are requested before the convolution, whose latency they cover, and each
// later unit's before the unit ahead of it is worked on.  256 sequences of 128
// heads of 64 and 128 states: 337 us, 6.5 TB/s; one sequence 5.2 us, in two kernels
// (the windows of B and C move on behind the blocks that read them).
#include "gdn_ssm.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = 8, kUnitRows = 64, kMaxUnits = 8;

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 r;
    r.x = *reinterpret_cast<uint32_t *>(&a);
    r.y = *reinterpret_cast<uint32_t *>(&b);
    *reinterpret_cast<uint2 *>(p) = r;
}
__device__ __forceinline__ void store4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }

// Loads that the same kernel's stores may follow: not through the read-only path.
__device__ __forceinline__ float4 load4_rw(const __nv_bfloat16 *p) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4_rw(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// Convolution and SiLU of channels c .. c + 3 of sequence n.  With `advance`
// the window's rows move up by one and the new row is appended.
template <typename T>
__device__ __forceinline__ float4 conv4(const SsmArgs &p, int n, int c, bool advance) {
    const int C = p.conv_dim();
    T *win = reinterpret_cast<T *>(p.conv_cache) + (int64_t)n * 3 * C + c;
    const float4 r0 = load4_rw(win), r1 = load4_rw(win + C), r2 = load4_rw(win + 2 * C);
    const float4 r3 = load4(reinterpret_cast<const T *>(p.xbc) + (int64_t)n * p.xbc_stride + c);
    const float4 *w = reinterpret_cast<const float4 *>(p.conv_w) + c;
    const float4 w0 = __ldg(w), w1 = __ldg(w + 1), w2 = __ldg(w + 2), w3 = __ldg(w + 3);
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.conv_b != nullptr)
        b = __ldg(reinterpret_cast<const float4 *>(p.conv_b + c));
    float4 o;
    o.x = siluf_(fmaf(w0.w, r3.x, fmaf(w0.z, r2.x, fmaf(w0.y, r1.x, fmaf(w0.x, r0.x, b.x)))));
    o.y = siluf_(fmaf(w1.w, r3.y, fmaf(w1.z, r2.y, fmaf(w1.y, r1.y, fmaf(w1.x, r0.y, b.y)))));
    o.z = siluf_(fmaf(w2.w, r3.z, fmaf(w2.z, r2.z, fmaf(w2.y, r1.z, fmaf(w2.x, r0.z, b.z)))));
    o.w = siluf_(fmaf(w3.w, r3.w, fmaf(w3.z, r2.w, fmaf(w3.y, r1.w, fmaf(w3.x, r0.w, b.w)))));
    if (advance) {
        store4(win, r1);
        store4(win + C, r2);
        store4(win + 2 * C, r3);
    }
    return o;
}

// grid: (unit blocks of all groups, batch).  `units`: units of a group,
// `per`: units of a block, `blocks`: blocks of a group.
template <typename T, int P, int S>
__global__ void __launch_bounds__(kThreads) ssm_decode_kernel(const SsmArgs p, int units, int per, int blocks) {
    constexpr int LPR = S / 4;          // lanes per state row
    constexpr int RPI = 32 / LPR;       // rows of a warp's step
    constexpr int NV = kUnitRows / kWarps / RPI; // steps of a unit
    __shared__ __align__(16) float bs[S], cs[S], xs[kMaxUnits * kUnitRows], ys[kMaxUnits * kUnitRows];
    __shared__ float dl[kMaxUnits], al[kMaxUnits]; // per unit: delta, decay
    const int n = blockIdx.y, j = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    const int u0 = blk * per, nu = min(per, units - u0);
    const int hpg = p.H / p.G;
    // first state row of the block within the sequence, and the matching x channel
    const int row0 = j * hpg * P + u0 * kUnitRows;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sub = lane / LPR, c4 = (lane % LPR) * 4;
    float *st = p.state + ((int64_t)n * p.H * P + row0 + warp * (kUnitRows / kWarps) + sub) * S + c4;

    float4 cur[NV], nxt[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        cur[i] = __ldcs(reinterpret_cast<const float4 *>(st + i * RPI * S));
#if __CUDA_ARCH__ >= 900
    asm volatile("griddepcontrol.launch_dependents;");
#endif
    // x of the block's rows, then B and C of its group.  Only this block has the
    // x channels, so it advances their windows; B's and C's are read by every
    // block of the group, which advances them only where it is the only one.
    const int nx = nu * kUnitRows / 4;
    for (int i = tid; i < nx + 2 * S / 4; i += kThreads) {
        if (i < nx) {
            *reinterpret_cast<float4 *>(xs + 4 * i) = conv4<T>(p, n, row0 + 4 * i, true);
        } else {
            const int k = 4 * (i - nx);
            const int c = p.H * P + (k < S ? j * S + k : p.G * S + j * S + k - S);
            *reinterpret_cast<float4 *>(k < S ? bs + k : cs + k - S) = conv4<T>(p, n, c, blocks == 1);
        }
    }
    if (tid < nu) {
        const int h = (row0 + tid * kUnitRows) / P;
        const float d = ssm_delta(to_f(reinterpret_cast<const T *>(p.dt)[(int64_t)n * p.dt_stride + h]),
                                  p.dt_bias ? __ldg(p.dt_bias + h) : 0.f, p.dt_min, p.dt_max);
        dl[tid] = d;
        al[tid] = expf(-expf(__ldg(p.A_log + h)) * d);
    }
    __syncthreads();
    const float4 bv = *reinterpret_cast<const float4 *>(bs + c4), cv = *reinterpret_cast<const float4 *>(cs + c4);
    for (int u = 0; u < nu; ++u) {
        float *su = st + (int64_t)u * kUnitRows * S;
        if (u + 1 < nu) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                nxt[i] = __ldcs(reinterpret_cast<const float4 *>(su + (int64_t)kUnitRows * S + i * RPI * S));
        }
        const float a = al[u], d = dl[u];
        const int r0 = u * kUnitRows + warp * (kUnitRows / kWarps);
        float acc[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float f = d * xs[r0 + i * RPI + sub];
            float4 v = cur[i];
            v.x = fmaf(f, bv.x, a * v.x);
            v.y = fmaf(f, bv.y, a * v.y);
            v.z = fmaf(f, bv.z, a * v.z);
            v.w = fmaf(f, bv.w, a * v.w);
            __stcs(reinterpret_cast<float4 *>(su + i * RPI * S), v);
            acc[i] = fmaf(v.x, cv.x, fmaf(v.y, cv.y, fmaf(v.z, cv.z, v.w * cv.w)));
        }
        // sums over the LPR lanes of a row, of NV rows at once: each exchange
        // halves the rows that a lane still carries
        int held = NV, o = LPR / 2;
#pragma unroll
        for (int step = 0; step < 5; ++step) {
            if (o == 0)
                break;
            if (held > 1) {
                const bool up = lane & o;
#pragma unroll
                for (int i = 0; i < NV / 2; ++i)
                    if (i < held / 2) {
                        const float keep = up ? acc[i + held / 2] : acc[i];
                        const float give = up ? acc[i] : acc[i + held / 2];
                        acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                held /= 2;
            } else {
                acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
            }
            o >>= 1;
        }
        // lane bits LPR/2, LPR/4, ... chose the upper half of 8 (4) rows, 4 (2), ...
        const int l = lane % LPR;
        int i = 0;
#pragma unroll
        for (int k = 0; (NV >> (k + 1)) > 0; ++k)
            i |= ((l >> (31 - __clz(LPR) - 1 - k)) & 1) * (NV >> (k + 1));
        if ((l & (LPR / NV - 1)) == 0)
            ys[r0 + i * RPI + sub] = acc[0];
        if (u + 1 < nu) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                cur[k] = nxt[k];
        }
    }
    __syncthreads();
    for (int i = tid; i < nu * kUnitRows; i += kThreads) {
        const int r = row0 + i, h = r / P;
        float y = ys[i];
        if (p.D != nullptr)
            y = fmaf(__ldg(p.D + h), xs[i], y);
        if (p.z != nullptr)
            y *= siluf_(to_f(reinterpret_cast<const T *>(p.z)[(int64_t)n * p.z_stride + r]));
        reinterpret_cast<T *>(p.y)[(int64_t)n * p.H * P + r] = from_f<T>(y);
    }
}

// The windows of the B and C channels, after every block of ssm_decode_kernel
// has read them.  Launched to start beside that kernel and wait for its end.
template <typename T> __global__ void __launch_bounds__(kThreads) ssm_window_kernel(const SsmArgs p) {
    const int C = p.conv_dim(), first = p.H * p.P;
    const int c = first + 4 * (blockIdx.x * kThreads + threadIdx.x), n = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= C)
        return;
    T *win = reinterpret_cast<T *>(p.conv_cache) + (int64_t)n * 3 * C + c;
    const float4 r1 = load4_rw(win + C), r2 = load4_rw(win + 2 * C);
    const float4 r3 = load4(reinterpret_cast<const T *>(p.xbc) + (int64_t)n * p.xbc_stride + c);
    store4(win, r1);
    store4(win + C, r2);
    store4(win + 2 * C, r3);
}

template <typename T, int P, int S> cudaError_t launch_t(const SsmArgs &p, cudaStream_t s) {
    const int units = p.H / p.G * P / kUnitRows;
    // one unit per block while that leaves SMs idle or barely filled
    const int64_t all = (int64_t)p.batch * p.G * units;
    int per = all <= 4 * 148 ? 1 : 4;
    if (per > units)
        per = units;
    const int blocks = (units + per - 1) / per;
    ssm_decode_kernel<T, P, S><<<dim3(p.G * blocks, p.batch), kThreads, 0, s>>>(p, units, per, blocks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || blocks == 1)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((2 * p.G * S / 4 + kThreads - 1) / kThreads, p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ssm_window_kernel<T>, p);
}

template <typename T> cudaError_t launch_s(const SsmArgs &p, cudaStream_t s) {
    if (p.P == 64)
        return p.S == 64 ? launch_t<T, 64, 64>(p, s) : launch_t<T, 64, 128>(p, s);
    return p.S == 64 ? launch_t<T, 128, 64>(p, s) : launch_t<T, 128, 128>(p, s);
}

} // namespace

cudaError_t launch_ssm_decode(const SsmArgs &p, cudaStream_t s) {
    return p.bf16 ? launch_s<__nv_bfloat16>(p, s) : launch_s<float>(p, s);
}

} // namespace gdn
