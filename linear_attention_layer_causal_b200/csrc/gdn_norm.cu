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

// Eight activations as loaded: 16 bytes of bf16 or 32 of float32.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? a.x : i < 4 ? a.y : i < 6 ? a.z : a.w;
        return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ float get(int i) const {
        const float4 v = i < 4 ? a : b;
        return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
    }
};
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

// v / scale as e4m3 rounds the float32 quotient.  The product with the
// reciprocal alone is off by up to 1.5 units and misses ties; one step with the
// remainder, which a fused multiply-add has exactly (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990), leaves
// about 2^-46 of the quotient before its rounding, and no such error reaches
// across a tie or the middle between a tie and the float32 next to it
// (tests/test_fp8_rounding.py goes through the quotients that come nearest).
// The remainder's sign is chosen so that -0 stays -0.
__device__ __forceinline__ void divide(float (&v)[8], float scale) {
    const float inv = 1.0f / scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = v[i] * inv;
        v[i] = fmaf(-fmaf(q, scale, -v[i]), inv, q);
    }
}

// One unit, at element `at`: r and v are written out where they are asked for, v
// stays.  Returns the unit's share of its block's maximum, which is taken over
// the bit patterns of |v|: they order like the values and put infinity and NaN
// above all of them, so that neither is lost.
template <typename T>
__device__ __forceinline__ uint32_t norm_unit(const NormArgs &p, bool active, int64_t at, float rs, const Raw8<float> &w,
                                              float (&v)[8]) {
    uint32_t m = 0u;
    if (active) {
        if (p.residual_out != nullptr)
            store8(reinterpret_cast<T *>(p.residual_out) + at, v);
        if (p.weight != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = v[i] * rs * (p.weight_offset + w.get(i));
        }
        if (p.y != nullptr)
            store8(reinterpret_cast<T *>(p.y) + at, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
    return m;
}
// The maximum over the 16 lanes that hold a block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
// A block below 2^-71 (its remainders could be subnormal), or with an infinity or a NaN.
__device__ __forceinline__ bool unusual(uint32_t m) { return m < 0x1c000000u || m >= 0x7f800000u; }

// The 8-bit values of one unit, and its block's scale.
template <bool DIVIDE>
__device__ __forceinline__ void quant_unit(const NormArgs &p, int64_t row, int col, uint32_t m, float (&v)[8]) {
    const float amax = __uint_as_float(m);
    // fmaxf would drop a NaN maximum
    const float scale = m > 0x7f800000u ? amax : fmaxf(amax / 448.0f, 1.17549435e-38f);
    if (DIVIDE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] / scale;
    } else {
        divide(v, scale);
    }
    uint2 b;
    b.x = e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16);
    b.y = e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16);
    *reinterpret_cast<uint2 *>(reinterpret_cast<uint8_t *>(p.q) + row * p.dim + col) = b;
    if ((col & 127) == 0)
        p.scale[row * ((p.dim + 127) / 128) + col / 128] = scale;
}

// The outputs of R units of a part, TPR apart from u on.  The units go through
// each step together, with one choice between the two quotients for a warp's
// units (4096 x 8192 bf16 with a residual: 40.9 us; unit by unit, each with its
// own choice, 47.2; every quotient divided 60.8).
template <typename T, int TPR, int R>
__device__ __forceinline__ void emit(const NormArgs &p, int64_t row, int first, int u, int units, float rs,
                                     const Raw8<float> (&w)[R], float (&v)[R][8]) {
    uint32_t m[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        m[i] = norm_unit<T>(p, u + i * TPR < units, row * p.dim + first + 8 * (u + i * TPR), rs, w[i], v[i]);
    if (p.q == nullptr)
        return;
    bool divided = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = block_max(m[i]);
        divided |= u + i * TPR < units && unusual(m[i]);
    }
    if (!__any_sync(0xffffffffu, divided)) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (u + i * TPR < units)
                quant_unit<false>(p, row, first + 8 * (u + i * TPR), m[i], v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (u + i * TPR < units)
                quant_unit<true>(p, row, first + 8 * (u + i * TPR), m[i], v[i]);
    }
}

// Blocks of an instance that an SM holds at once: the launch bounds give each
// the registers that this leaves it, and the host starts as many as run at once
// (8192 x 2048 bf16 with a residual 26.8 us, and 35.2 where the registers left
// room for three blocks of the four; 4096 x 2048 float32 19.5 with three, and
// 24.4 with a grid for four).
template <typename T, int TPR, int NU> constexpr int kResident =
    TPR > 256 ? 1 : sizeof(T) == 2 ? (NU == 1 ? 4 : 2) : NU == 1 ? 3 : NU == 2 ? 2 : 1;

// Row parts (norm groups) per `TPR` threads, NU units per thread in registers;
// NU = 0: parts of any length, two units at a time, read a second time for the
// output (4096 x 16384 bf16 quantised: 90.9 us; with one unit at a time 116).
// With fewer blocks than parts a block takes every gridDim-th part: its
// weights stay in registers (the host makes the step a multiple of the number
// of groups), and the next part is on its way while this one is worked on.
// 4096 x 8192 bf16 with a residual: 40.9 us, 5.8 TB/s; a block per row took 59.
// One row of 8192: 3.4 us, its launch and a chain of load, two sums and store.
template <typename T, int TPR, int NU>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, kResident<T, TPR, NU>) norm_kernel(const NormArgs p) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, R = NU > 0 ? NU : 2;
    __shared__ float red[2][kThreads / 32];
    const int tid = threadIdx.x % TPR;
    const int64_t parts = p.rows * p.groups, step = (int64_t)gridDim.x * (kThreads / TPR);
    int64_t part = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
    if (part >= parts)
        return; // whole warps: TPR is a multiple of 32
    const int len = p.dim / p.groups, first = (int)(part % p.groups) * len, units = len / 8;
    const bool has_res = p.residual != nullptr, has_norm = p.weight != nullptr;
    Raw8<T> x8[R], r8[R];
    Raw8<float> w[R];
    float v[R][8];
    // The units u0, u0 + TPR, .. of a part: every load is unconditional (units
    // behind the end read the last one), so that all of them are in flight together.
    auto load = [&](int64_t at, int u0) {
        const int64_t row = at / p.groups;
        const T *x = reinterpret_cast<const T *>(p.x) + row * p.x_stride + first;
        const T *res = reinterpret_cast<const T *>(p.residual) + row * p.dim + first;
#pragma unroll
        for (int i = 0; i < R; ++i)
            x8[i].load(x + 8 * min(u0 + i * TPR, units - 1));
        if (has_res) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                r8[i].load(res + 8 * min(u0 + i * TPR, units - 1));
        }
    };
    auto load_w = [&](int u0) {
        if (has_norm) {
#pragma unroll
            for (int i = 0; i < R; ++i)
                w[i].load(p.weight + first + 8 * min(u0 + i * TPR, units - 1));
        }
    };
    auto widen = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[i][k] = has_res ? x8[i].get(k) + r8[i].get(k) : x8[i].get(k);
    };
    float ss;
    auto square = [&](int u0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (u0 + i * TPR < units) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    ss = fmaf(v[i][k], v[i][k], ss);
            }
    };
    if (NU > 0) {
        load(part, tid);
        load_w(tid);
    }
    for (int turn = 0; part < parts; part += step, turn ^= 1) {
        const int64_t row = part / p.groups;
        ss = 0.f;
        if (NU > 0) {
            widen();
            if (part + step < parts)
                load(part + step, tid);
            square(tid);
        } else if (has_norm) {
            for (int u = tid; u < units; u += R * TPR) {
                load(part, u);
                widen();
                square(u);
            }
        }
        float rs = 1.f;
        if (has_norm) {
            ss = group_sum<32>(ss);
            if (TPR > 32) { // the other turn's sums may still be read by slower warps
                if ((tid & 31) == 0)
                    red[turn][tid >> 5] = ss;
                __syncthreads();
                ss = (tid & 31) < TPR / 32 ? red[turn][tid & 31] : 0.f;
                ss = group_sum<32>(ss);
            }
            rs = rsqrtf(ss / (float)len + p.eps);
        }
        if (NU > 0) {
            emit<T, TPR, R>(p, row, first, tid, units, rs, w, v);
        } else {
            for (int u = tid; (u & ~31) < units; u += R * TPR) {
                load(part, u);
                load_w(u);
                widen();
                emit<T, TPR, R>(p, row, first, u, units, rs, w, v);
            }
        }
    }
}

template <typename T, int TPR, int NU> cudaError_t go(const NormArgs &p, cudaStream_t s) {
    constexpr int kThreads = TPR < 256 ? 256 : TPR, PER = kThreads / TPR;
    const int64_t parts = p.rows * p.groups, all = (parts + PER - 1) / PER;
    int64_t blocks = all;
    const int64_t at_once = (int64_t)148 * kResident<T, TPR, NU>; // blocks that run at once
    if (NU > 0 && all > 3 * at_once && at_once >= p.groups)
        blocks = at_once / p.groups * p.groups; // the step is a multiple of the groups
    norm_kernel<T, TPR, NU><<<(unsigned)blocks, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_t(const NormArgs &p, cudaStream_t s) {
    const int units = p.dim / p.groups / 8;
    if (units <= 32)
        return go<T, 32, 1>(p, s);
    if (units <= 128)
        return go<T, 32, 4>(p, s);
    // few rows: the row over more threads, for its latency
    if (units > 256 && units <= 1024 && p.rows * p.groups <= 148)
        return go<T, 1024, 1>(p, s);
    if (units <= 256)
        return go<T, 256, 1>(p, s);
    if (units <= 512)
        return go<T, 256, 2>(p, s);
    if (units <= 1024) // float32: two units a thread leave room for 16 warps (4096 x 8192: 73.6 us; four units, 80.4)
        return sizeof(T) == 2 ? go<T, 256, 4>(p, s) : go<T, 512, 2>(p, s);
    return go<T, 256, 0>(p, s);
}

} // namespace

cudaError_t launch_norm(const NormArgs &p, cudaStream_t s) {
    return p.bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

} // namespace gdn
