// gdn_ssm.cu -- prefill of the selective state-space mixer in chunks of 64
// tokens on the tensor cores.
//
// With G_t the sum of the log-decays of a chunk up to token t, gamma = e^{G_63},
// and H the state entering the chunk (all per head; C, B per group):
//     y_t   = e^{G_t} H C_t + sum_{s <= t} M[t][s] x_s,
//     M[t][s] = e^{G_t - G_s} delta_s (C_t . B_s) + [s = t] D,
//     H     <- gamma H + sum_s x'_s B_s^T,   x'_s = e^{G_63 - G_s} delta_s x_s.
// Every exponent is <= 0: nothing overflows however strong the decay.
//
// Two kernels.  ssm_prep_kernel, per chunk and group: the convolved B and C, the
// products C_t . B_s, and the gates of the group's heads, once for all heads.
// ssm_scan_kernel, per sequence (or segment of it) and 128 state rows (two
// heads of 64 or one of 128): the three products above as tcgen05 MMAs of 128
// rows, with x^T, x'^T and H as the operand in TMEM and C, B and M in shared
// memory; two warps make the masks M, and 16 convolve x, keep the state in
// registers and gate and store the output.
// With few sequences each is cut into segments, and a first run of the scan
// kernel, without outputs, finds what each segment adds to the state.
//
// 4096 tokens of 128 heads of 64, 8 groups, 128 states, bfloat16: 208 us (by
// themselves: prep 31, summary 42, output pass 145), where moving the bytes would
// take 35 and the MMAs 50.  What bounds it is the 16 warps' instructions and their
// latency: two thirds of the issue slots, four such warps to a scheduler (the
// splits, the convolution, two SiLUs); the tensor core is busy for a quarter.
//
// Precision: every operand of a product is the sum of two 16-bit parts, each
// product three MMAs (the product of the two second parts is left out).  x' and B,
// which make the state, are float16 parts, 22 bits of each: the state that is left
// is as exact as a float32 recurrence's (2e-7 against 64 bits, where bfloat16
// parts left 4e-6 and took 197 us).  Where y is float32 so are all other operands;
// where it is bfloat16 they are bfloat16 parts, 2^-17 of each term under y's own
// 2^-9.  float16 has a narrow range, so its operands are scaled by powers of two:
// B and C by their largest in the chunk, x and x' by the largest of each row (for
// which the four threads of a row meet once a chunk), H by a bound of each row, M
// by the largest product and step and by D.  A value of 2^-17 of that largest has
// all its bits; what is smaller is held to 2^-39 of the largest (x' and B where
// they only just make H up: 2^-29).
// Log-decays are summed in 64 bits and M takes their difference as two floats: at
// G = -1000 one float's step alone is 6e-5.  The SiLUs' and masks' exponentials
// and reciprocals are the approximate ones, 2^-22 each.
#include <algorithm>
#include <type_traits>

#include "gdn_sm100.cuh"
#include "gdn_ssm.cuh"
#include "gdn_tmap.h"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kQ = 64;        // tokens of a chunk
constexpr int kMaskRec = 192; // floats of a (chunk, head) for M: G / ln 2, its low part, -ln 2 delta
constexpr int kGateRec = 128; // and for the rest: -ln 2 x' weight, e^G
constexpr int kScaleRec = 4;  // floats of a (chunk, group): what B and C are to be multiplied with
constexpr int kSMs = 148;
constexpr uint32_t kStatusTimeout = 1u;

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Chunks are numbered across the batch without a prefix sum: sequence n's
// first one is cu[n] / 64 + n, which leaves at least as many numbers as it has
// chunks, and at most total / 64 + batch in all.
__device__ __forceinline__ int64_t first_chunk(int64_t start, int n) { return start / kQ + n; }
int64_t max_chunks(int64_t N, int batch) { return N / kQ + batch; }

struct Layout { // workspace offsets in bytes
    size_t bc, cb, masks, gates, scales, seg, segdecay, total;
};
Layout layout(int G, int H, int P, int S, int64_t N, int batch, int slots) {
    const size_t chunks = (size_t)max_chunks(N, batch);
    const size_t tiles = (size_t)G * (((size_t)(H / G) * P + 127) / 128);
    Layout l;
    l.bc = kWorkspaceHeader;
    l.cb = l.bc + round_up(chunks * G * kQ * 4 * S * 2);
    l.masks = l.cb + round_up(chunks * G * kQ * kQ * 4);
    l.gates = l.masks + round_up(chunks * H * kMaskRec * 4);
    l.scales = l.gates + round_up(chunks * H * kGateRec * 4);
    l.seg = l.scales + round_up(chunks * G * kScaleRec * 4);
    l.segdecay = l.seg + (slots > 1 ? round_up((size_t)batch * tiles * slots * 128 * S * 4) : 0);
    l.total = l.segdecay + (slots > 1 ? round_up((size_t)batch * tiles * slots * 2 * 4) : 0);
    return l;
}

// Two floats in one 64-bit register pair, for values that sit in such pairs anyway
// (elsewhere the moves cost more than the paired instruction saves).
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Two floats as two 16-bit parts: hi = the nearest, lo = what is left, each
// packed with the first in the low half.  F16: float16 (22 bits in all, within
// its range), or bfloat16 (16 bits).
template <bool F16> __device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    float ha, hb;
    if (F16) {
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
        asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(ha), "=f"(hb) : "r"(hi));
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b - hb), "f"(a - ha));
    } else {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
        ha = __uint_as_float(hi << 16);
        hb = __uint_as_float(hi & 0xffff0000u);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(b - hb), "f"(a - ha));
    }
}

// Scales.  A largest value with the exponent field e is brought to 2^13 .. 2^14
// by up(e) and back by down(e); both are powers of two, down(e) = 1 / up(e), and
// a field below 14 counts as 14 (values near the smallest normal float).
__device__ __forceinline__ float up(int e) { return __int_as_float(min(267 - e, 253) << 23); }
__device__ __forceinline__ float down(int e) { return __int_as_float(max(e - 13, 1) << 23); }
__device__ __forceinline__ int exponent(float x) { return (__float_as_int(x) >> 23) & 0xff; }
// The largest magnitude of three; NaN where one is (magnitude_nan), or left out.
__device__ __forceinline__ float magnitude_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float magnitude(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 2^n, n clamped to the normal floats.
__device__ __forceinline__ float pow2(int n) { return __int_as_float((max(min(n, 127), -126) + 127) << 23); }
// The larger of each half, and the largest of all four halves.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ int largest_half(uint32_t a, uint32_t b) {
    const uint32_t m = max_halves(a, b);
    return (int)max(m >> 16, m & 0xffffu);
}

// Two outputs to their rows in shared memory, one conversion for both.
__device__ __forceinline__ void put2(__nv_bfloat16 *p, __nv_bfloat16 *q, float a, float b) {
    uint32_t v;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
    *reinterpret_cast<uint16_t *>(p) = (uint16_t)v;
    *reinterpret_cast<uint16_t *>(q) = (uint16_t)(v >> 16);
}
__device__ __forceinline__ void put2(float *p, float *q, float a, float b) {
    *p = a;
    *q = b;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// float32 outputs: every operand as float16 parts.  bfloat16 outputs: those of the state, x' and B, only.
template <typename T> constexpr bool kWhole = sizeof(T) == 4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// SiLU(x) = x / (1 + 2^p), p = -x log2(e); also times y, for a pair.
__device__ __forceinline__ float silu(float x) { return x * rcp(1.f + ex2(-kLog2e * x)); }
__device__ __forceinline__ float2 gated(f2 y, f2 x) {
    const float2 e = unpack(mul2(x, pack(-kLog2e, -kLog2e)));
    const float2 d = unpack(add2(pack(ex2(e.x), ex2(e.y)), pack(1.f, 1.f)));
    return unpack(mul2(mul2(x, pack(rcp(d.x), rcp(d.y))), y));
}
// SiLU(x) / -ln 2 = p / (1 + 2^p).
__device__ __forceinline__ float silu_scaled(float p) { return p * rcp(1.f + ex2(p)); }

// The row of xbc (or of the window before the sequence) that is token t of
// sequence n, t >= start - 3; nullptr for a zero row.
template <typename T> __device__ __forceinline__ const T *conv_row(const SsmArgs &p, int n, int64_t start, int64_t t) {
    if (t >= start)
        return reinterpret_cast<const T *>(p.xbc) + t * p.xbc_stride;
    if (p.init_conv == nullptr)
        return nullptr;
    return reinterpret_cast<const T *>(p.init_conv) + ((int64_t)n * 3 + 3 + (t - start)) * p.conv_dim();
}

// Channel c of the window after sequence n: the last three rows of [initial
// window; sequence].  Read before written: the windows may be the same.
template <typename T> __device__ __forceinline__ void final_window(const SsmArgs &p, int n, int64_t start, int64_t end, int c) {
    T v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const T *row = conv_row<T>(p, n, start, end - 3 + i);
        v[i] = row != nullptr ? row[c] : from_f<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        reinterpret_cast<T *>(p.final_conv)[((int64_t)n * 3 + i) * p.conv_dim() + c] = v[i];
}

// ------------------------------------------------------------------- prep

constexpr int kPrepThreads = 512;
template <int S> constexpr size_t prep_smem() { return (size_t)4 * kQ * (S + 8) * 2; }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// e^g to float32's precision: an exponent of -16 rounded to a float would leave 2^-21 of it.
__device__ __forceinline__ float exp_of(double g) {
    const float h = (float)g;
    return expf(h) * (1.f + (float)(g - (double)h));
}

// One chunk and group; the blocks of z = 1 have the gates.  Writes, for the scan kernel: the rows [64][4 S] of
// B hi | B lo | C hi | C lo (zero behind the sequence's end), scaled; what B and C
// were scaled back with; the 64 x 64 products C_t . B_s of the scaled ones, of
// s's and t's 16-blocks with s <= t (where outputs are float32, in the place of
// row 0, columns 16 to 18, also the two factors and the largest of them; else
// scaled back); and the records of each head of the group.
template <typename T, int S>
__global__ void __launch_bounds__(kPrepThreads, 2) ssm_prep_kernel(const SsmArgs p, uint16_t *bc, float *cb, float *masks, float *gates, float *scales,
                                                                uint32_t *status) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint32_t largest[2][kPrepThreads / 32];
    __shared__ float back[2]; // what the scaled B and C are to be multiplied with
    constexpr int LDS = S + 8; // row length in shared memory: rows 16 bytes apart in banks
    const int64_t id = blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;"); // the scan kernel's blocks may set up beside the last of these
    if (id == 0 && g == 0 && blockIdx.z == 0 && tid == 0)
        status[0] = status[1] = 0;
    // the sequence of this chunk number: the last n with first_chunk(cu[n]) <= id
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        int64_t s, e;
        seq_bounds(p.cu, mid, p.N, s, e);
        if (first_chunk(s, mid) <= id)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int n = lo;
    int64_t start, end;
    seq_bounds(p.cu, n, p.N, start, end);
    const int64_t t0 = start + (id - first_chunk(start, n)) * kQ;
    if (t0 < start || t0 >= end)
        return; // a number without a chunk
    const int ntok = (int)(end - t0 < kQ ? end - t0 : kQ);
    const int C = p.conv_dim();

    if (blockIdx.z == 1) { // gates: a warp per head, two neighbouring tokens per lane
        const int hpg = p.H / p.G;
        for (int k = warp; k < hpg; k += kPrepThreads / 32) {
            const int h = g * hpg + k;
            const double A = -exp((double)__ldg(p.A_log + h));
            const float bias = p.dt_bias != nullptr ? __ldg(p.dt_bias + h) : 0.f;
            float d[2];
            double s[2];
    #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 2 * lane + i;
                d[i] = 0.f;
                s[i] = 0.0;
                if (t < ntok) {
                    d[i] = ssm_delta(to_f(reinterpret_cast<const T *>(p.dt)[(t0 + t) * p.dt_stride + h]), bias, p.dt_min, p.dt_max);
                    // no decay below e^-10000 (zero in float32) and no increase; a NaN stays
                    const double a = d[i] == 0.f ? 0.0 : A * (double)d[i];
                    s[i] = a < -1e4 ? -1e4 : a;
                }
            }
            s[1] += s[0];
            double sum = s[1];
    #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += up;
            }
            double before = __shfl_up_sync(0xffffffffu, sum, 1);
            if (lane == 0)
                before = 0.0;
            const double all = __shfl_sync(0xffffffffu, sum, 31);
            float *mask = masks + (id * p.H + h) * kMaskRec + 2 * lane, *rec = gates + (id * p.H + h) * kGateRec + 2 * lane;
    #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const double G = before + s[i];
                const double G2 = G * 1.4426950408889634; // for base-2 exponentials
                const float gh = (float)G2;
                mask[i] = gh;
                mask[64 + i] = (float)(G2 - (double)gh);
                // times -ln 2: the scan kernel's x is SiLU(x) / -ln 2
                mask[128 + i] = -kLn2 * d[i];
                rec[i] = d[i] == 0.f ? 0.f : -kLn2 * (d[i] * exp_of(all - G));
                rec[64 + i] = exp_of(G);
            }
        }
        return;
    }

    // convolution and SiLU of four channels for a run of tokens
    constexpr int QUADS = 2 * S / 4, RUNS = kPrepThreads / QUADS, RUN = kQ / RUNS;
    {
        const int quad = tid % QUADS, r0 = tid / QUADS * RUN;
        const int which = quad * 4 / S, col = quad * 4 % S; // 0: B, 1: C
        const int c = p.H * p.P + which * p.G * S + g * S + col;
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __ldg(reinterpret_cast<const float4 *>(p.conv_w) + c + i);
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.conv_b != nullptr)
            b = __ldg(reinterpret_cast<const float4 *>(p.conv_b + c));
        float4 win[RUN + 3];
#pragma unroll
        for (int i = 0; i < RUN + 3; ++i) { // unconditional loads: all in flight together
            const int t = min(r0 + i - 3, ntok - 1);
            const T *row = conv_row<T>(p, n, start, t0 + t);
            win[i] = load4((row != nullptr ? row : reinterpret_cast<const T *>(p.xbc) + t0 * p.xbc_stride) + c);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (p.init_conv == nullptr && t0 + r0 + i - 3 < start)
                win[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const float4 ra = win[i], rb = win[i + 1], rc = win[i + 2], rd = win[i + 3];
            float v[4];
            v[0] = fmaf(w[0].w, rd.x, fmaf(w[0].z, rc.x, fmaf(w[0].y, rb.x, fmaf(w[0].x, ra.x, b.x))));
            v[1] = fmaf(w[1].w, rd.y, fmaf(w[1].z, rc.y, fmaf(w[1].y, rb.y, fmaf(w[1].x, ra.y, b.y))));
            v[2] = fmaf(w[2].w, rd.z, fmaf(w[2].z, rc.z, fmaf(w[2].y, rb.z, fmaf(w[2].x, ra.z, b.z))));
            v[3] = fmaf(w[3].w, rd.w, fmaf(w[3].z, rc.w, fmaf(w[3].y, rb.w, fmaf(w[3].x, ra.w, b.w))));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = silu(v[k]);
            if (r0 + i >= ntok)
                v[0] = v[1] = v[2] = v[3] = 0.f;
            most = magnitude_nan(magnitude_nan(most, v[0], v[1]), v[2], v[3]);
            win[i] = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (exponent(most) == 255) { // the largest finite value
            most = 0.f;
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                const float v[4] = {win[i].x, win[i].y, win[i].z, win[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    most = fabsf(v[k]) <= 3.402823466e38f ? fmaxf(most, fabsf(v[k])) : most;
            }
        }
        uint32_t m = (uint32_t)exponent(most);
        // over the threads of B, and over those of C
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (S == 128)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
        if (lane == 0)
            largest[which][warp] = m;
        if (S == 64 ? lane == 16 : lane == 0)
            largest[S == 64 ? which : 1 - which][warp] = S == 64 ? m : 0u;
        __syncthreads();
        m = 0u;
#pragma unroll
        for (int i = 0; i < kPrepThreads / 32; ++i)
            m = max(m, largest[which][i]);
        const int e = (int)m;
        const float f = up(which == 0 ? e + 10 : e); // B: 2^3 .. 2^4
        if (r0 == 0 && col == 0) {
            const float r = down(which == 0 ? e + 10 : e);
            back[which] = r;
            scales[(id * p.G + g) * kScaleRec + which] = r;
            if (kWhole<T>)
                cb[(id * p.G + g) * (kQ * kQ) + 16 + which] = r;
        }
        uint16_t *mine = reinterpret_cast<uint16_t *>(smem) + (2 * which * kQ + r0) * LDS + col; // hi; lo is kQ rows on
        uint16_t *out = bc + ((id * p.G + g) * kQ + r0) * (4 * S) + which * 2 * S + col;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            uint2 h, l;
            split2<true>(win[i].x * f, win[i].y * f, h.x, l.x);
            split2<true>(win[i].z * f, win[i].w * f, h.y, l.y);
            *reinterpret_cast<uint2 *>(mine + i * LDS) = h;
            *reinterpret_cast<uint2 *>(mine + (kQ + i) * LDS) = l;
            if (!kWhole<T> && which == 1) { // C for the read-out
                split2<false>(win[i].x, win[i].y, h.x, l.x);
                split2<false>(win[i].z, win[i].w, h.y, l.y);
            }
            *reinterpret_cast<uint2 *>(out + i * (4 * S)) = h;
            *reinterpret_cast<uint2 *>(out + i * (4 * S) + S) = l;
        }
    }

    __syncthreads();

    // C B^T: warp w has rows 16 (w % 4) .., columns 16 (w / 4) ..
    const int mt = warp & 3, nt = warp >> 2;
    uint32_t most = 0u; // the largest product
    if (nt <= mt) {
        float acc[2][4] = {};
        const uint32_t arow = (uint32_t)((mt * 16 + (lane & 15)) * LDS + (lane >> 4) * 8) * 2;
        const uint32_t brow = (uint32_t)((nt * 16 + (lane & 7) + (lane >> 4) * 8) * LDS + ((lane >> 3) & 1) * 8) * 2;
        const uint32_t sb = smem_u32(smem);
        constexpr uint32_t PART = kQ * LDS * 2;
#pragma unroll
        for (int k = 0; k < S; k += 16) {
            uint32_t ah[4], al[4], bh[4], bl[4];
            ldmatrix4(ah, sb + 2 * PART + arow + 2 * k);
            ldmatrix4(al, sb + 3 * PART + arow + 2 * k);
            ldmatrix4(bh, sb + brow + 2 * k);
            ldmatrix4(bl, sb + PART + brow + 2 * k);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mma_f16(acc[i], ah, bh[2 * i], bh[2 * i + 1]);
                mma_f16(acc[i], ah, bl[2 * i], bl[2 * i + 1]);
                mma_f16(acc[i], al, bh[2 * i], bh[2 * i + 1]);
            }
        }
        if (!kWhole<T>) {
            const float rb = back[0], rc = back[1];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                acc[j / 4][j % 4] = acc[j / 4][j % 4] * rb * rc;
        }
        if (kWhole<T>) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(acc[j / 4][j % 4]) & 0x7fffffffu;
                most = max(most, u < 0x7f800000u ? u : 0u);
            }
        }
        float *out = cb + (id * p.G + g) * (kQ * kQ) + (mt * 16 + (lane >> 2)) * kQ + nt * 16 + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            *reinterpret_cast<float2 *>(out + 8 * j) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(out + 8 * kQ + 8 * j) = make_float2(acc[j][2], acc[j][3]);
        }
    }
    if (kWhole<T>) {
        most = __reduce_max_sync(0xffffffffu, most);
        __shared__ uint32_t products[kPrepThreads / 32];
        if (lane == 0)
            products[warp] = most;
        __syncthreads();
        if (warp == 0) {
            most = __reduce_max_sync(0xffffffffu, lane < kPrepThreads / 32 ? products[lane] : 0u);
            if (lane == 0)
                cb[(id * p.G + g) * (kQ * kQ) + 18] = __uint_as_float(most);
        }
    }
}

// ------------------------------------------------------------------- scan

// Instruction descriptor of a dense kind::f16 MMA, float16 or bfloat16 operands, float32 sums.
constexpr uint32_t idesc(bool f16, int M, int N, bool b_mn) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B[smem]^T, one instruction (K = 16), where `issue`.
__device__ __forceinline__ void mma_f16_ts_if(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                               uint32_t issue) {
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Untiled bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <typename T, int P, int S> struct Scan {
    static constexpr int kHeads = 128 / P;            // of a block
    static constexpr int kCW = S / 4;                 // state columns of a worker warpgroup
    static constexpr int kHalf = 2 * S * kQ * 2;      // bytes of a chunk's B (or C): hi, lo
    static constexpr int kSlots = 3;                  // of them in shared memory: C, B, C, B, ... in turn
    static constexpr int kGateSlots = 4;              // of the chunks' weights: in use by two, on their way for two
    static constexpr int kMBytes = kHeads * 2 * kQ * kQ * 2; // M hi of the heads, then lo
    static constexpr int kMBufs = sizeof(T) == 2 ? 2 : 1;
    static constexpr int kCbBufs = kMBufs;
    static constexpr int kCbBytes = 3 * 32 * 32 * 4;  // C B^T without its upper right quarter
    static constexpr int kRow = 128 * sizeof(T);      // 128 channels of a token
    static constexpr int kXBytes = (kQ + 3) * kRow;   // x
    static constexpr int kOffM = kSlots * kHalf, kOffCb = kOffM + kMBufs * kMBytes, kOffX = kOffCb + kCbBufs * kCbBytes,
                         kOffZ = kOffX + kXBytes;
    // the summary pass's second buffer of x: over M and C B^T where it fits, else from z's room on
    static constexpr bool kOverM = kMBufs * kMBytes + kCbBufs * kCbBytes >= kXBytes;
    static constexpr int kOffX2 = kOverM ? kOffM : kOffZ;
    static constexpr size_t kSmem = 1024 + kOffZ + (kOverM ? kQ * kRow : kXBytes);
    // TMEM columns
    static constexpr uint32_t kDH = 0;             // x' B^T, then H hi and lo of the next chunk
    static constexpr uint32_t kYI = 128;           // H C^T
    static constexpr uint32_t kYA = 192;           // x^T M^T, 64 columns per head
    static constexpr uint32_t kXP = 320;           // x' hi, lo
    static constexpr uint32_t kX = 384;            // x hi, lo
    static constexpr uint32_t kYI2 = 448;          // the other buffer of H C^T
};
constexpr int kScanThreads = 640;
constexpr uint32_t kTmemCols = 512;

// B and C slots, M buffers, buffers of C B^T and of raw x, and single barriers
enum Bar {
    kBcFull = 0, kBcEmpty = 3, kMFull = 6, kIDone = 8, kCbFull = 10, kCbEmpty = 12, kRawFull = 14, kRawEmpty = 16, kHFull = 18, kXFull, kUDone, kDrain, kZFull, kZEmpty, kTold, kBars = kTold + 4
};

// What a block works on.
struct Unit {
    int n, seg, tile, h0, nh, g;
    int start, end; // (there are fewer than 2^31 tokens)
    int c0;         // first chunk of the segment within the sequence
    int nc;         // chunks of the segment
};

template <int P>
__device__ __forceinline__ Unit unit_of(const SsmArgs &p, int segments, int tiles_per_group) {
    Unit u;
    u.tile = blockIdx.x;
    u.seg = blockIdx.y;
    u.n = blockIdx.z;
    u.g = u.tile / tiles_per_group;
    const int hpg = p.H / p.G, heads = 128 / P, first = u.tile % tiles_per_group * heads;
    u.h0 = u.g * hpg + first;
    u.nh = min(heads, hpg - first);
    int64_t start, end;
    seq_bounds(p.cu, u.n, p.N, start, end);
    u.start = (int)start;
    u.end = (int)end;
    const int64_t all = (end - start + kQ - 1) / kQ;
    u.c0 = (int)(all * u.seg / segments);
    u.nc = (int)(all * (u.seg + 1) / segments) - u.c0;
    return u;
}

struct ScanArgs {
    SsmArgs p;
    const float *cb, *masks, *gates, *scales;
    float *seg, *segdecay;
    uint32_t *status;
    int segments, fine, tiles_per_group; // the summary pass cuts every segment into `fine`
};

// Warpgroup 0: a warp that loads, a warp that issues the MMAs, two that make M.
// The other four take the same steps, each on 16 tokens of a chunk and a quarter
// of the state's columns: while the tensor core has Y and U of chunk c, they gate
// and store the output of chunk c - 1 and convolve x of chunk c + 1.  With a
// role per warpgroup instead (x, state, output) every role was one or two warps
// of a scheduler, too few to hide their own latencies.  They meet only through
// the mbarriers of what they share, so that a warp in its exponentials runs
// beside one in its splits (with two meetings of all 16 a chunk, and copies of x
// and z by their own threads, the output pass took 160 us for 145, with bfloat16
// parts throughout).
// SUMMARY: only the states of the segments but the last, from zero (the first
// from the initial state, which is also copied); no output.
template <typename T, int P, int S, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads, 1)
    ssm_scan_kernel(const __grid_constant__ CUtensorMap tbc, const __grid_constant__ CUtensorMap tcb,
                    const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tz, const ScanArgs a) {
    using K = Scan<T, P, S>;
    constexpr int NH = K::kHeads, CW = K::kCW;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ __align__(16) float gate[K::kGateSlots][NH][kGateRec], mask[K::kCbBufs][NH][kMaskRec];
    __shared__ __align__(16) float bcscale[K::kGateSlots][kScaleRec]; // what B and C of a chunk are to be multiplied with
    __shared__ float mscale[4][NH]; // and M of each head (M runs up to two chunks ahead of its reader)
    // What a row's four working threads tell each other: the exponent fields of their largest |x'| and, in the low byte
    // and halved, |x|, with 0x80 if some x is not finite.  (The summary pass: those of |x'|, in two buffers in turn.)
    __shared__ __align__(8) uint16_t told[128][4];
    __shared__ uint32_t tmem_base, abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint8_t *sm = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t b0 = smem_u32(bars);
    auto bar = [&](int i) { return b0 + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = warp & 3, wg = warp >> 2;
    const SsmArgs &p = a.p;
    const Unit u = unit_of<P>(p, SUMMARY ? a.segments * a.fine : a.segments, a.tiles_per_group);
    const int64_t id0 = first_chunk(u.start, u.n) + u.c0;
    volatile uint32_t *abort_v = &abort_flag;

    if (tid == 0) {
        for (int i = 0; i < K::kSlots; ++i) {
            mbar_init(bar(kBcFull + i), 1);
            mbar_init(bar(kBcEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kMFull + i), 2);
            mbar_init(bar(kIDone + i), 1);
        }
        mbar_init(bar(kXFull), 16);
        mbar_init(bar(kHFull), 16);
        for (int i = 0; i < 4; ++i)
            mbar_init(bar(kTold + i), 4);
        mbar_init(bar(kUDone), 1);
        mbar_init(bar(kDrain), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kCbFull + i), 1);
            mbar_init(bar(kCbEmpty + i), 2);
            mbar_init(bar(kRawFull + i), 1);
            mbar_init(bar(kRawEmpty + i), 16);
        }
        mbar_init(bar(kZFull), 1);
        mbar_init(bar(kZEmpty), 16);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_base), kTmemCols);
    if (!SUMMARY) { // the masks' zeros: what lies above their diagonal blocks is never written
        for (int i = tid; i < K::kMBufs * K::kMBytes / 16; i += kScanThreads)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + K::kOffM + 16 * i), "r"(0) : "memory");
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // Everything above may run beside the prep kernel, what follows reads its results (a short prompt 13.0 us for
    // 15.6).  A summary pass does not let the output pass set up beside it: a long document took 378 us for 350.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    // A wait that runs out (about a second, unless the caller armed less) makes every role stop at its next
    // wait.  Whichever role it was, what is in flight is waited for before the block ends: the loading thread waits
    // for its copies and the MMA warp for its MMAs on every path, because a role that gave up has not.
    auto wait = [&](int i, uint32_t parity, bool patient = false) {
        bool ok = mbar_test_wait(bar(i), parity);
        // the loads and M run ahead: they ask now and then, and leave the schedulers to the others
        for (int k = 0; patient && !ok && k < 16; ++k) {
            __nanosleep(200);
            ok = mbar_test_wait(bar(i), parity);
        }
        if (!ok)
            ok = !*abort_v && mbar_wait_sleeping(bar(i), parity, p.wait_limit);
        if (!ok) {
            *abort_v = 1;
            atomicOr(a.status, kStatusTimeout);
        }
        return ok;
    };
    auto wait_all = [&](int i, uint32_t parity, bool patient = false) { return __all_sync(0xffffffffu, wait(i, parity, patient)); };
    auto arrive = [&](int i) { // by a warp
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    auto i_done = [&](int c, bool patient = false) { return wait_all(kIDone + (c & 1), (c >> 1) & 1, patient); };
    const int tok0 = u.start + u.c0 * kQ;
    // raw x: the summary pass has two buffers
    auto raw_slot = [](int c) { return SUMMARY ? c & 1 : 0; };
    auto raw_phase = [](int c) { return (uint32_t)(SUMMARY ? c >> 1 : c) & 1; };
    const int row = 32 * q + lane;          // a worker thread's state row
    const int hl = P == 64 ? q >> 1 : 0;    // its head within the block (uniform over the warp)
    const bool live = hl < u.nh;
    const int64_t chan = (int64_t)u.h0 * P + row; // its x channel
    if (wg == 0) {
        // 128 x (64 + 4 x 104) registers are what the block was launched with (640 x 96)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 0) {
            if (lane == 0) { // ---- loads
                const int gbytes = u.nh * kGateRec * 4, mbytes = u.nh * kMaskRec * 4;
                // slots of B and C in the order of their use: C B C B ..., or B B ... in the summary
                int slot = 0, used = 0;
                uint32_t ph = 1;
                auto load_bc = [&](int y, int from) {
                    if (!wait(kBcEmpty + slot, ph, true))
                        return false;
                    mbar_arrive_expect_tx(bar(kBcFull + slot), K::kHalf);
                    for (int k = 0; k < 2 * S / 64; ++k) // boxes of 64 channels: hi, lo
                        tma_load_2d(base + slot * K::kHalf + k * 8192, &tbc, 64 * k + from, y, bar(kBcFull + slot));
                    used = used < K::kSlots ? used + 1 : K::kSlots;
                    if (++slot == K::kSlots) {
                        slot = 0;
                        ph ^= 1;
                    }
                    return true;
                };
                // In the order in which the room for them comes free: that of z of chunk c - 2 does before that of
                // x of chunk c, and both before C B^T's and B's.  Rows of x before the sequence or behind it, and of z behind it, are another
                // sequence's, or zeros; channels of absent heads are whatever lies there.  Neither is used.
                // A worker that gave up gives its room back without having waited for what was on its way there: hence
                // the look at the flag.
                int cbs = 0, raws = 0, zs = 0; // loaded so far
                bool ok = true;
                for (int c = 0; ok && c < (SUMMARY ? u.nc : u.nc + 2); ++c) {
                    const int at = SUMMARY ? u.nc - 1 - c : c; // the summary goes backwards
                    const int y = (int)(((id0 + at) * p.G + u.g) * kQ);
                    if (!SUMMARY && c < u.nc && !(ok = load_bc(y, 2 * S))) // C
                        break;
                    if (!SUMMARY && c >= 2 && p.z != nullptr) {
                        if (!(ok = wait(kZEmpty, (c & 1) ^ 1) && !*abort_v))
                            break;
                        mbar_arrive_expect_tx(bar(kZFull), kQ * K::kRow);
                        tma_load_2d(base + K::kOffZ, &tz, u.h0 * P, tok0 + (c - 2) * kQ, bar(kZFull));
                        ++zs;
                    }
                    if (c < u.nc) {
                        const int rs = raw_slot(c);
                        if (!(ok = wait(kRawEmpty + rs, raw_phase(c) ^ 1) && !*abort_v))
                            break;
                        // (x's room is free, so the weights of the chunk four before are done with too)
                        mbar_arrive_expect_tx(bar(kRawFull + rs), K::kXBytes + gbytes + kScaleRec * 4);
                        bulk_load(smem_u32(bcscale[c % K::kGateSlots]), a.scales + ((id0 + at) * p.G + u.g) * kScaleRec, kScaleRec * 4, bar(kRawFull + rs));
                        bulk_load(smem_u32(gate[c % K::kGateSlots]), a.gates + ((id0 + at) * p.H + u.h0) * kGateRec, gbytes, bar(kRawFull + rs));
                        tma_load_2d(base + (rs ? K::kOffX2 : K::kOffX), &tx, u.h0 * P, tok0 + at * kQ - 3, bar(kRawFull + rs));
                        ++raws;
                        if (!SUMMARY) {
                            const int cs = c % K::kCbBufs;
                            const uint32_t to = base + K::kOffCb + cs * K::kCbBytes;
                            if (!(ok = wait(kCbEmpty + cs, ((c / K::kCbBufs) & 1) ^ 1, true)))
                                break;
                            mbar_arrive_expect_tx(bar(kCbFull + cs), K::kCbBytes + mbytes);
                            bulk_load(smem_u32(mask[cs]), a.masks + ((id0 + c) * p.H + u.h0) * kMaskRec, mbytes, bar(kCbFull + cs));
                            tma_load_2d(to, &tcb, 0, y, bar(kCbFull + cs));
                            tma_load_2d(to + 4096, &tcb, 0, y + 32, bar(kCbFull + cs));
                            tma_load_2d(to + 8192, &tcb, 32, y + 32, bar(kCbFull + cs));
                            ++cbs;
                        }
                        ok = load_bc(y, 0); // B
                    }
                }
                // The copies in flight land: each buffer's last one, since its room was given back for it only
                // after the one before had landed.
                for (int c = max(cbs - K::kCbBufs, 0); c < cbs; ++c)
                    mbar_wait_sleeping(bar(kCbFull + c % K::kCbBufs), (c / K::kCbBufs) & 1, kDefaultWaitLimit);
                if (zs > 0)
                    mbar_wait_sleeping(bar(kZFull), (zs - 1) & 1, kDefaultWaitLimit);
                for (int c = max(raws - 2, 0); c < raws; ++c)
                    if (SUMMARY || c == raws - 1)
                        mbar_wait_sleeping(bar(kRawFull + raw_slot(c)), raw_phase(c), kDefaultWaitLimit);
                for (int k = 0; k < used; ++k) {
                    if (--slot < 0) {
                        slot = K::kSlots - 1;
                        ph ^= 1;
                    }
                    mbar_wait_sleeping(bar(kBcFull + slot), ph ^ 1, kDefaultWaitLimit);
                }
            }
        } else if (warp == 1) { // ---- MMAs
            const uint32_t issue = elect_one();
            bool ok = true;
            int slot = 0;
            uint32_t sph = 0;
            auto next_slot = [&]() {
                if (++slot == K::kSlots) {
                    slot = 0;
                    sph ^= 1;
                }
            };
            for (int c = 0; SUMMARY && c < u.nc; ++c) {
                // D[row][s] = sum_t x'[row][t] B[t][s], two buffers of x' and of D
                ok = wait_all(kBcFull + slot, sph) && wait_all(c & 1 ? kXFull : kHFull, (c >> 1) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const uint32_t bh = base + slot * K::kHalf, bl = bh + S * 128, d = tmem + K::kDH + (c & 1) * 128;
#pragma unroll
                for (int kk = 0; kk < kQ / 16; ++kk) {
                    const uint32_t xh = tmem + (c & 1 ? K::kX : K::kXP) + 8 * kk, xl = xh + 32;
                    mma_f16_ts_if(d, xh, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc(true, 128, S, true),
                                   kk > 0, issue);
                    mma_f16_ts_if(d, xh, sdesc_sw128(bl + 2048 * kk, 8192, 1024), idesc(true, 128, S, true), 1, issue);
                    mma_f16_ts_if(d, xl, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc(true, 128, S, true), 1, issue);
                }
                mma_commit_if(bar(kIDone + (c & 1)), issue);
                mma_commit_if(bar(kBcEmpty + slot), issue);
                next_slot();
            }
            // (The loops over kk are not unrolled here: the 16 working warps fill the instruction caches, and a
            // long document took 349 us for 344.)
            for (int c = 0; !SUMMARY && c < u.nc; ++c) {
                const uint32_t ph = c & 1;
                ok = wait_all(kBcFull + slot, sph) && wait_all(kHFull, ph);
                if (!ok)
                    break;
                tc_fence_after();
                // Y: D[row][t] = sum_s H[row][s] C[t][s].  H hi of 16 columns kk sits beside lo in the
                // quarter of DH that its warpgroup owns.
                const uint32_t ch = base + slot * K::kHalf, cl = ch + S * 128, yi = tmem + (ph ? K::kYI2 : K::kYI);
#pragma unroll 1
                for (int kk = 0; kk < S / 16; ++kk) {
                    const uint32_t hh = tmem + K::kDH + kk / (CW / 16) * CW + kk % (CW / 16) * 8, hlo = hh + CW / 2;
                    const uint32_t off = kk / 4 * 8192 + kk % 4 * 32;
                    mma_f16_ts_if(yi, hh, sdesc_sw128(ch + off, 16, 1024), idesc(kWhole<T>, 128, 64, false), kk > 0, issue);
                    mma_f16_ts_if(yi, hh, sdesc_sw128(cl + off, 16, 1024), idesc(kWhole<T>, 128, 64, false), 1, issue);
                    mma_f16_ts_if(yi, hlo, sdesc_sw128(ch + off, 16, 1024), idesc(kWhole<T>, 128, 64, false), 1, issue);
                }
                mma_commit_if(bar(kBcEmpty + slot), issue);
                next_slot();
                ok = wait_all(kBcFull + slot, sph);
                if (!ok)
                    break;
                tc_fence_after();
                // U: D[row][s] = sum_t x'[row][t] B[t][s], over H once the MMAs above have read it
                const uint32_t bh = base + slot * K::kHalf, bl = bh + S * 128;
#pragma unroll 1
                for (int kk = 0; kk < kQ / 16; ++kk) {
                    const uint32_t xh = tmem + K::kXP + 8 * kk, xl = xh + 32;
                    mma_f16_ts_if(tmem + K::kDH, xh, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc(true, 128, S, true), kk > 0, issue);
                    mma_f16_ts_if(tmem + K::kDH, xh, sdesc_sw128(bl + 2048 * kk, 8192, 1024), idesc(true, 128, S, true), 1, issue);
                    mma_f16_ts_if(tmem + K::kDH, xl, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc(true, 128, S, true), 1, issue);
                }
                mma_commit_if(bar(kUDone), issue);
                mma_commit_if(bar(kBcEmpty + slot), issue);
                next_slot();
                const int mb = c % K::kMBufs;
                ok = wait_all(kXFull, ph) && wait_all(kMFull + mb, (c / K::kMBufs) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                // I: D[row][64 h + t] = sum_s x[row][s] M_h[t][s]; a head's rows read their own 64 columns.
                // The masks are whole, with zeros above the diagonal: leaving the 16-blocks of zeros out by
                // smaller MMAs took 3000 cycles instead of 768 (each then waits for the one before it).
                const uint32_t mh = base + K::kOffM + mb * K::kMBytes, ml = mh + NH * kQ * kQ * 2;
#pragma unroll 1
                for (int kk = 0; kk < kQ / 16; ++kk) {
                    const uint32_t xh = tmem + K::kX + 8 * kk, xl = xh + 32;
                    mma_f16_ts_if(tmem + K::kYA, xh, sdesc_sw128(mh + 32 * kk, 16, 1024), idesc(kWhole<T>, 128, 64 * NH, false), kk > 0, issue);
                    mma_f16_ts_if(tmem + K::kYA, xh, sdesc_sw128(ml + 32 * kk, 16, 1024), idesc(kWhole<T>, 128, 64 * NH, false), 1, issue);
                    mma_f16_ts_if(tmem + K::kYA, xl, sdesc_sw128(mh + 32 * kk, 16, 1024), idesc(kWhole<T>, 128, 64 * NH, false), 1, issue);
                }
                mma_commit_if(bar(kIDone + (c & 1)), issue);
            }
            // the MMAs in flight end before their memory is given back
            mma_commit_if(bar(kDrain), issue);
            mbar_wait_sleeping(bar(kDrain), 0, kDefaultWaitLimit);
        } else { // ---- M: the decay masks times C B^T, as operands; two warps
            const int odd = lane & 1; // a thread has a row and every other group of 8 columns
            float D[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h)
                D[h] = p.D != nullptr && h < u.nh ? -kLn2 * __ldg(p.D + u.h0 + h) : 0.f;
            for (int c = 0; c < (SUMMARY ? 0 : u.nc); ++c) {
                const int mb = c % K::kMBufs, cs = c % K::kCbBufs;
                // the chunk that last had this buffer: its products are done
                if (!wait_all(kCbFull + cs, (c / K::kCbBufs) & 1, true) || (c >= K::kMBufs && !i_done(c - K::kMBufs, true)))
                    break;
                const uint32_t mbuf = base + K::kOffM + mb * K::kMBytes;
                float fm[NH], Ds[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    fm[h] = 1.f;
                    Ds[h] = D[h];
                }
                if (kWhole<T>) {
                    // the largest C . B times the largest delta, of which no mask is above 1, brought below 2^14; D, which is
                    // to be added to it, may ask for less, to be below that too
                    const uint8_t *factors = sm + K::kOffCb + cs * K::kCbBytes + 64; // (row 0, column 16)
                    const int bc = 254 - exponent(*reinterpret_cast<const float *>(factors)) - exponent(*reinterpret_cast<const float *>(factors + 4));
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        uint32_t most = 0u;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t v = __float_as_uint(mask[cs][h][128 + 2 * lane + k]) & 0x7fffffffu;
                            most = max(most, v < 0x7f800000u ? v : 0u);
                        }
                        const int m = 266 - exponent(*reinterpret_cast<const float *>(factors + 8)) - (int)(__reduce_max_sync(0xffffffffu, most) >> 23);
                        const int n = max(min(min(bc + m, 140 - exponent(D[h])), 126), -126);
                        fm[h] = pow2(n - bc);
                        Ds[h] = D[h] * pow2(n);
                        if (warp == 2 && lane == 0)
                            mscale[c & 3][h] = pow2(-n);
                    }
                }
                // 16-blocks (row, column): (0, 0) (3, 0) (3, 1) (3, 2) (3, 3) of one warp, (1, 0) (1, 1) (2, 0)
                // (2, 1) (2, 2) of the other
#pragma unroll 1 // (unrolled: 223 us for 197 at 4096 tokens, for the same reason)
                for (int blk = 0; blk < 5; ++blk) {
                    const int rb = warp == 2 ? (blk == 0 ? 0 : 3) : (blk < 2 ? 1 : 2);
                    const int i = warp == 2 ? (blk == 0 ? 0 : blk - 1) : (blk < 2 ? blk : blk - 2);
                    const int t = 16 * rb + (lane >> 1), s0 = 16 * i + 8 * odd;
                    // rows of 32 columns (the second half's from row 32 on), 16-byte pieces swizzled by the row
                    const uint8_t *cbr = sm + K::kOffCb + cs * K::kCbBytes + (t + (s0 >> 5) * 32) * 128;
                    const int piece = (s0 & 31) >> 2;
                    float v[8];
                    *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(cbr + ((piece ^ (t & 7)) << 4));
                    *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(cbr + (((piece + 1) ^ (t & 7)) << 4));
#pragma unroll
                    for (int h = 0; h < NH; ++h) { // an absent head's mask is never used
                        const float *rec = mask[cs][h];
                        const float gh = rec[t], gl = rec[64 + t], Dh = Ds[h], f = fm[h];
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
                            const float4 sh = *reinterpret_cast<const float4 *>(rec + s0 + k);
                            const float4 sl = *reinterpret_cast<const float4 *>(rec + 64 + s0 + k);
                            const float4 sd = *reinterpret_cast<const float4 *>(rec + 128 + s0 + k);
                            float m[4];
                            m[0] = ex2((gh - sh.x) + (gl - sl.x)) * ((kWhole<T> ? sd.x * f : sd.x) * v[k]);
                            m[1] = ex2((gh - sh.y) + (gl - sl.y)) * ((kWhole<T> ? sd.y * f : sd.y) * v[k + 1]);
                            m[2] = ex2((gh - sh.z) + (gl - sl.z)) * ((kWhole<T> ? sd.z * f : sd.z) * v[k + 2]);
                            m[3] = ex2((gh - sh.w) + (gl - sl.w)) * ((kWhole<T> ? sd.w * f : sd.w) * v[k + 3]);
                            if (i == rb) { // the diagonal block
                                const int at = t - s0 - k; // the diagonal's column among the four
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    m[j] = at < j ? 0.f : at == j ? m[j] + Dh : m[j];
                            }
                            split2<kWhole<T>>(m[0], m[1], hi[k / 2], lo[k / 2]);
                            split2<kWhole<T>>(m[2], m[3], hi[k / 2 + 1], lo[k / 2 + 1]);
                        }
                        // K-major rows of 128 bytes, 16-byte pieces swizzled by the row
                        const uint32_t at = mbuf + h * kQ * kQ * 2 + t * 128 + (((s0 >> 3) ^ (t & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + NH * kQ * kQ * 2), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
                    }
                }
                fence_proxy_async_smem();
                arrive(kMFull + mb);
                arrive(kCbEmpty + cs);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int part = wg - 1;
        const int64_t ys = (int64_t)p.H * P;
        float w0 = 0.f, w1 = 0.f, w2 = 0.f, w3 = 0.f, wb = 0.f;
        if (live) { // times -log2(e), as the exponential of the SiLU takes its argument
            const float4 w = __ldg(reinterpret_cast<const float4 *>(p.conv_w) + chan);
            w0 = -kLog2e * w.x; w1 = -kLog2e * w.y; w2 = -kLog2e * w.z; w3 = -kLog2e * w.w;
            if (p.conv_b != nullptr)
                wb = -kLog2e * __ldg(p.conv_b + chan);
        }
        // the state: CW columns of a row
        const int tiles = gridDim.x, slots = a.segments * a.fine;
        const int64_t unit0 = ((int64_t)u.n * tiles + u.tile) * slots; // of this sequence and tile in the workspace
        f2 h[CW / 2];
        // A state of the workspace has its 4-column pieces 128 rows apart, so that a warp's accesses are whole lines
        // (the caller's have rows of S).
        constexpr int kApart = 128 * 4;
        auto seg_at = [&](int s) { return a.seg + (unit0 + s) * 128 * S + CW * part * 128 + row * 4; };
        auto store_state = [&](float *dst, int apart) {
#pragma unroll
            for (int i = 0; i < CW / 2; i += 2)
                *reinterpret_cast<ulonglong2 *>(dst + i / 2 * apart) = make_ulonglong2(h[i], h[i + 1]);
        };
        auto add_state = [&](const float *src, int apart, float d, float f) { // h = d h + f src
            const f2 dd = pack(d, d), ff = pack(f, f);
#pragma unroll
            for (int i = 0; i < CW / 2; i += 2) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(src + i / 2 * apart);
                h[i] = fma2(ff, v.x, mul2(dd, h[i]));
                h[i + 1] = fma2(ff, v.y, mul2(dd, h[i + 1]));
            }
        };
        const int64_t gstate = (((int64_t)u.n * p.H + u.h0) * P + row) * S + CW * part;
        // When a wait gave up, the rest runs without waiting: the outputs are invalid anyway.  (It still arrives at
        // the barriers, with the flag set before: the loading thread looks at that before it loads over x or z.)
        bool ok = true;
        // x of the chunk of tokens t0 .., the i-th that is loaded: tokens 16 part ..
        auto take_x = [&](int i, int t0, float (&x)[16]) {
            const int rs = raw_slot(i);
            ok = ok && wait_all(kRawFull + rs, raw_phase(i));
            float r[19]; // tokens -3, .., 15
            const T *src = reinterpret_cast<const T *>(sm + (rs ? K::kOffX2 : K::kOffX)) + (16 * part) * 128 + row;
#pragma unroll
            for (int t = 0; t < 19; ++t)
                r[t] = to_f(src[t * 128]);
            if (part == 0 && t0 == u.start) { // before the sequence: the window
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const T *before = conv_row<T>(p, u.n, u.start, u.start - 3 + t);
                    r[t] = live && before != nullptr ? to_f(before[chan]) : 0.f;
                }
            }
            arrive(kRawEmpty + rs);
#pragma unroll
            for (int t = 0; t < 16; ++t)
                x[t] = silu_scaled(fmaf(w3, r[t + 3], fmaf(w2, r[t + 2], fmaf(w1, r[t + 1], fmaf(w0, r[t], wb)))));
            const int valid = live ? min(u.end - t0, kQ) - 16 * part : 0;
            if (valid < 16) {
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t >= valid)
                        x[t] = 0.f;
            }
        };
        // h = f h + r times the accumulator at column `at`; r (or f) of 1 costs nothing
        auto add_acc = [&](auto f, auto r, uint32_t at) {
            constexpr bool F = std::is_same<decltype(f), float>::value, R = std::is_same<decltype(r), float>::value;
            const f2 ff = pack((float)f, (float)f), rr = pack((float)r, (float)r);
#pragma unroll
            for (int i = 0; i < CW; i += 16) {
                float v[16];
                tmem_ld16(tmem + lanes + at + CW * part + i, v);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const f2 u = pack(v[2 * k], v[2 * k + 1]);
                    if (F && R)
                        h[i / 2 + k] = fma2(ff, h[i / 2 + k], mul2(rr, u));
                    else
                        h[i / 2 + k] = F ? fma2(ff, h[i / 2 + k], u) : fma2(rr, u, h[i / 2 + k]);
                }
            }
        };
        // The four warps of the same rows meet: what each told is there for the others.  In the loops they arrive when
        // they have told it and wait when they need it (with a meeting there the output pass took 147 us for 144.6).
        auto meet = [&]() { __syncwarp(); asm volatile("bar.sync %0, 128;" ::"r"(1 + q) : "memory"); };
        auto told_by_all = [&]() { return *reinterpret_cast<const uint2 *>(told[row]); };
        // x' = x w
        auto weigh = [&](const float (&x)[16], const float4 *wt, f2 (&xw)[8]) {
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                const ulonglong2 w = reinterpret_cast<const ulonglong2 *>(wt)[k / 2];
                xw[k] = mul2(pack(x[2 * k], x[2 * k + 1]), w.x);
                xw[k + 1] = mul2(pack(x[2 * k + 2], x[2 * k + 3]), w.y);
            }
        };
        auto largest = [&](const f2 (&v)[8]) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 f = unpack(v[k]);
                m = magnitude(m, f.x, f.y);
            }
            return m;
        };
        // f v in float16 parts, or v in bfloat16 parts, as an operand at column `to`
        auto put = [&](auto f16, const f2 (&v)[8], float f, uint32_t to) {
            const f2 ff = pack(f, f);
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 u = unpack(f16.value ? mul2(ff, v[k]) : v[k]);
                split2<f16.value>(u.x, u.y, hi[k], lo[k]);
            }
            tmem_st8(tmem + lanes + to + 8 * part, hi);
            tmem_st8(tmem + lanes + to + 32 + 8 * part, lo);
        };
        using whole = std::integral_constant<bool, kWhole<T>>;
#pragma unroll
        for (int i = 0; i < CW / 2; ++i)
            h[i] = 0ull;
        if (SUMMARY) {
            if (u.seg == 0) { // the output pass must not read what it may be asked to overwrite
                if (live && p.init_state != nullptr)
                    add_state(p.init_state + gstate, 4, 0.f, 1.f);
                store_state(seg_at(0), kApart);
#pragma unroll
                for (int i = 0; i < CW / 2; ++i)
                    h[i] = 0ull;
            }
            // Backwards: a chunk's share is taken times the decay from its end to the segment's.
            float decay = 1.f, r0 = 0.f, r1 = 0.f; // r0, r1: what U of the last chunk and of the one before is to be multiplied with
#pragma unroll 1
            for (int c = 0; c < u.nc; ++c) {
                float x[16];
                take_x(c, tok0 + (u.nc - 1 - c) * kQ, x);
                const float *rec = gate[c % K::kGateSlots][hl];
                const float4 *wt = reinterpret_cast<const float4 *>(rec + 16 * part);
                f2 xw[8];
                weigh(x, wt, xw);
                reinterpret_cast<uint8_t *>(told[row])[4 * (c & 1) + part] = (uint8_t)exponent(largest(xw));
                arrive(kTold + q);
                if (c >= 2) {
                    ok = ok && i_done(c - 2);
                    tc_fence_after();
                    add_acc(1, r1, K::kDH + (c & 1) * 128);
                }
                ok = ok && wait_all(kTold + q, c & 1);
                const uint32_t t = reinterpret_cast<const uint32_t *>(told[row])[c & 1];
                const int e = largest_half(t & 0x00ff00ffu, (t >> 8) & 0x00ff00ffu);
                put(std::true_type(), xw, up(e), c & 1 ? K::kX : K::kXP);
                r1 = r0;
                r0 = down(e) * bcscale[c % K::kGateSlots][0] * decay;
                decay *= live ? rec[64 + 63] : 0.f;
                tmem_wait_st();
                tc_fence_before();
                arrive(c & 1 ? kXFull : kHFull);
            }
            if (u.nc > 0) {
                ok = ok && i_done(u.nc - 1);
                tc_fence_after();
                if (u.nc > 1)
                    add_acc(1, r1, K::kDH + (u.nc & 1) * 128);
                add_acc(1, r0, K::kDH + ((u.nc - 1) & 1) * 128);
            }
            if (u.seg == 0 && live && p.init_state != nullptr)
                add_state(p.init_state + gstate, 4, 1.f, decay);
            if (ok) {
                store_state(seg_at(u.seg + 1), kApart);
                if (lane == 0 && part == 0 && (q & 1) == 0)
                    a.segdecay[(unit0 + u.seg) * 2 + hl] = decay;
            }
        } else {
            if (slots == 1) {
                if (live && p.init_state != nullptr)
                    add_state(p.init_state + gstate, 4, 0.f, 1.f);
            } else {
                // state 1 is the end of the first summary segment; each later one is its segment's own part
                const int to = u.seg * a.fine;
                add_state(seg_at(to > 0 ? 1 : 0), kApart, 0.f, 1.f);
#pragma unroll 1
                for (int s = 2; s <= to; ++s)
                    add_state(seg_at(s), kApart, a.segdecay[(unit0 + s - 1) * 2 + hl], 1.f);
            }
            // A bound of the row's |H|: the largest of the state that enters, then with every chunk gamma times it and 64
            // times the largest x' and B.  It may be far above H, but above the sum of the magnitudes that make H up only by
            // as much as x' and B vary.  The state is kept scaled by it, and x' so that U comes out in the state's units.
            float bound = 0.f;
            auto scale_state = [&](float f) {
                const f2 ff = pack(f, f);
#pragma unroll
                for (int i = 0; i < CW / 2; ++i)
                    h[i] = mul2(ff, h[i]);
            };
            if (kWhole<T>) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < CW / 2; ++i) {
                    const float2 v = unpack(h[i]);
                    m = fabsf(v.x) <= 3.402823466e38f ? fmaxf(m, fabsf(v.x)) : m;
                    m = fabsf(v.y) <= 3.402823466e38f ? fmaxf(m, fabsf(v.y)) : m;
                }
                told[row][part] = (uint16_t)exponent(m);
                meet();
                const uint2 t = told_by_all();
                bound = pow2(largest_half(t.x, t.y) - 126);
                meet();
                scale_state(up(exponent(bound)));
            }
            // kWhole: gamma in the state's units, from those before chunk c to those after it; else what its U is to be
            // multiplied with
            float step = 0.f;
            // exponent fields of the row's largest x of a chunk and of the bound before it, and the first token here whose x
            // or an earlier one is not finite, by bytes
            uint32_t now = 0u;
#pragma unroll 1
            for (int c = -1; c < u.nc; ++c) {
                const bool more = c + 1 < u.nc;
                const int t0 = tok0 + c * kQ; // of chunk c
                const int slot = c & (K::kGateSlots - 1), next = (c + 1) & (K::kGateSlots - 1);
                // -- x of chunk c + 1: tokens 16 part ..
                float x[16];
                const float4 *wt = reinterpret_cast<const float4 *>(gate[next][hl] + 16 * part);
                f2 xw[8];
                uint32_t mine = 0u; // what this thread tells, and its first x that is not finite
                if (more) {
                    take_x(c + 1, t0 + kQ, x);
                    weigh(x, wt, xw);
                    mine = (uint32_t)exponent(largest(xw)) << 8;
                    float mx = 0.f;
                    uint32_t first = 16;
#pragma unroll
                    for (int t = 0; t < 16; t += 2)
                        mx = magnitude_nan(mx, x[t], x[t + 1]);
                    if (exponent(mx) == 255) {
                        mx = 0.f;
#pragma unroll
                        for (int t = 15; t >= 0; --t) {
                            if (!(fabsf(x[t]) <= 3.402823466e38f))
                                first = t;
                            else
                                mx = fmaxf(mx, fabsf(x[t]));
                        }
                        mine |= 0x80;
                    }
                    mine |= (kWhole<T> ? (uint32_t)exponent(mx) >> 1 : 0u) | first << 24;
                }
                // -- the state entering chunk c + 1, and x' of that chunk
                if (c >= 0) {
                    ok = ok && wait_all(kUDone, c & 1);
                    tc_fence_after();
                }
                if (more) { // (all four have read what was told before, or U would not be done)
                    told[row][part] = (uint16_t)mine;
                    arrive(kTold + q);
                }
                if (c >= 0) {
                    if constexpr (kWhole<T>)
                        add_acc(step, 1, K::kDH);
                    else
                        add_acc(live ? gate[slot][hl][64 + 63] : 0.f, step, K::kDH);
                }
                uint32_t then = 0u;
                if (more) {
#pragma unroll
                    for (int i = 0; i < CW; i += 16) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float2 v = unpack(h[i / 2 + k]);
                            split2<kWhole<T>>(v.x, v.y, hi[k], lo[k]);
                        }
                        tmem_st8(tmem + lanes + K::kDH + CW * part + i / 2, hi);
                        tmem_st8(tmem + lanes + K::kDH + CW * part + CW / 2 + i / 2, lo);
                    }
                    ok = ok && wait_all(kTold + q, (c + 1) & 1);
                    const uint2 t = told_by_all();
                    const int ew = largest_half(t.x, t.y) >> 8;
                    then = mine & 0xff000000u;
                    if (kWhole<T>)
                        then |= (uint32_t)(2 * largest_half(t.x & 0x007f007fu, t.y & 0x007f007fu) + 1) | (uint32_t)exponent(bound) << 8;
                    if ((t.x | t.y) & 0x00800080u) { // some x is not finite: in an earlier part?
                        const uint32_t bad = (t.x & 0x80u) >> 7 | (t.x & 0x800000u) >> 22 | (t.y & 0x80u) >> 5 | (t.y & 0x800000u) >> 20;
                        if (bad & ((1u << part) - 1u))
                            then &= 0xffffffu;
                    }
                    const float fb = bcscale[next][0];
                    float f = up(ew);
                    if (kWhole<T>) {
                        // x' is below 2^(ew - 126) and B below 2^4 times its factor (x' of zeros must not ask for infinity)
                        const float gamma = live ? gate[next][hl][64 + 63] : 0.f, back = down(exponent(bound));
                        bound = fmaf(gamma, bound, pow2(max(ew, 24) - 116) * fb);
                        f = up(exponent(bound));
                        step = gamma * f * back;
                        f *= fb;
                    } else {
                        step = down(ew) * fb;
                    }
                    if (S == 128) // again: 128 columns leave no registers to keep it
                        weigh(x, wt, xw);
                    put(std::true_type(), xw, f, K::kXP);
                    tmem_wait_st();
                    tc_fence_before();
                    arrive(kHFull);
                }
                // -- the output of chunk c out of the accumulators, and x of chunk c + 1 as operand
                float y[16];
                if (c >= 0) {
                    ok = ok && i_done(c);
                    tc_fence_after();
                    float e[16];
                    tmem_ld16(tmem + lanes + ((c & 1) ? K::kYI2 : K::kYI) + 16 * part, y);
                    tmem_ld16(tmem + lanes + K::kYA + 64 * hl + 16 * part, e);
                    tmem_wait_ld();
                    const float ry = down((now >> 8) & 0xff) * bcscale[slot][1], rm = down(now & 0xff) * mscale[c & 3][hl];
                    const f2 ry2 = pack(ry, ry), rm2 = pack(rm, rm);
                    const ulonglong2 *eg = reinterpret_cast<const ulonglong2 *>(gate[slot][hl] + 64 + 16 * part);
                    // e^G times the state's part, and the masks' part
                    auto sum = [&](f2 f, f2 state, f2 masks) {
                        return unpack(kWhole<T> ? fma2(mul2(f, ry2), state, mul2(rm2, masks)) : fma2(f, state, masks));
                    };
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const ulonglong2 f = eg[k / 4];
                        const float2 a0 = sum(f.x, pack(y[k], y[k + 1]), pack(e[k], e[k + 1]));
                        const float2 a1 = sum(f.y, pack(y[k + 2], y[k + 3]), pack(e[k + 2], e[k + 3]));
                        y[k] = a0.x; y[k + 1] = a0.y; y[k + 2] = a1.x; y[k + 3] = a1.y;
                    }
                }
                const uint32_t bad = now >> 24;
                now = then;
                if (more) {
                    // A non-finite x would reach the tokens before it in its chunk (as 0 times it): the
                    // product takes 0 instead, and the output is set from that token on.
                    if ((now >> 24) < 16) {
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (!(fabsf(x[t]) <= 3.402823466e38f))
                                x[t] = 0.f;
                    }
                    f2 xs[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        xs[k] = pack(x[2 * k], x[2 * k + 1]);
                    put(whole(), xs, up((int)(now & 0xff)), K::kX);
                    tmem_wait_st();
                    tc_fence_before();
                    arrive(kXFull);
                }
                if (c < 0)
                    continue;
                // -- the output of chunk c: gate and store
                if (bad < 16) {
#pragma unroll
                    for (int t = 0; t < 16; ++t)
                        if (t >= (int)bad)
                            y[t] = __uint_as_float(0x7fffffffu);
                }
                // through shared memory, over z where there is one, so that a warp stores its 32 channels of 8 tokens
                // at a time (2-byte stores of a channel took 3400 cycles a chunk)
                T *yr = reinterpret_cast<T *>(smem_raw + (base - smem_u32(smem_raw)) + K::kOffZ) + (16 * part) * 128 + row;
                if (p.z != nullptr) {
                    ok = ok && wait_all(kZFull, c & 1);
#pragma unroll
                    for (int t = 0; t < 16; t += 2) {
                        const float2 v = gated(pack(y[t], y[t + 1]), pack(to_f(yr[t * 128]), to_f(yr[(t + 1) * 128])));
                        y[t] = v.x;
                        y[t + 1] = v.y;
                    }
                }
#pragma unroll
                for (int t = 0; t < 16; t += 2)
                    put2(yr + t * 128, yr + (t + 1) * 128, y[t], y[t + 1]);
                __syncwarp();
                if (live) {
                    constexpr int LANES = 2 * (int)sizeof(T), ROWS = 32 / LANES; // lanes of a row's 32 channels, rows at once
                    const int valid = min(u.end - t0, kQ) - 16 * part;
                    const int t = lane / LANES, k = lane % LANES;
                    const uint8_t *from = sm + K::kOffZ + (16 * part + t) * K::kRow + 32 * q * (int)sizeof(T) + 16 * k;
                    char *dst = reinterpret_cast<char *>(reinterpret_cast<T *>(p.y) + (int64_t)(t0 + 16 * part + t) * ys + u.h0 * P + 32 * q) + 16 * k;
#pragma unroll
                    for (int i = 0; i < 16; i += ROWS) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(from + i * K::kRow);
                        if (t + i < valid)
                            *reinterpret_cast<uint4 *>(dst + i * ys * (int64_t)sizeof(T)) = v;
                    }
                }
                if (p.z != nullptr) {
                    fence_proxy_async_smem();
                    arrive(kZEmpty);
                } else {
                    __syncwarp();
                }
            }
            if (ok && u.seg == a.segments - 1 && live && p.final_state != nullptr) {
                if (kWhole<T>)
                    scale_state(down(exponent(bound)));
                store_state(p.final_state + gstate, 4);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, kTmemCols);
    }
    // The window after the sequence, by the blocks that have its first chunk (a short sequence's first segments may
    // have none): they alone read the initial window of their x channels, and have; B's and C's was read by the
    // kernel before this one.
    if (!SUMMARY && p.final_conv != nullptr && (u.nc > 0 ? u.c0 == 0 : u.seg == 0 && u.start == u.end)) {
        for (int i = tid; i < u.nh * P; i += kScanThreads)
            final_window<T>(p, u.n, u.start, u.end, u.h0 * P + i);
        if (u.tile % a.tiles_per_group == 0) {
            for (int i = tid; i < 2 * S; i += kScanThreads)
                final_window<T>(p, u.n, u.start, u.end, p.H * P + (i < S ? u.g * S + i : p.G * S + u.g * S + i - S));
        }
    }
}

// The windows of a call without tokens.
template <typename T> __global__ void __launch_bounds__(256) ssm_final_conv_kernel(const SsmArgs p) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < p.conv_dim())
        final_window<T>(p, blockIdx.y, 0, 0, c);
}

// The cut of the sequences: segments of the output pass, and how many parts the
// summary pass before it cuts each into.  The lengths are on the device, so that
// the choice knows their sum only; of several sequences the longest is taken to
// have 2.3 times the mean (that of five cut at random).  Costs are in chunks of
// the output pass, 4.5 us: a chunk of the summary pass takes 1.3 us, a block
// about 6 us to start and end, the summary pass 13 us by itself.
// Measured with 32 heads of 64 and 128 states, 1 and the chosen number of
// segments: 1024 tokens 80 and 36 us (8); 4096, 64, 64, 64 tokens 284 and 117
// (4); 512, 512 48 and 34 (4); what it costs where the lengths are alike after
// all: four of 700 tokens 64 and 68 (4).
struct Cut {
    int segments, fine;
};
Cut choose_cut(const gdn_ssm_config *c, int64_t N, int batch) {
    const int64_t tiles = c->num_groups * (((int64_t)(c->num_heads / c->num_groups) * c->head_dim + 127) / 128);
    const int64_t L = batch > 0 ? (N / batch + kQ - 1) / kQ : 0;
    const double all = (double)tiles * ((double)N / kQ + 0.5 * batch); // chunks
    const double longest = batch > 1 ? (double)std::min<int64_t>(N, N / batch * 23 / 10) / kQ + 0.5 : (double)L;
    // `share` of the chunks in `blocks` blocks, the longest sequence's in `parts`
    const auto run = [&](double share, int64_t blocks, int parts) {
        const double one = batch > 1 ? longest / parts : (double)((L + parts - 1) / parts);
        return batch > 1 ? std::max(one, share * all / kSMs + 0.5 * one) : one * (double)((blocks + kSMs - 1) / kSMs);
    };
    Cut best{1, 1};
    double cost = 0.0;
    const int from = c->segments > 0 ? c->segments : 1, to = c->segments > 0 ? c->segments : kMaxSegments;
    for (int s = from; s <= to && (s == from || L / s >= 2); ++s) {
        const int64_t blocks = tiles * batch * s;
        for (int f = 1; f <= (s > 1 ? 4 : 1) && s * f <= kMaxSegments && (f == 1 || L / (s * f) >= 4); ++f) {
            double t = run(1.0, blocks, s) + 1.5 * (double)blocks / kSMs;
            if (s > 1)
                t += 3.0 + 0.28 * run((double)(s - 1) / s, tiles * batch * (s - 1) * f, s * f);
            if ((s == from && f == 1) || t < 0.95 * cost) {
                best = Cut{s, f};
                cost = t;
            }
        }
    }
    return best;
}

template <typename T, int P, int S> cudaError_t launch_t(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    using K = Scan<T, P, S>;
    const Layout l = layout(p.G, p.H, P, S, p.N, p.batch, p.segments * p.fine);
    char *ws = reinterpret_cast<char *>(p.ws);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);
    const int tpg = (p.H / p.G * P + 127) / 128;
    const int64_t chunks = max_chunks(p.N, p.batch);
    cudaError_t e = cudaSuccess;
    ScanArgs a{p, (float *)(ws + l.cb), (float *)(ws + l.masks), (float *)(ws + l.gates), (float *)(ws + l.scales), (float *)(ws + l.seg), (float *)(ws + l.segdecay), status, p.segments, p.fine, tpg};
    if (p.N > 0) {
        e = cudaFuncSetAttribute(ssm_prep_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem<S>());
        if (e != cudaSuccess)
            return e;
        ssm_prep_kernel<T, S><<<dim3((unsigned)chunks, p.G, 2), kPrepThreads, prep_smem<S>(), s>>>(
            p, (uint16_t *)(ws + l.bc), (float *)(ws + l.cb), (float *)(ws + l.masks), (float *)(ws + l.gates), (float *)(ws + l.scales), status);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = record_if(begin, s);
        if (e != cudaSuccess)
            return e;
        CUtensorMap tbc, tcb, tx, tz{};
        const CUtensorMapDataType type = sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
        if (!encode_2d(&tbc, ws + l.bc, 4 * S, (uint64_t)chunks * p.G * kQ, 4 * S * 2, 64, kQ, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_DATA_TYPE_FLOAT16) ||
            !encode_2d(&tcb, ws + l.cb, kQ, (uint64_t)chunks * p.G * kQ, kQ * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_2d(&tx, p.xbc, p.conv_dim(), p.N, p.xbc_stride * sizeof(T), 128, kQ + 3, CU_TENSOR_MAP_SWIZZLE_NONE, type) ||
            (p.z != nullptr && !encode_2d(&tz, p.z, (uint64_t)p.H * P, p.N, p.z_stride * sizeof(T), 128, kQ, CU_TENSOR_MAP_SWIZZLE_NONE, type)))
            return cudaErrorInvalidValue;
        const auto launch_after = [&](auto kernel, int segments) { // its start may be beside the end of the kernel before it
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(p.G * tpg, segments, p.batch);
            cfg.blockDim = dim3(kScanThreads);
            cfg.dynamicSmemBytes = K::kSmem;
            cfg.stream = s;
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at.val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            return cudaLaunchKernelEx(&cfg, kernel, tbc, tcb, tx, tz, a);
        };
        if (p.segments > 1) {
            e = cudaFuncSetAttribute(ssm_scan_kernel<T, P, S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
            if (e != cudaSuccess)
                return e;
            e = launch_after(ssm_scan_kernel<T, P, S, true>, (p.segments - 1) * p.fine);
            if (e != cudaSuccess)
                return e;
        }
        e = cudaFuncSetAttribute(ssm_scan_kernel<T, P, S, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
        if (e != cudaSuccess)
            return e;
        e = launch_after(ssm_scan_kernel<T, P, S, false>, p.segments);
        if (e == cudaSuccess)
            e = record_if(end, s);
        return e;
    }
    // no tokens: the states and windows pass through
    if (p.final_state != nullptr && p.final_state != p.init_state) {
        const size_t bytes = (size_t)p.batch * p.H * P * S * 4;
        e = p.init_state != nullptr ? cudaMemcpyAsync(p.final_state, p.init_state, bytes, cudaMemcpyDeviceToDevice, s)
                                    : cudaMemsetAsync(p.final_state, 0, bytes, s);
    }
    if (e == cudaSuccess && p.final_conv != nullptr) {
        ssm_final_conv_kernel<T><<<dim3((p.conv_dim() + 255) / 256, p.batch), 256, 0, s>>>(p);
        e = cudaGetLastError();
    }
    return e;
}

template <typename T> cudaError_t launch_ps(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    if (p.P == 64)
        return p.S == 64 ? launch_t<T, 64, 64>(p, begin, end, s) : launch_t<T, 64, 128>(p, begin, end, s);
    return p.S == 64 ? launch_t<T, 128, 64>(p, begin, end, s) : launch_t<T, 128, 128>(p, begin, end, s);
}

} // namespace

void ssm_cut(const gdn_ssm_config *c, int batch, int64_t N, int *segments, int *fine) {
    const Cut k = N > 0 ? choose_cut(c, N, batch) : Cut{1, 1};
    *segments = k.segments;
    *fine = k.fine;
}

size_t ssm_workspace_bytes(const gdn_ssm_config *c, int batch, int64_t N) {
    if (N == 0)
        return 0;
    const Cut k = choose_cut(c, N, batch);
    return layout(c->num_groups, c->num_heads, c->head_dim, c->state_dim, N, batch, k.segments * k.fine).total;
}

// The rows of B and C in the workspace are addressed by 32-bit TMA coordinates.
bool ssm_addressable(const gdn_ssm_config *c, int batch, int64_t N) {
    return max_chunks(N, batch) * c->num_groups <= INT32_MAX / kQ;
}

cudaError_t launch_ssm_prefill(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    return p.bf16 ? launch_ps<__nv_bfloat16>(p, begin, end, s) : launch_ps<float>(p, begin, end, s);
}

} // namespace gdn
