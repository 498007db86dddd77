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
// memory, and the rest in warpgroups of their own: convolving x (X), the decay
// masks M (M), the state in registers (S, two of them), the output (Y).
//
// Precision: every operand of a product is the sum of two bfloat16 parts, each
// product three MMAs (the product of the two second parts is left out): about
// 2^-17 of each term, where single bfloat16 operands would put 2^-9 on the
// float32 state.  Log-decays are summed in 64 bits and M takes their difference
// as two floats: at G = -1000 one float's step alone is 6e-5.
#include "gdn_sm100.cuh"
#include "gdn_ssm.cuh"
#include "gdn_tmap.h"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kQ = 64;        // tokens of a chunk
constexpr int kGateRec = 320; // floats of a (chunk, head): G, its low part, delta, x' weight, e^G
constexpr int kSMs = 148;
constexpr uint32_t kStatusTimeout = 1u;

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

// Chunks are numbered across the batch without a prefix sum: sequence n's
// first one is cu[n] / 64 + n, which leaves at least as many numbers as it has
// chunks, and at most total / 64 + batch in all.
__device__ __forceinline__ int64_t first_chunk(int64_t start, int n) { return start / kQ + n; }
int64_t max_chunks(int64_t N, int batch) { return N / kQ + batch; }

struct Layout { // workspace offsets in bytes
    size_t bc, cb, gates, seg, segdecay, total;
};
Layout layout(int G, int H, int P, int S, int64_t N, int batch, int segments) {
    const size_t chunks = (size_t)max_chunks(N, batch);
    const size_t tiles = (size_t)G * (((size_t)(H / G) * P + 127) / 128);
    Layout l;
    l.bc = kWorkspaceHeader;
    l.cb = l.bc + round_up(chunks * G * kQ * 4 * S * 2);
    l.gates = l.cb + round_up(chunks * G * kQ * kQ * 4);
    l.seg = l.gates + round_up(chunks * H * kGateRec * 4);
    l.segdecay = l.seg + (segments > 1 ? round_up((size_t)batch * tiles * segments * 128 * S * 4) : 0);
    l.total = l.segdecay + (segments > 1 ? round_up((size_t)batch * tiles * segments * 2 * 4) : 0);
    return l;
}

// Two floats as bfloat16 parts: hi = the nearest, lo = what is left, each
// packed with `a` in the low half.
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xffff0000u);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb), "f"(ra));
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// SiLU of two values with one reciprocal: 1 / a = b / (a b).  Below -40 the
// function is taken at -40 (-1.7e-16), so that a b stays below 2^116; the
// exponents' arguments drop a NaN, so that one value's does not reach the other.
__device__ __forceinline__ void silu2(float &x, float &y) {
    const float a = 1.f + ex2(-kLog2e * fmaxf(x, -40.f)), b = 1.f + ex2(-kLog2e * fmaxf(y, -40.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
    x = max_nan(x, -40.f) * (r * b);
    y = max_nan(y, -40.f) * (r * a);
}

// The row of xbc (or of the window before the sequence) that is token t of
// sequence n, t >= start - 3; nullptr for a zero row.
template <typename T> __device__ __forceinline__ const T *conv_row(const SsmArgs &p, int n, int64_t start, int64_t t) {
    if (t >= start)
        return reinterpret_cast<const T *>(p.xbc) + t * p.xbc_stride;
    if (p.init_conv == nullptr)
        return nullptr;
    return reinterpret_cast<const T *>(p.init_conv) + ((int64_t)n * 3 + 3 + (t - start)) * p.conv_dim();
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ------------------------------------------------------------------- prep

constexpr int kPrepThreads = 256;
template <int S> constexpr size_t prep_smem() { return (size_t)4 * kQ * (S + 8) * 2; }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One chunk and group.  Writes, for the scan kernel: the rows [64][4 S] of
// B hi | B lo | C hi | C lo (zero behind the sequence's end), the 64 x 64
// products C_t . B_s of s's and t's 16-blocks with s <= t, and a gate record
// for each head of the group.
template <typename T, int S>
__global__ void __launch_bounds__(kPrepThreads) ssm_prep_kernel(const SsmArgs p, __nv_bfloat16 *bc, float *cb, float *gates,
                                                                uint32_t *status) {
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int LDS = S + 8; // row length in shared memory: rows 16 bytes apart in banks
    const int64_t id = blockIdx.x;
    const int g = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (id == 0 && g == 0 && tid == 0)
        *status = 0;
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
        __nv_bfloat16 *mine = reinterpret_cast<__nv_bfloat16 *>(smem) + (2 * which * kQ + r0) * LDS + col; // hi; lo is kQ rows on
        __nv_bfloat16 *out = bc + ((id * p.G + g) * kQ + r0) * (4 * S) + which * 2 * S + col;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const float4 ra = win[i], rb = win[i + 1], rc = win[i + 2], rd = win[i + 3];
            float v[4];
            v[0] = fmaf(w[0].w, rd.x, fmaf(w[0].z, rc.x, fmaf(w[0].y, rb.x, fmaf(w[0].x, ra.x, b.x))));
            v[1] = fmaf(w[1].w, rd.y, fmaf(w[1].z, rc.y, fmaf(w[1].y, rb.y, fmaf(w[1].x, ra.y, b.y))));
            v[2] = fmaf(w[2].w, rd.z, fmaf(w[2].z, rc.z, fmaf(w[2].y, rb.z, fmaf(w[2].x, ra.z, b.z))));
            v[3] = fmaf(w[3].w, rd.w, fmaf(w[3].z, rc.w, fmaf(w[3].y, rb.w, fmaf(w[3].x, ra.w, b.w))));
            silu2(v[0], v[1]);
            silu2(v[2], v[3]);
            if (r0 + i >= ntok)
                v[0] = v[1] = v[2] = v[3] = 0.f;
            uint2 h, l;
            split2(v[0], v[1], h.x, l.x);
            split2(v[2], v[3], h.y, l.y);
            *reinterpret_cast<uint2 *>(out + i * (4 * S)) = h;
            *reinterpret_cast<uint2 *>(out + i * (4 * S) + S) = l;
            *reinterpret_cast<uint2 *>(mine + i * LDS) = h;
            *reinterpret_cast<uint2 *>(mine + (kQ + i) * LDS) = l;
        }
    }

    // gates: a warp per head, two neighbouring tokens per lane
    const int hpg = p.H / p.G;
    for (int k = warp; k < hpg; k += kPrepThreads / 32) {
        const int h = g * hpg + k;
        const double A = -(double)expf(__ldg(p.A_log + h));
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
        float *rec = gates + (id * p.H + h) * kGateRec + 2 * lane;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double G = before + s[i];
            const float gh = (float)G;
            rec[i] = gh;
            rec[64 + i] = (float)(G - (double)gh);
            rec[128 + i] = d[i];
            rec[192 + i] = d[i] == 0.f ? 0.f : d[i] * expf((float)(all - G));
            rec[256 + i] = expf(gh);
        }
    }
    __syncthreads();

    // C B^T: warp w has rows 16 (w % 4) .., columns 32 (w / 4) ..
    const int mt = warp & 3, nh = warp >> 2;
    if (2 * nh <= mt) {
        float acc[4][4] = {};
        const uint32_t arow = (uint32_t)((mt * 16 + (lane & 15)) * LDS + (lane >> 4) * 8) * 2;
        const uint32_t brow = (uint32_t)((nh * 32 + (lane & 7) + (lane >> 4) * 8) * LDS + ((lane >> 3) & 1) * 8) * 2;
        const uint32_t sb = smem_u32(smem);
        constexpr uint32_t PART = kQ * LDS * 2;
#pragma unroll
        for (int k = 0; k < S; k += 16) {
            uint32_t ah[4], al[4];
            ldmatrix4(ah, sb + 2 * PART + arow + 2 * k);
            ldmatrix4(al, sb + 3 * PART + arow + 2 * k);
#pragma unroll
            for (int j = 0; j < 2; ++j) { // 16 columns at a time
                uint32_t bh[4], bl[4];
                ldmatrix4(bh, sb + brow + j * 16 * LDS * 2 + 2 * k);
                ldmatrix4(bl, sb + PART + brow + j * 16 * LDS * 2 + 2 * k);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma_bf16(acc[2 * j + i], ah, bh[2 * i], bh[2 * i + 1]);
                    mma_bf16(acc[2 * j + i], ah, bl[2 * i], bl[2 * i + 1]);
                    mma_bf16(acc[2 * j + i], al, bh[2 * i], bh[2 * i + 1]);
                }
            }
        }
        float *out = cb + (id * p.G + g) * (kQ * kQ) + (mt * 16 + (lane >> 2)) * kQ + nh * 32 + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            *reinterpret_cast<float2 *>(out + 8 * j) = make_float2(acc[j][0], acc[j][1]);
            *reinterpret_cast<float2 *>(out + 8 * kQ + 8 * j) = make_float2(acc[j][2], acc[j][3]);
        }
    }
}

// ------------------------------------------------------------------- scan

// Instruction descriptor of a dense kind::f16 MMA, bfloat16 operands, float32 sums.
constexpr uint32_t idesc_bf16(int M, int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] B[smem]^T, one instruction (K = 16), where `issue`.
__device__ __forceinline__ void mma_bf16_ts_if(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
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
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
// Untiled bulk copy of `bytes` (a multiple of 16, both ends 16-byte aligned).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

template <int P, int S> struct Scan {
    static constexpr int kHeads = 128 / P;      // of a block
    static constexpr int kStages = 2;           // chunks of B and C in shared memory
    static constexpr int kGateSlots = 4;
    static constexpr int kStageBytes = 4 * S * kQ * 2;
    static constexpr int kMBytes = kHeads * 2 * kQ * kQ * 2; // M hi, lo of each head; two buffers
    static constexpr size_t kSmem = 1024 + kStages * kStageBytes + 2 * kMBytes;
    // TMEM columns
    static constexpr uint32_t kDH = 0;             // x' B^T, then H hi and lo of the next chunk
    static constexpr uint32_t kYI = 128;           // H C^T
    static constexpr uint32_t kYA = 192;           // x^T M^T, 64 columns per head
    static constexpr uint32_t kXP = 320;           // x' hi, lo
    static constexpr uint32_t kX = 384;            // x hi, lo
};
constexpr int kScanThreads = 896;
constexpr uint32_t kTmemCols = 512;

// pairs (by the chunk's parity), the gate slots, and single barriers
enum Bar { kBcFull = 0, kBcEmpty = 2, kMFull = 4, kIDone = 6, kGFull = 8, kGEmpty = 12, kXpFull = 16, kXFull, kHFull, kUDone, kYEmpty, kDrain, kBars };

// What a block works on.
struct Unit {
    int n, seg, tile, h0, nh, g;
    int64_t start, end;
    int64_t c0; // first chunk of the segment within the sequence
    int nc;     // chunks of the segment
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
    seq_bounds(p.cu, u.n, p.N, u.start, u.end);
    const int64_t all = (u.end - u.start + kQ - 1) / kQ;
    u.c0 = all * u.seg / segments;
    u.nc = (int)(all * (u.seg + 1) / segments - u.c0);
    return u;
}

struct ScanArgs {
    SsmArgs p;
    const float *cb, *gates;
    float *seg, *segdecay;
    uint32_t *status;
    int segments, tiles_per_group;
};

// SUMMARY: only the states of the segments but the last, from zero (the first
// from the initial state, which is also copied); no output.
template <typename T, int P, int S, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads, 1)
    ssm_scan_kernel(const __grid_constant__ CUtensorMap tbc, const ScanArgs a) {
    using K = Scan<P, S>;
    constexpr int NH = K::kHeads, CW = S / 2; // state columns of an S warpgroup
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ __align__(16) float gate[K::kGateSlots][NH][kGateRec];
    __shared__ int bad[2][2][128]; // per half of a chunk and row: the first token with a non-finite x
    __shared__ uint32_t tmem_base, abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t mbase = base + K::kStages * K::kStageBytes;
    const uint32_t b0 = smem_u32(bars);
    auto bar = [&](int i) { return b0 + 8u * i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = warp & 3, wg = warp >> 2;
    const SsmArgs &p = a.p;
    const Unit u = unit_of<P>(p, a.segments, a.tiles_per_group);
    const int64_t id0 = first_chunk(u.start, u.n) + u.c0;
    volatile uint32_t *abort_v = &abort_flag;

    if (tid == 0) {
        const int consumers = SUMMARY ? 16 : 26;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBcFull + i), 1);
            mbar_init(bar(kBcEmpty + i), 1);
            mbar_init(bar(kMFull + i), 2);
            mbar_init(bar(kIDone + i), 1);
        }
        for (int i = 0; i < K::kGateSlots; ++i) {
            mbar_init(bar(kGFull + i), 1);
            mbar_init(bar(kGEmpty + i), consumers);
        }
        mbar_init(bar(kXpFull), 8);
        mbar_init(bar(kXFull), 8);
        mbar_init(bar(kHFull), 8);
        mbar_init(bar(kUDone), 1);
        mbar_init(bar(kYEmpty), 8);
        mbar_init(bar(kDrain), 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_base), kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    // A wait that runs out (about a second) makes every role stop at its next
    // wait; what is in flight is waited for before the block ends.
    auto wait = [&](int i, uint32_t parity) {
        const bool ok = !*abort_v && mbar_wait_sleeping(bar(i), parity, kDefaultWaitLimit);
        if (!ok) {
            *abort_v = 1;
            atomicOr(a.status, kStatusTimeout);
        }
        return ok;
    };
    auto wait_all = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)); };
    auto arrive = [&](int i) { // by a warp
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(i));
    };
    const int row = 32 * q + lane;          // state row of a thread of the X, S, Y warpgroups
    const int hl = P == 64 ? q >> 1 : 0;    // its head within the block (uniform over the warp)
    const bool live = hl < u.nh;
    const int64_t chan = (int64_t)u.h0 * P + row; // its x channel

    if (wg == 0) {
        // 128 x (64 + 2 x 64 + 2 x 104 + 2 x 48) registers, of 896 x 72 that the block was launched with
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 0 && lane == 0) { // ---- loads
            const int gbytes = u.nh * kGateRec * 4;
            int c = 0;
            for (; c < u.nc; ++c) {
                const int s = c & 1, gs = c % K::kGateSlots;
                if (!wait(kGEmpty + gs, ((c / K::kGateSlots) & 1) ^ 1))
                    break;
                mbar_arrive_expect_tx(bar(kGFull + gs), gbytes);
                bulk_load(smem_u32(gate[gs]), a.gates + ((id0 + c) * p.H + u.h0) * kGateRec, gbytes, bar(kGFull + gs));
                if (!wait(kBcEmpty + s, ((c >> 1) & 1) ^ 1)) {
                    mbar_wait_bounded(bar(kGFull + gs), (c / K::kGateSlots) & 1, kDefaultWaitLimit);
                    break;
                }
                // boxes of 64 channels: B hi, B lo, C hi, C lo
                constexpr int BOXES = (SUMMARY ? 2 : 4) * S / 64;
                mbar_arrive_expect_tx(bar(kBcFull + s), BOXES * 8192);
                const int y = (int)(((id0 + c) * p.G + u.g) * kQ);
                for (int k = 0; k < BOXES; ++k)
                    tma_load_2d(base + s * K::kStageBytes + k * 8192, &tbc, 64 * k, y, bar(kBcFull + s));
            }
            if (c < u.nc) { // gave up: the copies in flight land before the block may end
                for (int k = c - 1; k >= 0 && k >= c - 4; --k) {
                    mbar_wait_bounded(bar(kGFull + k % K::kGateSlots), (k / K::kGateSlots) & 1, kDefaultWaitLimit);
                    if (k >= c - 2)
                        mbar_wait_bounded(bar(kBcFull + (k & 1)), (k >> 1) & 1, kDefaultWaitLimit);
                }
            }
        } else if (warp == 1) { // ---- MMAs
            const uint32_t issue = elect_one();
            bool ok = true;
            for (int c = 0; c < u.nc; ++c) {
                const uint32_t st = base + (c & 1) * K::kStageBytes;
                const uint32_t bh = st, bl = st + S * 128, ch = st + 2 * S * 128, cl = st + 3 * S * 128;
                const uint32_t ph = c & 1;
                ok = wait_all(kBcFull + (c & 1), (c >> 1) & 1) && wait_all(kHFull, ph);
                if (!SUMMARY) {
                    ok = ok && wait_all(kYEmpty, ph ^ 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    // Y: D[row][t] = sum_s H[row][s] C[t][s].  H hi of 16 columns kk sits beside lo in the
                    // half of DH that its S warpgroup owns.
#pragma unroll
                    for (int kk = 0; kk < S / 16; ++kk) {
                        const uint32_t hh = tmem + K::kDH + kk / (CW / 16) * CW + kk % (CW / 16) * 8, hlo = hh + CW / 2;
                        const uint32_t off = kk / 4 * 8192 + kk % 4 * 32;
                        mma_bf16_ts_if(tmem + K::kYI, hh, sdesc_sw128(ch + off, 16, 1024), idesc_bf16(128, 64, false), kk > 0, issue);
                        mma_bf16_ts_if(tmem + K::kYI, hh, sdesc_sw128(cl + off, 16, 1024), idesc_bf16(128, 64, false), 1, issue);
                        mma_bf16_ts_if(tmem + K::kYI, hlo, sdesc_sw128(ch + off, 16, 1024), idesc_bf16(128, 64, false), 1, issue);
                    }
                }
                ok = ok && wait_all(kXpFull, ph);
                if (!ok)
                    break;
                tc_fence_after();
                // U: D[row][s] = sum_t x'[row][t] B[t][s], over H once the MMAs above have read it
#pragma unroll
                for (int kk = 0; kk < kQ / 16; ++kk) {
                    const uint32_t xh = tmem + K::kXP + 8 * kk, xl = xh + 32;
                    mma_bf16_ts_if(tmem + K::kDH, xh, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc_bf16(128, S, true), kk > 0, issue);
                    mma_bf16_ts_if(tmem + K::kDH, xh, sdesc_sw128(bl + 2048 * kk, 8192, 1024), idesc_bf16(128, S, true), 1, issue);
                    mma_bf16_ts_if(tmem + K::kDH, xl, sdesc_sw128(bh + 2048 * kk, 8192, 1024), idesc_bf16(128, S, true), 1, issue);
                }
                mma_commit_if(bar(kBcEmpty + (c & 1)), issue);
                mma_commit_if(bar(kUDone), issue);
                if (!SUMMARY) {
                    ok = wait_all(kXFull, ph) && wait_all(kMFull + (c & 1), (c >> 1) & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    // I: D[row][t] = sum_{s <= t} x[row][s] M[t][s] for each head's M; all 128 rows take part, a
                    // head's rows read their own.  Tokens before a 16-block of s take nothing from it.
                    for (int h = 0; h < u.nh; ++h) {
                        const uint32_t mh = mbase + (c & 1) * K::kMBytes + h * 2 * kQ * kQ * 2, ml = mh + kQ * kQ * 2;
#pragma unroll
                        for (int kk = 0; kk < kQ / 16; ++kk) {
                            const uint32_t xh = tmem + K::kX + 8 * kk, xl = xh + 32;
                            const uint32_t d = tmem + K::kYA + 64 * h + 16 * kk, off = 2048 * kk + 32 * kk;
                            mma_bf16_ts_if(d, xh, sdesc_sw128(mh + off, 16, 1024), idesc_bf16(128, 64 - 16 * kk, false), kk > 0, issue);
                            mma_bf16_ts_if(d, xh, sdesc_sw128(ml + off, 16, 1024), idesc_bf16(128, 64 - 16 * kk, false), 1, issue);
                            mma_bf16_ts_if(d, xl, sdesc_sw128(mh + off, 16, 1024), idesc_bf16(128, 64 - 16 * kk, false), 1, issue);
                        }
                    }
                    mma_commit_if(bar(kIDone + (c & 1)), issue);
                }
            }
            if (!ok) { // the MMAs in flight end before their memory is given back
                mma_commit_if(bar(kDrain), issue);
                mbar_wait_bounded(bar(kDrain), 0, kDefaultWaitLimit);
            }
        } else if (warp >= 2) { // ---- M: the decay masks times C B^T, as operands; two warps
            const int odd = lane & 1; // a thread has a row and every other group of 8 columns
            const float D0 = p.D != nullptr ? __ldg(p.D + u.h0) : 0.f;
            const float D1 = p.D != nullptr && u.nh > 1 ? __ldg(p.D + u.h0 + 1) : 0.f;
            for (int c = 0; c < (SUMMARY ? 0 : u.nc); ++c) {
                const int gs = c % K::kGateSlots;
                // 16-blocks of rows 0 and 3, or 1 and 2, columns up to the end of the row's block: (row, column)
                // blocks (0, 0) (3, 0) (3, 1) (3, 2) (3, 3) of one warp, (1, 0) (1, 1) (2, 0) (2, 1) (2, 2) of the other
                auto block_of = [&](int k, int &rb, int &i) {
                    rb = warp == 2 ? (k == 0 ? 0 : 3) : (k < 2 ? 1 : 2);
                    i = warp == 2 ? (k == 0 ? 0 : k - 1) : (k < 2 ? k : k - 2);
                };
                const float *cbc = a.cb + ((id0 + c) * p.G + u.g) * (kQ * kQ) + (lane >> 1) * kQ + 8 * odd;
                auto load_cb = [&](int k, float (&v)[8]) {
                    int rb, i;
                    block_of(k, rb, i);
                    const float4 *src = reinterpret_cast<const float4 *>(cbc + 16 * rb * kQ + 16 * i);
                    *reinterpret_cast<float4 *>(v) = __ldg(src);
                    *reinterpret_cast<float4 *>(v + 4) = __ldg(src + 1);
                };
                float v[8], next[8];
                load_cb(0, v);
                // I of two chunks ago has read this buffer
                if (!wait_all(kGFull + gs, (c / K::kGateSlots) & 1) || (c > 1 && !wait_all(kIDone + (c & 1), ((c >> 1) & 1) ^ 1)))
                    break;
                const uint32_t mbuf = mbase + (c & 1) * K::kMBytes;
#pragma unroll 1
                for (int blk = 0; blk < 5; ++blk) {
                    int rb, i;
                    block_of(blk, rb, i);
                    if (blk < 4)
                        load_cb(blk + 1, next);
                    const int t = 16 * rb + (lane >> 1), s0 = 16 * i + 8 * odd;
#pragma unroll 1
                    for (int h = 0; h < u.nh; ++h) {
                        const float *rec = gate[gs][h];
                        const float gh = rec[t], gl = rec[64 + t];
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 8; k += 4) {
                            const float4 sh = *reinterpret_cast<const float4 *>(rec + s0 + k);
                            const float4 sl = *reinterpret_cast<const float4 *>(rec + 64 + s0 + k);
                            const float4 sd = *reinterpret_cast<const float4 *>(rec + 128 + s0 + k);
                            float m[4];
                            m[0] = ex2(kLog2e * ((gh - sh.x) + (gl - sl.x))) * sd.x * v[k];
                            m[1] = ex2(kLog2e * ((gh - sh.y) + (gl - sl.y))) * sd.y * v[k + 1];
                            m[2] = ex2(kLog2e * ((gh - sh.z) + (gl - sl.z))) * sd.z * v[k + 2];
                            m[3] = ex2(kLog2e * ((gh - sh.w) + (gl - sl.w))) * sd.w * v[k + 3];
                            if (i == rb) { // the diagonal block
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    if (s0 + k + j > t)
                                        m[j] = 0.f;
                                    if (s0 + k + j == t)
                                        m[j] += h == 0 ? D0 : D1;
                                }
                            }
                            split2(m[0], m[1], hi[k / 2], lo[k / 2]);
                            split2(m[2], m[3], hi[k / 2 + 1], lo[k / 2 + 1]);
                        }
                        // K-major rows of 128 bytes, 16-byte pieces swizzled by the row
                        const uint32_t at = mbuf + h * 2 * kQ * kQ * 2 + t * 128 + (((s0 >> 3) ^ (t & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]) : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kQ * kQ * 2), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]) : "memory");
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = next[k];
                }
                fence_proxy_async_smem();
                arrive(kMFull + (c & 1));
                arrive(kGEmpty + gs);
            }
        }
    } else if (wg < 3) { // ---- X: convolution of x, then x' and x as operands; 32 tokens of a chunk per warpgroup
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const int half = wg - 1;
        float w0 = 0.f, w1 = 0.f, w2 = 0.f, w3 = 0.f, wb = 0.f, win[3] = {0.f, 0.f, 0.f};
        if (live) {
            const float4 w = __ldg(reinterpret_cast<const float4 *>(p.conv_w) + chan);
            w0 = w.x; w1 = w.y; w2 = w.z; w3 = w.w;
            if (p.conv_b != nullptr)
                wb = __ldg(p.conv_b + chan);
            if (u.nc > 0 && half == 0) {
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const T *src = conv_row<T>(p, u.n, u.start, u.start + u.c0 * kQ - 3 + i);
                    win[i] = src != nullptr ? to_f(src[chan]) : 0.f;
                }
            }
        }
        for (int c = 0; c < u.nc; ++c) {
            const int64_t t0 = u.start + (u.c0 + c) * kQ;
            const int ntok = (int)(u.end - t0 < kQ ? u.end - t0 : kQ), last = ntok - 1;
            // a half without a head of its own reads the other's channels, and takes none of them
            const T *src = reinterpret_cast<const T *>(p.xbc) + t0 * p.xbc_stride + (live ? chan : chan - 64);
            float x[32], r[3];
            {
                // unconditional loads, the last token in the place of those behind it: all are in flight together
                T raw[35];
#pragma unroll
                for (int t = 0; t < 35; ++t) {
                    const int k = 32 * half + t - 3;
                    raw[t] = src[(int64_t)(k < last ? k < 0 && c == 0 ? 0 : k : last) * p.xbc_stride];
                }
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    r[t] = half == 0 && c == 0 ? win[t] : to_f(raw[t]);
#pragma unroll
                for (int t = 0; t < 32; ++t)
                    x[t] = to_f(raw[t + 3]);
            }
            { // the next chunk's channels to L2, a 128-byte line per thread
                const int t = kQ + (tid & 63), line = (tid >> 6) & 3;
                if (t0 + t < u.end && line < (int)sizeof(T))
                    prefetch_l2(src - row + line * (128 / sizeof(T)) + t * p.xbc_stride);
            }
            float zero = 0.f;
#pragma unroll
            for (int t = 0; t < 32; t += 2) {
                const float ra = x[t], rb = x[t + 1];
                x[t] = fmaf(w3, ra, fmaf(w2, r[2], fmaf(w1, r[1], fmaf(w0, r[0], wb))));
                x[t + 1] = fmaf(w3, rb, fmaf(w2, ra, fmaf(w1, r[2], fmaf(w0, r[1], wb))));
                r[0] = r[2];
                r[1] = ra;
                r[2] = rb;
                silu2(x[t], x[t + 1]);
            }
            const int valid = live ? ntok - 32 * half : 0;
#pragma unroll
            for (int t = 0; t < 32; ++t) {
                if (t >= valid)
                    x[t] = 0.f;
                zero = fmaf(x[t], 0.f, zero);
            }
            const int gs = c % K::kGateSlots;
            if (!wait_all(kGFull + gs, (c / K::kGateSlots) & 1) || !wait_all(kUDone, (c & 1) ^ 1))
                break;
            tc_fence_after();
            const float4 *wt = reinterpret_cast<const float4 *>(gate[gs][hl] + 192 + 32 * half);
#pragma unroll
            for (int t = 0; t < 32; t += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 w = wt[(t + k) / 4];
                    split2(x[t + k] * w.x, x[t + k + 1] * w.y, hi[k / 2], lo[k / 2]);
                    split2(x[t + k + 2] * w.z, x[t + k + 3] * w.w, hi[k / 2 + 1], lo[k / 2 + 1]);
                }
                tmem_st8(tmem + lanes + K::kXP + 16 * half + t / 2, hi);
                tmem_st8(tmem + lanes + K::kXP + 32 + 16 * half + t / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(kXpFull);
            arrive(kGEmpty + gs);
            if (SUMMARY)
                continue;
            if (c > 0 && !wait_all(kIDone + ((c - 1) & 1), ((c - 1) >> 1) & 1))
                break;
            tc_fence_after();
            // A non-finite x would reach the tokens before it in its 16-block (as 0 times it): the
            // product takes 0 instead, and the output is set from that token on.
            int first = kQ;
            if (zero != 0.f) {
#pragma unroll
                for (int t = 31; t >= 0; --t)
                    if (!(fabsf(x[t]) <= 3.402823466e38f)) {
                        first = 32 * half + t;
                        x[t] = 0.f;
                    }
            }
            bad[c & 1][half][row] = first;
#pragma unroll
            for (int t = 0; t < 32; t += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    split2(x[t + 2 * k], x[t + 2 * k + 1], hi[k], lo[k]);
                tmem_st8(tmem + lanes + K::kX + 16 * half + t / 2, hi);
                tmem_st8(tmem + lanes + K::kX + 32 + 16 * half + t / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(kXFull);
        }
    } else if (wg < 5) { // ---- S: the state, CW columns of a row per thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int half = wg - 3;
        const int tiles = gridDim.x;
        float h[CW];
        auto seg_at = [&](int s) { // state `s` of this sequence and tile in the workspace
            return a.seg + ((((int64_t)u.n * tiles + u.tile) * a.segments + s) * 128 + row) * S + CW * half;
        };
        auto load_state = [&](const float *src) {
#pragma unroll
            for (int i = 0; i < CW; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src + i);
                h[i] = v.x; h[i + 1] = v.y; h[i + 2] = v.z; h[i + 3] = v.w;
            }
        };
        auto store_state = [&](float *dst) {
#pragma unroll
            for (int i = 0; i < CW; i += 4)
                *reinterpret_cast<float4 *>(dst + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
        };
        const int64_t gstate = (((int64_t)u.n * p.H + u.h0) * P + row) * S + CW * half;
#pragma unroll
        for (int i = 0; i < CW; ++i)
            h[i] = 0.f;
        if (SUMMARY || a.segments == 1) {
            if (u.seg == 0 && live && p.init_state != nullptr)
                load_state(p.init_state + gstate);
            if (SUMMARY && u.seg == 0)
                store_state(seg_at(0)); // the output pass must not read what it may be asked to overwrite
        } else {
            // state 1 is the end of segment 0; each later one is its segment's own part
            load_state(seg_at(u.seg > 0 ? 1 : 0));
            for (int s = 2; s <= u.seg; ++s) {
                const float d = a.segdecay[(((int64_t)u.n * tiles + u.tile) * a.segments + s - 1) * 2 + hl];
                const float *src = seg_at(s);
#pragma unroll
                for (int i = 0; i < CW; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + i);
                    h[i] = fmaf(d, h[i], v.x);
                    h[i + 1] = fmaf(d, h[i + 1], v.y);
                    h[i + 2] = fmaf(d, h[i + 2], v.z);
                    h[i + 3] = fmaf(d, h[i + 3], v.w);
                }
            }
        }
        float decay = 1.f;
        bool ok = true;
        for (int c = 0; c <= u.nc; ++c) {
            if (c > 0) {
                const int gs = (c - 1) % K::kGateSlots;
                ok = wait_all(kGFull + gs, ((c - 1) / K::kGateSlots) & 1);
                const float gamma = live ? gate[gs][hl][256 + 63] : 0.f;
                decay *= gamma;
                arrive(kGEmpty + gs);
                ok = ok && wait_all(kUDone, (c - 1) & 1);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < CW; i += 16) {
                    float v[2][8];
                    tmem_ld8(tmem + lanes + K::kDH + CW * half + i, v[0]);
                    tmem_ld8(tmem + lanes + K::kDH + CW * half + i + 8, v[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        h[i + k] = fmaf(gamma, h[i + k], v[k / 8][k % 8]);
                }
            }
            if (c == u.nc)
                break;
            if (!SUMMARY) {
#pragma unroll
                for (int i = 0; i < CW; i += 16) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        split2(h[i + 2 * k], h[i + 2 * k + 1], hi[k], lo[k]);
                    tmem_st8(tmem + lanes + K::kDH + CW * half + i / 2, hi);
                    tmem_st8(tmem + lanes + K::kDH + CW * half + CW / 2 + i / 2, lo);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            arrive(kHFull);
        }
        if (ok && SUMMARY) {
            store_state(seg_at(u.seg + 1));
            if (lane == 0 && half == 0 && (q & 1) == 0)
                a.segdecay[(((int64_t)u.n * tiles + u.tile) * a.segments + u.seg) * 2 + hl] = decay;
        } else if (ok && u.seg == a.segments - 1 && live && p.final_state != nullptr) {
            store_state(p.final_state + gstate);
        }
    } else { // ---- Y: the output; 32 tokens of a chunk per warpgroup
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        const int half = wg - 5;
        const int64_t ys = (int64_t)p.H * P;
        for (int c = 0; c < (SUMMARY ? 0 : u.nc); ++c) {
            const int64_t t0 = u.start + (u.c0 + c) * kQ;
            const int ntok = (int)(u.end - t0 < kQ ? u.end - t0 : kQ), last = ntok - 1;
            const int gs = c % K::kGateSlots;
            const T *zc = reinterpret_cast<const T *>(p.z) + t0 * p.z_stride + (live ? chan : chan - 64);
            if (p.z != nullptr) { // the next chunk's gate inputs to L2, a 128-byte line per thread
                const int t = kQ + (tid & 63), line = (tid >> 6) & 3;
                if (t0 + t < u.end && line < (int)sizeof(T))
                    prefetch_l2(zc - row + line * (128 / sizeof(T)) + t * p.z_stride);
            }
            T raw[8]; // z of 8 tokens, on its way while what comes before it is worked on
            auto load_z = [&](int first) {
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    raw[t] = zc[(int64_t)(first + t < last ? first + t : last) * p.z_stride];
            };
            if (p.z != nullptr)
                load_z(32 * half);
            if (!wait_all(kGFull + gs, (c / K::kGateSlots) & 1) || !wait_all(kIDone + (c & 1), (c >> 1) & 1))
                break;
            tc_fence_after();
            int nf = bad[c & 1][0][row];
            if (half == 1)
                nf = min(nf, bad[c & 1][1][row]);
#pragma unroll 1
            for (int first = 32 * half; first < 32 * half + 32; first += 8) {
                float y[8], e[8];
                tmem_ld8(tmem + lanes + K::kYI + first, y);
                tmem_ld8(tmem + lanes + K::kYA + 64 * hl + first, e);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(gate[gs][hl] + 256 + first + k);
                    y[k] = fmaf(f.x, y[k], e[k]);
                    y[k + 1] = fmaf(f.y, y[k + 1], e[k + 1]);
                    y[k + 2] = fmaf(f.z, y[k + 2], e[k + 2]);
                    y[k + 3] = fmaf(f.w, y[k + 3], e[k + 3]);
                }
                if (first == 32 * half + 24) {
                    tc_fence_before();
                    arrive(kYEmpty);
                    arrive(kGEmpty + gs);
                }
                if (p.z != nullptr) {
#pragma unroll
                    for (int t = 0; t < 8; t += 2) {
                        float za = to_f(raw[t]), zb = to_f(raw[t + 1]);
                        silu2(za, zb);
                        y[t] *= za;
                        y[t + 1] *= zb;
                    }
                    if (first < 32 * half + 24)
                        load_z(first + 8);
                }
                if (nf < first + 8) {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (first + t >= nf)
                            y[t] = __uint_as_float(0x7fffffffu);
                }
                T *dst = reinterpret_cast<T *>(p.y) + (t0 + first) * ys + chan;
                const int valid = live ? ntok - first : 0;
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    if (t < valid)
                        dst[t * ys] = from_f<T>(y[t]);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// The last three pre-conv rows of [initial window; sequence].
template <typename T> __global__ void __launch_bounds__(256) ssm_final_conv_kernel(const SsmArgs p) {
    const int C = p.conv_dim(), c = blockIdx.x * 256 + threadIdx.x, n = blockIdx.y;
    if (c >= C)
        return;
    int64_t s, e;
    seq_bounds(p.cu, n, p.N, s, e);
    T v[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const T *row = conv_row<T>(p, n, s, e - 3 + i);
        v[i] = row != nullptr ? row[c] : from_f<T>(0.f);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        reinterpret_cast<T *>(p.final_conv)[((int64_t)n * 3 + i) * C + c] = v[i];
}

// The library's choice of segments per sequence, from the time of the busiest
// SM in chunks: a block's pass over its chunks, and the summary pass before it
// at about half of that a chunk.
int choose_segments(int G, int H, int P, int64_t N, int batch) {
    const int64_t units = (int64_t)batch * G * ((int64_t)(H / G) * P + 127) / 128;
    const int64_t L = (N / (batch > 0 ? batch : 1) + kQ - 1) / kQ;
    int best = 1;
    double cost = 0;
    for (int s = 1; s <= kMaxSegments && (s == 1 || L / s >= 4); ++s) {
        const int64_t len = (L + s - 1) / s;
        const double t = (double)((units * s + kSMs - 1) / kSMs) * len +
                         (s > 1 ? 3.0 + 0.5 * (double)((units * (s - 1) + kSMs - 1) / kSMs) * len : 0.0);
        if (s == 1 || t < 0.95 * cost) {
            best = s;
            cost = t;
        }
    }
    return best;
}

template <typename T, int P, int S> cudaError_t launch_t(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    using K = Scan<P, S>;
    const int segments = p.N > 0 ? p.segments : 1;
    const Layout l = layout(p.G, p.H, P, S, p.N, p.batch, segments);
    char *ws = reinterpret_cast<char *>(p.ws);
    uint32_t *status = reinterpret_cast<uint32_t *>(ws);
    const int tpg = (p.H / p.G * P + 127) / 128;
    const int64_t chunks = max_chunks(p.N, p.batch);
    cudaError_t e = cudaSuccess;
    ScanArgs a{p, (float *)(ws + l.cb), (float *)(ws + l.gates), (float *)(ws + l.seg), (float *)(ws + l.segdecay), status, segments, tpg};
    if (p.N > 0) {
        e = cudaFuncSetAttribute(ssm_prep_kernel<T, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem<S>());
        if (e != cudaSuccess)
            return e;
        ssm_prep_kernel<T, S><<<dim3((unsigned)chunks, p.G), kPrepThreads, prep_smem<S>(), s>>>(
            p, (__nv_bfloat16 *)(ws + l.bc), (float *)(ws + l.cb), (float *)(ws + l.gates), status);
        e = record_if(begin, s);
        if (e != cudaSuccess)
            return e;
        CUtensorMap tbc;
        if (!encode_2d(&tbc, ws + l.bc, 4 * S, (uint64_t)chunks * p.G * kQ, 4 * S * 2, 64, kQ, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_DATA_TYPE_BFLOAT16))
            return cudaErrorInvalidValue;
        if (segments > 1) {
            e = cudaFuncSetAttribute(ssm_scan_kernel<T, P, S, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
            if (e != cudaSuccess)
                return e;
            ssm_scan_kernel<T, P, S, true><<<dim3(p.G * tpg, segments - 1, p.batch), kScanThreads, K::kSmem, s>>>(tbc, a);
        }
        e = cudaFuncSetAttribute(ssm_scan_kernel<T, P, S, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::kSmem);
        if (e != cudaSuccess)
            return e;
        ssm_scan_kernel<T, P, S, false><<<dim3(p.G * tpg, segments, p.batch), kScanThreads, K::kSmem, s>>>(tbc, a);
        e = cudaGetLastError();
        if (e == cudaSuccess)
            e = record_if(end, s);
    } else if (p.final_state != nullptr && p.final_state != p.init_state) { // no tokens: the states pass through
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

int ssm_segments(const gdn_ssm_config *c, int batch, int64_t N) {
    if (N == 0)
        return 1;
    return c->segments > 0 ? c->segments : choose_segments(c->num_groups, c->num_heads, c->head_dim, N, batch);
}

size_t ssm_workspace_bytes(const gdn_ssm_config *c, int batch, int64_t N) {
    if (N == 0)
        return 0;
    return layout(c->num_groups, c->num_heads, c->head_dim, c->state_dim, N, batch, ssm_segments(c, batch, N)).total;
}

// The rows of B and C in the workspace are addressed by 32-bit TMA coordinates.
bool ssm_addressable(const gdn_ssm_config *c, int batch, int64_t N) {
    return max_chunks(N, batch) * c->num_groups <= INT32_MAX / kQ;
}

cudaError_t launch_ssm_prefill(const SsmArgs &p, cudaEvent_t begin, cudaEvent_t end, cudaStream_t s) {
    return p.bf16 ? launch_ps<__nv_bfloat16>(p, begin, end, s) : launch_ps<float>(p, begin, end, s);
}

} // namespace gdn
