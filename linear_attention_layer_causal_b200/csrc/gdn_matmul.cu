// gdn_matmul.cu -- product of e4m3 operands with one float32 scale for each
// 1 x 128 block of a and each 128 x 128 block of w:
//     out[m][n] = sum_b sa[m][b] sw[n / 128][b] sum_{k in block b} a[m][k] w[n][k].
// The scales change with the block, so the inner sum of every block is finished
// in the tensor core's accumulator and then added, scaled, to a float32 register
// sum.  Two kernels:
//   - wide_kernel (tcgen05, operands by TMA): a 128 x BN tile of out per block.
//   - narrow_kernel (few rows of a): bound by reading w once; w goes from global
//     memory straight into the registers of mma.sync.
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sm100.cuh"
#include "gdn_tmap.h"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kSMs = 148;
constexpr int kBK = 128;              // k of a stage: one scale block
constexpr int kABytes = 128 * kBK;    // 128 rows of a
constexpr uint32_t kStatusTimeout = 1u;

// ------------------------------------------------------------------- wide

// Instruction descriptor of a dense kind::f8f6f4 MMA, e4m3 x e4m3 -> float32,
// both operands K-major.
constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]^T, one instruction (K = 32 bytes), where `issue`.
__device__ __forceinline__ void mma_f8_ss_if(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t issue) {
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(issue)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// acc.xy += s.xy * v.xy in one instruction.
__device__ __forceinline__ void fma2(unsigned long long &acc, unsigned long long s, unsigned long long v) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(s), "l"(v));
}
__device__ __forceinline__ unsigned long long pack2(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// float at `addr` of this block's shared memory, read from block `rank` of the cluster
__device__ __forceinline__ float ld_dsmem(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

template <int BN> struct Wide {
    static constexpr int kStages = BN == 256 ? 4 : 6;
    static constexpr int kStageBytes = kABytes + BN * kBK;
    static constexpr int kGroups = BN / 128;           // epilogue warpgroups
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes;
};

// 128 columns of one row from registers to out.
template <typename O>
__device__ __forceinline__ void store_row(const MatmulArgs &p, int64_t m, int64_t n0, const unsigned long long (&acc)[64],
                                          bool vec) {
    O *dst = reinterpret_cast<O *>(p.out) + m * p.out_stride + n0;
    constexpr int V = 16 / sizeof(O);
    if (vec && n0 + 128 <= p.N) {
#pragma unroll
        for (int i = 0; i < 128; i += V) {
            Vec16<O> v;
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 f = unpack2(acc[(i + k) / 2]);
                v.set(k, f.x);
                v.set(k + 1, f.y);
            }
            st16(dst + i, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const float2 f = unpack2(acc[i]);
            if (n0 + 2 * i < p.N)
                dst[2 * i] = from_f<O>(f.x);
            if (n0 + 2 * i + 1 < p.N)
                dst[2 * i + 1] = from_f<O>(f.y);
        }
    }
}

// Tile t of tiles_m x tiles_n, in bands of 16 row tiles so that the tiles in
// flight together share rows of a and of w in L2.
__device__ __forceinline__ void tile_of(int64_t t, int tiles_m, int tiles_n, int &tm, int &tn) {
    constexpr int kBand = 16;
    const int64_t per = (int64_t)kBand * tiles_n;
    const int band = (int)(t / per), first = band * kBand;
    const int rows = min(kBand, tiles_m - first);
    const int64_t r = t - band * per;
    tm = first + (int)(r % rows);
    tn = (int)(r / rows);
}

// Persistent over tiles (ks = 1), or one tile per cluster of ks blocks that
// share its blocks of k and join their sums through shared memory.
// Warp 0 loads, warp 1 issues the MMAs; the other warpgroups each take 128
// columns: a thread adds its row's finished block to 128 register sums while
// the tensor core works on the next one in the other half of TMEM.
template <int BN, typename O>
__global__ void __launch_bounds__(Wide<BN>::kThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tw, const MatmulArgs p,
                int tiles_m, int tiles_n, int ks, uint32_t *status) {
    using W = Wide<BN>;
    constexpr int ST = W::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * ST + 4];
    __shared__ uint32_t tmem_base, abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * ST, tfull = empty + 8 * ST, tempty = tfull + 16;
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    const int KB = (int)((p.K + kBK - 1) / kBK);
    const int part = ks > 1 ? (int)cluster_rank() : 0;
    const int kb0 = (int)((int64_t)KB * part / ks), kb1 = (int)((int64_t)KB * (part + 1) / ks);
    const int64_t t0 = blockIdx.x / ks, dt = gridDim.x / ks;
    volatile uint32_t *abort_v = &abort_flag;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 4 * W::kGroups);
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (blockIdx.x == 0)
            *status = 0;
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_base), 2 * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    // A wait that runs out (about a second) makes every role stop at its next
    // wait; what is in flight is waited for below, and the status word says so.
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (mbar_try_wait_spin(bar, parity))
            return true;
        if (!*abort_v && mbar_wait_bounded(bar, parity, kDefaultWaitLimit))
            return true;
        *abort_v = 1;
        atomicOr(status, kStatusTimeout);
        return false;
    };

    if (warp < 4) {
        if (BN == 256)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0 && lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            int issued = 0;
            for (int64_t t = t0; ok && t < tiles; t += dt) {
                int tm, tn;
                tile_of(t, tiles_m, tiles_n, tm, tn);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = wait(empty + 8 * s, ph ^ 1)))
                        break;
                    mbar_arrive_expect_tx(full + 8 * s, W::kStageBytes);
                    const uint32_t dst = base + s * W::kStageBytes;
                    tma_load_2d(dst, &ta, kb * kBK, tm * 128, full + 8 * s);
                    tma_load_2d(dst + kABytes, &tw, kb * kBK, tn * BN, full + 8 * s);
                    issued = issued < ST ? issued + 1 : ST;
                    if (++s == ST) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) { // the copies in flight land before the block may end
                for (int i = 0; i < issued; ++i) {
                    if (--s < 0) {
                        s = ST - 1;
                        ph ^= 1;
                    }
                    mbar_wait_bounded(full + 8 * s, ph, kDefaultWaitLimit);
                }
            }
        } else if (warp == 1) {
            const uint32_t issue = elect_one();
            int s = 0, b = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int64_t t = t0; ok && t < tiles; t += dt) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!(ok = wait(tempty + 8 * b, bph ^ 1) && wait(full + 8 * s, ph)))
                        break;
                    tc_fence_after();
                    const uint32_t at = base + s * W::kStageBytes;
#pragma unroll
                    for (int k = 0; k < kBK / 32; ++k)
                        mma_f8_ss_if(tmem + b * BN, sdesc_sw128(at + 32 * k, 16, 1024),
                                     sdesc_sw128(at + kABytes + 32 * k, 16, 1024), idesc_e4m3(128, BN), k > 0, issue);
                    mma_commit_if(empty + 8 * s, issue);
                    mma_commit_if(tfull + 8 * b, issue);
                    if (++s == ST) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (++b == 2) {
                        b = 0;
                        bph ^= 1;
                    }
                }
            }
            if (!ok) { // the MMAs in flight end before their memory is given back
                mma_commit_if(tfull + 8 * b, issue);
                mbar_wait_bounded(tfull + 8 * b, bph, kDefaultWaitLimit);
            }
        }
    } else {
        if (BN == 256)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int wg = (warp - 4) >> 2, q = warp & 3; // TMEM lanes 32 q .. of this warp
        const bool vec = ((uintptr_t)p.out & 15) == 0 && (p.out_stride * sizeof(O)) % 16 == 0;
        int b = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int64_t t = t0; ok && t < tiles; t += dt) {
            int tm, tn;
            tile_of(t, tiles_m, tiles_n, tm, tn);
            const int64_t m = (int64_t)tm * 128 + 32 * q + lane, n0 = (int64_t)tn * BN + 128 * wg;
            // rows and columns behind the end have zero operands; their scales are any valid ones
            const float *sa = p.a_scale + (m < p.M ? m : p.M - 1) * KB;
            const float *sw = p.w_scale + (n0 < p.N ? n0 / 128 : 0) * KB;
            unsigned long long acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i)
                acc[i] = 0ull;
            float next = kb0 < kb1 ? __ldg(sa + kb0) * __ldg(sw + kb0) : 0.f;
            for (int kb = kb0; kb < kb1; ++kb) {
                const unsigned long long sc = pack2(next, next);
                if (kb + 1 < kb1)
                    next = __ldg(sa + kb + 1) * __ldg(sw + kb + 1);
                ok = wait(tfull + 8 * b, bph);
                if (__any_sync(0xffffffffu, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = tmem + b * BN + 128 * wg + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float v[32];
                    tmem_ld32(at + 32 * c, v);
                    tmem_wait_ld();
                    if (c == 3) { // all of this half of TMEM is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(tempty + 8 * b);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        fma2(acc[16 * c + i], sc, pack2(v[2 * i], v[2 * i + 1]));
                }
                if (++b == 2) {
                    b = 0;
                    bph ^= 1;
                }
            }
            if (ks == 1) {
                if (ok && m < p.M)
                    store_row<O>(p, m, n0, acc, vec);
            } else {
                // own sums to the (now idle) stages; the odd row length keeps the banks apart
                float *dst = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));
#pragma unroll
                for (int i = 0; i < 64; ++i) {
                    const float2 f = unpack2(acc[i]);
                    dst[(32 * q + lane) * (BN + 1) + 128 * wg + 2 * i] = f.x;
                    dst[(32 * q + lane) * (BN + 1) + 128 * wg + 2 * i + 1] = f.y;
                }
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (ks > 1) {
        // this block sums its share of the columns over the cluster, in the order of k
        cluster_sync();
        const int64_t t = t0;
        int tm, tn;
        tile_of(t, tiles_m, tiles_n, tm, tn);
        const int cols = BN / ks, c0 = cols * part;
        for (int i = tid; i < cols * 128; i += W::kThreads) {
            const int c = i % cols, r = i / cols;
            const int64_t m = (int64_t)tm * 128 + r, n = (int64_t)tn * BN + c0 + c;
            if (m < p.M && n < p.N) {
                float v = 0.f;
                for (int k = 0; k < ks; ++k)
                    v += ld_dsmem(base + 4u * (r * (BN + 1) + c0 + c), k);
                reinterpret_cast<O *>(p.out)[m * p.out_stride + n] = from_f<O>(v);
            }
        }
        cluster_sync(); // the others may still be reading this block's sums
    }
    if (warp == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, 2 * BN);
    }
}

template <int BN, typename O> cudaError_t go_wide(const MatmulArgs &p, int tiles_m, int tiles_n, int ks, cudaStream_t s) {
    using W = Wide<BN>;
    CUtensorMap ta, tw;
    if (!encode_2d(&ta, p.a, p.K, p.M, p.K, kBK, 128, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !encode_2d(&tw, p.w, p.K, p.N, p.K, kBK, BN, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(wide_kernel<BN, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)W::kSmem);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ks > 1 ? tiles * ks : (tiles < kSMs ? tiles : kSMs)));
    cfg.blockDim = dim3(W::kThreads);
    cfg.dynamicSmemBytes = W::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, wide_kernel<BN, O>, ta, tw, p, tiles_m, tiles_n, ks,
                              reinterpret_cast<uint32_t *>(p.ws));
}

// ------------------------------------------------------------------ narrow

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kNarrowWarps = 8;

// Up to 8 NT rows of a.  A warp takes 16 rows of w and a share of the blocks of
// k: the 16 rows are the M of m16n8k32, the rows of a its N.  Both operands
// take 16 consecutive bytes of k per thread where the instruction's layout
// names 4 scattered groups of 4: the same permutation of k on both sides, so
// the sum is the same and every load is 16 bytes wide.
// wk warps of a block share 16 rows of w and join in shared memory.
template <int NT, typename O>
__global__ void __launch_bounds__(kNarrowWarps * 32) narrow_kernel(const MatmulArgs p, int wk) {
    __shared__ float sums[kNarrowWarps][NT * 4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rows = kNarrowWarps / wk; // 16-row groups of the block
    const int64_t n0 = ((int64_t)blockIdx.x * rows + warp / wk) * 16;
    const int KB = (int)((p.K + kBK - 1) / kBK), part = warp % wk;
    const int kb0 = (int)((int64_t)KB * part / wk), kb1 = (int)((int64_t)KB * (part + 1) / wk);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float acc[NT][4] = {};
    if (n0 < p.N) {
        const uint8_t *w0 = reinterpret_cast<const uint8_t *>(p.w) + (n0 + g) * p.K + 16 * t;
        const uint8_t *w1 = w0 + 8 * p.K;
        const bool in0 = n0 + g < p.N, in1 = n0 + g + 8 < p.N;
        const uint8_t *a = reinterpret_cast<const uint8_t *>(p.a) + g * p.K + 16 * t;
        const float *sw = p.w_scale + n0 / 128 * KB;
#pragma unroll 2
        for (int kb = kb0; kb < kb1; ++kb) {
            uint4 wr[2][2], ar[2][NT];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = (int64_t)kb * kBK + 64 * h;
                const bool in = k + 16 * t < p.K;
                wr[h][0] = in && in0 ? __ldcs(reinterpret_cast<const uint4 *>(w0 + k)) : zero;
                wr[h][1] = in && in1 ? __ldcs(reinterpret_cast<const uint4 *>(w1 + k)) : zero;
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    ar[h][i] = in && 8 * i + g < p.M ? __ldg(reinterpret_cast<const uint4 *>(a + 8 * i * p.K + k)) : zero;
            }
            const float s = __ldg(sw + kb);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mma_e4m3(c, wr[h][0].x, wr[h][1].x, wr[h][0].y, wr[h][1].y, ar[h][i].x, ar[h][i].y);
                    mma_e4m3(c, wr[h][0].z, wr[h][1].z, wr[h][0].w, wr[h][1].w, ar[h][i].z, ar[h][i].w);
                }
                const int m = 8 * i + 2 * t;
                const float s0 = m < p.M ? s * __ldg(p.a_scale + (int64_t)m * KB + kb) : 0.f;
                const float s1 = m + 1 < p.M ? s * __ldg(p.a_scale + (int64_t)(m + 1) * KB + kb) : 0.f;
                acc[i][0] = fmaf(s0, c[0], acc[i][0]);
                acc[i][1] = fmaf(s1, c[1], acc[i][1]);
                acc[i][2] = fmaf(s0, c[2], acc[i][2]);
                acc[i][3] = fmaf(s1, c[3], acc[i][3]);
            }
        }
    }
    if (wk > 1) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sums[warp][4 * i + e][lane] = acc[i][e];
        __syncthreads();
        if (part != 0)
            return;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                for (int k = 1; k < wk; ++k)
                    acc[i][e] += sums[warp + k][4 * i + e][lane];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t m = 8 * i + 2 * t + (e & 1), n = n0 + g + 8 * (e >> 1);
            if (m < p.M && n < p.N)
                reinterpret_cast<O *>(p.out)[m * p.out_stride + n] = from_f<O>(acc[i][e]);
        }
}

template <int NT, typename O> cudaError_t go_narrow(const MatmulArgs &p, cudaStream_t s) {
    const int64_t groups = (p.N + 15) / 16;
    const int KB = (int)((p.K + kBK - 1) / kBK);
    // enough warps to keep some 40 KB of w in flight on every SM, at least one block of k each
    int wk = 1;
    while (wk < kNarrowWarps && groups * wk < 16 * kSMs && 2 * wk <= KB)
        wk *= 2;
    const int rows = kNarrowWarps / wk;
    narrow_kernel<NT, O><<<(unsigned)((groups + rows - 1) / rows), kNarrowWarps * 32, 0, s>>>(p, wk);
    return cudaGetLastError();
}

template <typename O> cudaError_t launch_t(const MatmulArgs &p, cudaStream_t s) {
    if (p.M <= 8)
        return go_narrow<1, O>(p, s);
    if (p.M <= 16)
        return go_narrow<2, O>(p, s);
    if (p.M <= 32)
        return go_narrow<4, O>(p, s);
    const int tiles_m = (int)((p.M + 127) / 128);
    const int KB = (int)((p.K + kBK - 1) / kBK);
    const int64_t wide = (int64_t)tiles_m * ((p.N + 255) / 256);
    if (wide >= kSMs)
        return go_wide<256, O>(p, tiles_m, (int)((p.N + 255) / 256), 1, s);
    const int tiles_n = (int)((p.N + 127) / 128);
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    int ks = 1;
    while (ks < 8 && tiles * ks * 2 <= kSMs && 2 * ks <= KB)
        ks *= 2;
    return go_wide<128, O>(p, tiles_m, tiles_n, ks, s);
}

} // namespace

// The first word of the workspace is the status word of the wide kernel.
size_t matmul_workspace_bytes(int64_t, int64_t, int64_t) { return kWorkspaceHeader; }

cudaError_t launch_matmul(const MatmulArgs &p, cudaStream_t s) {
    return p.out_bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

} // namespace gdn
