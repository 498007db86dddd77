// gdn_matmul.cu -- product of e4m3 operands with one float32 scale for each
// 1 x 128 block of a and each 128 x 128 block of w:
//     out[m][n] = sum_b sa[m][b] sw[n / 128][b] sum_{k in block b} a[m][k] w[n][k].
// The scales change with the block, so the inner sum of every block is finished
// in the tensor core's accumulator and then added, scaled, to a float32 register
// sum.  Both kernels are one loop over blocks of k with five roles: a TMA warp,
// an MMA warp (tcgen05, e4m3), two warps that stage the scales, and warpgroups
// that read each finished block from TMEM and add it.
//   - wide_kernel: 128 rows of a by 256 rows of w, persistent over tiles.
//   - thin_kernel: 128 rows of w by BN <= 128 rows of a, the k axis split over
//     a cluster; for few rows of a, where reading w once is the bound.
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_per_device.h"
#include "gdn_sm100.cuh"
#include "gdn_tmap.h"

namespace gdn {
namespace {

using namespace sm100;

constexpr int kSMs = 148;
constexpr int kBK = 128;              // k of a stage: one scale block
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
// The address in block `rank` of the cluster of this block's shared-memory address.
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_dsmem(uint32_t addr, unsigned long long x, unsigned long long y) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(x), "l"(y) : "memory");
}

// Scales of four blocks of k at a time, staged in shared memory by two warps.
constexpr int kScaleSlots = 4;

// Barriers and roles shared by the two kernels.  A wait that runs out (about a
// second) makes every role stop at its next wait, and the status word says so.
// Whichever role it was, what is in flight is waited for before the block ends:
// the loading thread waits for its copies and the MMA warp for its MMAs on
// every path, because a role that gave up has not.
struct Waiter {
    volatile uint32_t *abort_flag;
    uint32_t *status;
    long long limit;
    // A bound that was armed may be shorter than the sleep of a try_wait.
    __device__ bool polled(uint32_t bar, uint32_t parity) const {
        for (const long long t0 = clock64(); clock64() - t0 <= limit;)
            if (mbar_test_wait(bar, parity))
                return true;
        return false;
    }
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_test_wait(bar, parity))
            return true;
        if (!*abort_flag && (limit >= kDefaultWaitLimit ? mbar_wait_bounded(bar, parity, limit) : polled(bar, parity)))
            return true;
        *abort_flag = 1;
        atomicOr(status, kStatusTimeout);
        return false;
    }
};

// Position in a ring of N slots and the parity of its current round.
template <int N> struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            ph ^= 1;
        }
    }
    __device__ __forceinline__ void back() {
        if (--i < 0) {
            i = N - 1;
            ph ^= 1;
        }
    }
};

// TMA role, one thread: the blocks kb0 .. kb1 of the rows at ra (RA of them) and rw (RW).
template <int ST, int RA, int RW>
__device__ __forceinline__ bool load_blocks(const Waiter &wait, Ring<ST> &r, int &issued, uint32_t base, uint32_t full,
                                            uint32_t empty, const CUtensorMap *ta, const CUtensorMap *tw, int ra, int rw,
                                            int kb0, int kb1) {
    for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait(empty + 8 * r.i, r.ph ^ 1))
            return false;
        mbar_arrive_expect_tx(full + 8 * r.i, (RA + RW) * kBK);
        const uint32_t dst = base + r.i * ((RA + RW) * kBK);
        tma_load_2d(dst, ta, kb * kBK, ra, full + 8 * r.i);
        tma_load_2d(dst + RA * kBK, tw, kb * kBK, rw, full + 8 * r.i);
        issued = issued < ST ? issued + 1 : ST;
        r.next();
    }
    return true;
}

// After the last load, or a failed wait: the copies in flight land before the
// block may end.  The thread sleeps: with polls, one row of 12352 x 2048 took 9.2
// us for 8.7.
template <int ST> __device__ __forceinline__ void drain_loads(Ring<ST> r, int issued, uint32_t full) {
    for (int i = 0; i < issued; ++i) {
        r.back();
        mbar_wait_sleeping(full + 8 * r.i, r.ph, kDefaultWaitLimit);
    }
}

// Scale role, two warps: scales of RS consecutive rows of `sc` (row length KB, the last valid row for
// rows behind `rows`), four blocks at a time, as [slot][4][RS] floats, each times `w` of that block
// where w is given.
template <int RS>
__device__ __forceinline__ bool load_scales(const Waiter &wait, Ring<kScaleSlots> &r, float *ring, uint32_t sfull,
                                            uint32_t sempty, const float *sc, int64_t first, int64_t rows, int KB,
                                            const float *w, int kb0, int kb1, int who, int lane) {
    for (int kb = kb0; kb < kb1; kb += 4) {
        const bool ok = wait(sempty + 8 * r.i, r.ph ^ 1);
        if (__any_sync(0xffffffffu, !ok))
            return false;
        float *dst = ring + r.i * 4 * RS;
        for (int row = 32 * who + lane; row < RS; row += 64) {
            const int64_t at = first + row < rows ? first + row : rows - 1;
            const float *src = sc + at * KB + kb;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (kb + 4 <= kb1 && ((uintptr_t)src & 15) == 0) {
                *reinterpret_cast<float4 *>(v) = __ldg(reinterpret_cast<const float4 *>(src));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (kb + j < kb1)
                        v[j] = __ldg(src + j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                dst[j * RS + row] = w != nullptr && kb + j < kb1 ? v[j] * __ldg(w + kb + j) : v[j];
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(sfull + 8 * r.i);
        r.next();
    }
    return true;
}

// MMA role, one warp: D of buffer b (BN columns) = the block's RA x 128 by RW x 128 product.
template <int ST, int NB, int RA, int RW, int BN, bool A_IS_W>
__device__ __forceinline__ bool issue_blocks(const Waiter &wait, Ring<ST> &r, Ring<NB> &d, uint32_t base, uint32_t full,
                                             uint32_t empty, uint32_t tfull, uint32_t tempty, uint32_t tmem, int blocks,
                                             uint32_t issue) {
    for (int kb = 0; kb < blocks; ++kb) {
        const bool ok = wait(tempty + 8 * d.i, d.ph ^ 1) && wait(full + 8 * r.i, r.ph);
        if (__any_sync(0xffffffffu, !ok))
            return false;
        tc_fence_after();
        const uint32_t a = base + r.i * ((RA + RW) * kBK), w = a + RA * kBK;
#pragma unroll
        for (int k = 0; k < kBK / 32; ++k)
            mma_f8_ss_if(tmem + d.i * BN, sdesc_sw128((A_IS_W ? w : a) + 32 * k, 16, 1024),
                         sdesc_sw128((A_IS_W ? a : w) + 32 * k, 16, 1024), idesc_e4m3(128, BN), k > 0, issue);
        mma_commit_if(empty + 8 * r.i, issue);
        mma_commit_if(tfull + 8 * d.i, issue);
        r.next();
        d.next();
    }
    return true;
}

// After the last MMA, or a failed wait: the MMAs in flight end before their
// memory is given back.  A barrier of its own, used once: an accumulator's may
// still be in the phase before the one that would be asked for, which a test of
// its parity takes for the phase's end.
__device__ __forceinline__ void drain_mma(uint32_t drain, uint32_t issue) {
    mma_commit_if(drain, issue);
    mbar_wait_bounded(drain, 0, kDefaultWaitLimit);
}

// 64 columns of one row from registers to out.
template <typename O>
__device__ __forceinline__ void store_row(const MatmulArgs &p, int64_t m, int64_t n0, const unsigned long long (&acc)[32],
                                          bool vec) {
    O *dst = reinterpret_cast<O *>(p.out) + m * p.out_stride + n0;
    constexpr int V = 16 / sizeof(O);
    if (vec && n0 + 64 <= p.N) {
#pragma unroll
        for (int i = 0; i < 64; i += V) {
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
        for (int i = 0; i < 32; ++i) {
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

constexpr int kWideN = 256, kWideStages = 4, kWideThreads = 640;
constexpr size_t kWideSmem = 1024 + (size_t)kWideStages * (128 + kWideN) * kBK;

// Four warpgroups take 64 columns each: a thread adds its row's finished block
// to 64 register sums while the tensor core works on the next one in the other
// half of TMEM.  Reading TMEM is latency that only other warps hide: two
// warpgroups of 128 columns took 146 us at 4096 x 12352 x 2048, four take 128.
// 4096 x 8192 x 16384: 500 us, 2190 TFLOP/s, in short runs, 600 us and 1830 TFLOP/s
// called back to back, at the power limit; what bounds it is this reading and
// adding, 32768 values for each 128 x 256 x 128 products.
template <typename O>
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tw, const MatmulArgs p,
                int tiles_m, int tiles_n, uint32_t *status) {
    constexpr int ST = kWideStages, BN = kWideN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * ST + 4 + 2 * kScaleSlots + 1];
    __shared__ float scales[kScaleSlots * 4 * 128];
    __shared__ uint32_t tmem_base, abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * ST, tfull = empty + 8 * ST, tempty = tfull + 16,
                   sfull = tempty + 16, sempty = sfull + 8 * kScaleSlots, drain = sempty + 8 * kScaleSlots;
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    const int KB = (int)((p.K + kBK - 1) / kBK);
    const Waiter wait{&abort_flag, status, p.wait_limit};
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 16);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(sfull + 8 * i, 2);
            mbar_init(sempty + 8 * i, 16);
        }
        mbar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (blockIdx.x == 0 && wait.limit >= kDefaultWaitLimit) // (see launch_matmul)
            status[0] = status[1] = 0;
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_base), 2 * BN);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    int tm, tn;
    if (warp < 4) {
        // 128 x 32 + 512 x 112 registers are what the block was launched with (640 x 96)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == 0 && lane == 0) {
            Ring<ST> r;
            int issued = 0;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                tile_of(t, tiles_m, tiles_n, tm, tn);
                ok = load_blocks<ST, 128, BN>(wait, r, issued, base, full, empty, &ta, &tw, tm * 128, tn * BN, 0, KB);
            }
            drain_loads(r, issued, full);
        } else if (warp == 1) {
            const uint32_t issue = elect_one();
            Ring<ST> r;
            Ring<2> d;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x)
                ok = issue_blocks<ST, 2, 128, BN, BN, false>(wait, r, d, base, full, empty, tfull, tempty, tmem, KB, issue);
            drain_mma(drain, issue);
        } else if (warp >= 2) {
            Ring<kScaleSlots> r;
            for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                tile_of(t, tiles_m, tiles_n, tm, tn);
                ok = load_scales<128>(wait, r, scales, sfull, sempty, p.a_scale, (int64_t)tm * 128, p.M, KB, nullptr, 0,
                                      KB, warp - 2, lane);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        const int wg = (warp - 4) >> 2, q = warp & 3; // TMEM lanes 32 q .. of this warp
        const bool vec = ((uintptr_t)p.out & 15) == 0 && (p.out_stride * sizeof(O)) % 16 == 0;
        Ring<2> d;
        Ring<kScaleSlots> r;
        for (int64_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            tile_of(t, tiles_m, tiles_n, tm, tn);
            const int64_t m = (int64_t)tm * 128 + 32 * q + lane, n0 = (int64_t)tn * BN + 64 * wg;
            // columns behind the end have zero operands; their scale is any valid one
            const float *sw = p.w_scale + (n0 < p.N ? n0 / 128 : 0) * KB;
            unsigned long long acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
                acc[i] = 0ull;
            float w = __ldg(sw);
            for (int kb = 0; kb < KB; ++kb) {
                if ((kb & 3) == 0) {
                    ok = wait(sfull + 8 * r.i, r.ph);
                    if (__any_sync(0xffffffffu, !ok)) {
                        ok = false;
                        break;
                    }
                }
                const float f = w * scales[(r.i * 4 + (kb & 3)) * 128 + 32 * q + lane];
                const unsigned long long sc = pack2(f, f);
                if (kb + 1 < KB)
                    w = __ldg(sw + kb + 1);
                if ((kb & 3) == 3 || kb + 1 == KB) {
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(sempty + 8 * r.i);
                    r.next();
                }
                ok = wait(tfull + 8 * d.i, d.ph);
                if (__any_sync(0xffffffffu, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = tmem + d.i * BN + 64 * wg + ((uint32_t)(32 * q) << 16);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[32];
                    tmem_ld32(at + 32 * c, v);
                    tmem_wait_ld();
                    if (c == 1) { // all of this half of TMEM is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(tempty + 8 * d.i);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        fma2(acc[16 * c + i], sc, pack2(v[2 * i], v[2 * i + 1]));
                }
                d.next();
            }
            if (ok && m < p.M)
                store_row<O>(p, m, n0, acc, vec);
        }
    }
    __syncwarp();
    __syncthreads();
    if (warp == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, 2 * BN);
    }
}

template <typename O> cudaError_t go_wide(const MatmulArgs &p, cudaStream_t s) {
    const int tiles_m = (int)((p.M + 127) / 128), tiles_n = (int)((p.N + kWideN - 1) / kWideN);
    CUtensorMap ta, tw;
    if (!encode_2d(&ta, p.a, p.K, p.M, p.K, kBK, 128, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !encode_2d(&tw, p.w, p.K, p.N, p.K, kBK, kWideN, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(wide_kernel<O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWideSmem);
    if (e != cudaSuccess)
        return e;
    const int64_t tiles = (int64_t)tiles_m * tiles_n;
    wide_kernel<O><<<(unsigned)(tiles < kSMs ? tiles : kSMs), kWideThreads, kWideSmem, s>>>(
        ta, tw, p, tiles_m, tiles_n, reinterpret_cast<uint32_t *>(p.ws));
    return cudaGetLastError();
}

// ------------------------------------------------------------------- thin

template <int BN> struct Thin {
    static constexpr int kStages = BN == 128 ? 6 : BN == 64 ? 8 : BN == 32 ? 9 : 11;
    static constexpr int kBuffers = BN == 16 ? 8 : 4;     // accumulators in TMEM
    static constexpr int kTmem = BN * kBuffers;
    static constexpr int kGroups = BN == 128 ? 2 : 1;     // warpgroups that add, each BN / kGroups columns
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr size_t kStageBytes = (size_t)kStages * (128 + BN) * kBK;
    static constexpr size_t kJoinBytes = 136 * (BN + 4) * 4; // ks join_rows(ks) <= 133 rows, 16 bytes apart in banks
    static constexpr size_t kSmem = 1024 + (kStageBytes > kJoinBytes ? kStageBytes : kJoinBytes);
};

// Rows of a tile that a block of the cluster adds up, at most.
__device__ __forceinline__ int join_rows(int ks) { return (128 + ks - 1) / ks; }

// One tile per cluster of ks blocks, which split its blocks of k and join their
// sums through shared memory, in the order of k.  A thread has one row of w
// and BN / kGroups rows of a.
template <int BN, typename O>
__global__ void __launch_bounds__(Thin<BN>::kThreads, 1)
    thin_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tw, const MatmulArgs p,
                int tiles_n, int ks, uint32_t *status) {
    using T = Thin<BN>;
    constexpr int ST = T::kStages, NB = T::kBuffers, COLS = BN / T::kGroups, LD = COLS < 32 ? COLS : 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[2 * ST + 2 * NB + 2 * kScaleSlots + 1];
    __shared__ __align__(16) float scales[kScaleSlots * 4 * BN];
    __shared__ uint32_t tmem_base, abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    float *join = reinterpret_cast<float *>(smem_raw + (base - smem_u32(smem_raw)));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * ST, tfull = empty + 8 * ST, tempty = tfull + 8 * NB,
                   sfull = tempty + 8 * NB, sempty = sfull + 8 * kScaleSlots, drain = sempty + 8 * kScaleSlots;
    const int KB = (int)((p.K + kBK - 1) / kBK);
    const int part = ks > 1 ? (int)cluster_rank() : 0;
    const int kb0 = KB * part / ks, kb1 = KB * (part + 1) / ks;
    const int tile = blockIdx.x / ks, tm = tile / tiles_n, tn = tile % tiles_n;
    const int64_t m0 = (int64_t)tm * BN, n0 = (int64_t)tn * 128;
    const Waiter wait{&abort_flag, status, p.wait_limit};
    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(tfull + 8 * i, 1);
            mbar_init(tempty + 8 * i, 4 * T::kGroups);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(sfull + 8 * i, 2);
            mbar_init(sempty + 8 * i, 4 * T::kGroups);
        }
        mbar_init(drain, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (blockIdx.x == 0 && wait.limit >= kDefaultWaitLimit) // (see launch_matmul)
            status[0] = status[1] = 0;
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_base), T::kTmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            Ring<ST> r;
            int issued = 0;
            load_blocks<ST, BN, 128>(wait, r, issued, base, full, empty, &ta, &tw, (int)m0, (int)n0, kb0, kb1);
            drain_loads(r, issued, full);
        }
    } else if (warp == 1) {
        const uint32_t issue = elect_one();
        Ring<ST> r;
        Ring<NB> d;
        issue_blocks<ST, NB, BN, 128, BN, true>(wait, r, d, base, full, empty, tfull, tempty, tmem, kb1 - kb0, issue);
        drain_mma(drain, issue);
    } else if (warp < 4) {
        Ring<kScaleSlots> r;
        load_scales<BN>(wait, r, scales, sfull, sempty, p.a_scale, m0, p.M, KB, p.w_scale + (int64_t)tn * KB, kb0, kb1,
                        warp - 2, lane);
    } else {
        const int wg = (warp - 4) >> 2, q = warp & 3;
        Ring<NB> d;
        Ring<kScaleSlots> r;
        unsigned long long acc[COLS / 2];
#pragma unroll
        for (int i = 0; i < COLS / 2; ++i)
            acc[i] = 0ull;
        for (int kb = kb0; kb < kb1; ++kb) {
            const int j = (kb - kb0) & 3;
            ok = (j != 0 || wait(sfull + 8 * r.i, r.ph)) && wait(tfull + 8 * d.i, d.ph);
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t at = tmem + d.i * BN + COLS * wg + ((uint32_t)(32 * q) << 16);
            const ulonglong2 *sc = reinterpret_cast<const ulonglong2 *>(scales + (r.i * 4 + j) * BN + COLS * wg);
#pragma unroll
            for (int c = 0; c < COLS; c += LD) {
                float v[LD];
                if constexpr (LD == 16)
                    tmem_ld16(at + c, v);
                else
                    tmem_ld32(at + c, v);
                tmem_wait_ld();
                if (c + LD == COLS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(tempty + 8 * d.i);
                }
#pragma unroll
                for (int i = 0; i < LD / 4; ++i) {
                    const ulonglong2 s2 = sc[c / 4 + i];
                    fma2(acc[c / 2 + 2 * i], s2.x, pack2(v[4 * i], v[4 * i + 1]));
                    fma2(acc[c / 2 + 2 * i + 1], s2.y, pack2(v[4 * i + 2], v[4 * i + 3]));
                }
            }
            d.next();
            if (j == 3 || kb + 1 == kb1) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(sempty + 8 * r.i);
                r.next();
            }
        }
        const int row = 32 * q + lane;
        if (ks == 1) {
            const int64_t n = n0 + row;
            if (ok && n < p.N) {
                O *dst = reinterpret_cast<O *>(p.out) + (m0 + COLS * wg) * p.out_stride + n;
#pragma unroll
                for (int i = 0; i < COLS / 2; ++i) {
                    const float2 f = unpack2(acc[i]);
                    if (m0 + COLS * wg + 2 * i < p.M)
                        dst[2 * i * p.out_stride] = from_f<O>(f.x);
                    if (m0 + COLS * wg + 2 * i + 1 < p.M)
                        dst[(2 * i + 1) * p.out_stride] = from_f<O>(f.y);
                }
            }
        } else {
            // each block of the cluster adds up its share of the rows: send it the sums, once the stages,
            // which hold them, are idle in all blocks
            __syncwarp();
            cluster_sync();
            const int to = row * ks / 128, r0 = (128 * to + ks - 1) / ks;
            const uint32_t dst = mapa(smem_u32(join), to) + 4u * ((part * join_rows(ks) + row - r0) * (BN + 4) + COLS * wg);
#pragma unroll
            for (int i = 0; i < COLS / 4; ++i)
                if (m0 + COLS * wg + 4 * i < p.M)
                    st_dsmem(dst + 16 * i, acc[2 * i], acc[2 * i + 1]);
        }
    }
    if (warp < 4 && ks > 1) {
        __syncwarp();
        cluster_sync();
    }
    __syncwarp();
    __syncthreads();
    if (ks > 1) {
        cluster_sync();
        const int quads = (int)((p.M - m0 < BN ? p.M - m0 : BN) + 3) / 4; // of rows of a that exist
        const int r0 = (128 * part + ks - 1) / ks, nr = (128 * (part + 1) + ks - 1) / ks - r0;
        for (int i = tid; i < quads * nr; i += T::kThreads) {
            const int c = i / nr * 4, r = i % nr;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < ks; ++k) {
                const float4 u = *reinterpret_cast<const float4 *>(join + (k * join_rows(ks) + r) * (BN + 4) + c);
                v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
            }
            const int64_t m = m0 + c, n = n0 + r0 + r;
            O *dst = reinterpret_cast<O *>(p.out) + m * p.out_stride + n;
            if (n < p.N) {
                dst[0] = from_f<O>(v.x);
                if (m + 1 < p.M)
                    dst[p.out_stride] = from_f<O>(v.y);
                if (m + 2 < p.M)
                    dst[2 * p.out_stride] = from_f<O>(v.z);
                if (m + 3 < p.M)
                    dst[3 * p.out_stride] = from_f<O>(v.w);
            }
        }
    }
    if (warp == 1) {
        tmem_relinquish();
        tmem_dealloc(tmem, T::kTmem);
    }
}

template <int BN, typename O> cudaLaunchConfig_t thin_config(unsigned blocks, int ks, cudaLaunchAttribute *at, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(Thin<BN>::kThreads);
    cfg.dynamicSmemBytes = Thin<BN>::kSmem;
    cfg.stream = s;
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = ks;
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of 1 .. 8 blocks that run at once, as the runtime counts them (the
// SMs of a cluster are of one GPC, so 148 SMs hold fewer clusters of 8 than
// 18).  Asked once per device; it decides a launch shape only.
struct Capacity {
    int clusters[9];
};
template <int BN, typename O> cudaError_t thin_capacity(const Capacity **cap) {
    static PerDevice<Capacity> known;
    int device = -1;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return e;
    return known.get(device, [](Capacity *c) {
        cudaError_t err = cudaFuncSetAttribute(thin_kernel<BN, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Thin<BN>::kSmem);
        for (int ks = 1; ks <= 8 && err == cudaSuccess; ++ks) {
            cudaLaunchAttribute at{};
            const cudaLaunchConfig_t cfg = thin_config<BN, O>(400 * ks, ks, &at, nullptr);
            err = cudaOccupancyMaxActiveClusters(&c->clusters[ks], thin_kernel<BN, O>, &cfg);
        }
        return err;
    }, cap);
}

// Blocks of a cluster for this many tiles and blocks of k: the most that still
// all run at once, with two blocks of k each at least.
template <int BN, typename O> cudaError_t thin_split(int64_t tiles, int KB, int *ks) {
    const Capacity *cap = nullptr;
    const cudaError_t e = thin_capacity<BN, O>(&cap);
    if (e != cudaSuccess)
        return e;
    *ks = 1;
    for (int k = 2; k <= 8 && 2 * k <= KB; ++k)
        if (tiles <= cap->clusters[k])
            *ks = k;
    return cudaSuccess;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int BN, typename O> cudaError_t go_thin(const MatmulArgs &p, cudaStream_t s) {
    using T = Thin<BN>;
    const int64_t tiles_n = ceil_div(p.N, 128), tiles = ceil_div(p.M, BN) * tiles_n;
    int ks;
    cudaError_t e = thin_split<BN, O>(tiles, (int)ceil_div(p.K, kBK), &ks);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(thin_kernel<BN, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)T::kSmem);
    if (e != cudaSuccess)
        return e;
    CUtensorMap ta, tw;
    if (!encode_2d(&ta, p.a, p.K, p.M, p.K, kBK, BN, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
        !encode_2d(&tw, p.w, p.K, p.N, p.K, kBK, 128, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_DATA_TYPE_UINT8))
        return cudaErrorInvalidValue;
    cudaLaunchAttribute at{};
    const cudaLaunchConfig_t cfg = thin_config<BN, O>((unsigned)(tiles * ks), ks, &at, s);
    return cudaLaunchKernelEx(&cfg, thin_kernel<BN, O>, ta, tw, p, (int)tiles_n, ks, reinterpret_cast<uint32_t *>(p.ws));
}

template <typename O> cudaError_t launch_t(const MatmulArgs &p, cudaStream_t s) {
    if (p.M <= 16)
        return go_thin<16, O>(p, s);
    if (p.M <= 32)
        return go_thin<32, O>(p, s);
    if (p.M <= 64)
        return go_thin<64, O>(p, s);
    // Both kernels take 0.5 to 0.6 us for a block of k, the wide one for twice
    // the columns; the one whose busiest SM has fewer blocks runs (the thin one
    // if equal: 14.0 us against 15.5 at 128 x 12352 x 2048).  At 512 x 8192
    // x 8192 that is the wide one (128 tiles in one round, 64 blocks; thin: 256
    // tiles in two rounds; 37 us against 66), at 301 x 1003 x 4112 the thin one (24 tiles in
    // 5 parts, 7 blocks, 12 us; wide: 12 tiles of 33 blocks).
    const int64_t KB = ceil_div(p.K, kBK), tm = ceil_div(p.M, 128), tt = tm * ceil_div(p.N, 128);
    int ks;
    const cudaError_t e = thin_split<128, O>(tt, (int)KB, &ks);
    if (e != cudaSuccess)
        return e;
    if (ceil_div(tm * ceil_div(p.N, kWideN), kSMs) * KB < ceil_div(tt * ks, kSMs) * ceil_div(KB, ks))
        return go_wide<O>(p, s);
    return go_thin<128, O>(p, s);
}

} // namespace

// The first word of the workspace is the kernels' status word.
size_t matmul_workspace_bytes(int64_t, int64_t, int64_t) { return kWorkspaceHeader; }

// The status words are cleared by the first block, which starts first: long
// before another one's wait of a second can run out.  An armed bound may run out
// before that, and its report would be lost: there they are cleared ahead.
cudaError_t launch_matmul(const MatmulArgs &p, cudaStream_t s) {
    if (p.wait_limit < kDefaultWaitLimit) {
        const cudaError_t e = cudaMemsetAsync(p.ws, 0, 2 * sizeof(uint32_t), s);
        if (e != cudaSuccess)
            return e;
    }
    return p.out_bf16 ? launch_t<__nv_bfloat16>(p, s) : launch_t<float>(p, s);
}

} // namespace gdn
