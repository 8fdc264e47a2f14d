// linear_tc.cu -- D = A B^T with the epilogue of mhc_linear on sm_100a tensor cores (bf16 operands,
// fp32 accumulation): the forward product and both products of its backward.
//
// Operands may have either index contiguous: TMA brings 64-wide boxes into 128-byte-swizzled shared
// memory and the MMA descriptors say whether a row of a box runs along K or along M / N, so
// dz W and dz^T x need no transposed copies.  Rows and columns past the operands read as zero.
//
// Two kernels:
//   * gemm_pair_kernel, for products with enough tiles to fill the device.  A cluster of two CTAs
//     forms 256 x BN tiles with cta_group::2 MMAs (M = 256): each CTA loads its 128 rows of A and
//     half of B's rows, so a byte of shared memory feeds twice the MMA work of a single CTA's tile.
//     Persistent: the accumulators are double buffered in TMEM, and the epilogue of one tile runs
//     under the MMAs of the next.  Warp roles (320 threads): 0 TMA, 1 MMA issue (first CTA of the
//     pair), 2-9 epilogue.
//   * gemm_split_kernel, for the others (single tokens, small or thin products).  The side with
//     contiguous output goes on the 128 MMA rows, so a few tokens are a narrow MMA N and a warp's
//     stores are contiguous.  A cluster of S CTAs shares a tile by splitting K; the partial tiles
//     meet in shared memory, where CTA r adds up its share of the columns in rank order: no
//     atomics, no workspace.  It is bound by streaming the larger operand from HBM.
//
// Every wait on an mbarrier is bounded in time; on expiry the kernel records the wait in a status
// word, lets its copies and MMAs in flight finish and returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "activation.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace mhc {

// Status of the bounded waits since the last read: 0 = fine, otherwise an OR of the codes of the
// waits that expired (mhc_device_status).
__device__ unsigned int g_linear_status;

namespace lintc {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int BK = 64;                  // K per stage: one 128-byte row
constexpr int ROW = 128;                // bytes
constexpr int BLK = 64 * ROW;           // a 64 x 64 box of an operand whose M / N index is contiguous
constexpr int THREADS = 320;
constexpr int EPI = 8;                  // epilogue warps: two per TMEM lane quarter
constexpr unsigned long long kWaitNs = 1000000000ull;    // 1 s per wait
constexpr unsigned long long kDrainNs = 2000000000ull;   // 2 s for the drains at exit
constexpr unsigned long long kLandNs = 2000000ull;       // after a failed wait: loads in flight land
constexpr uint32_t kSuspendNs = 20000;

enum : unsigned { E_STAGE = 1u, E_ACC = 2u, E_DRAIN = 4u };

// instruction descriptor, kind::f16: D fp32, A and B bf16
__host__ __device__ constexpr uint32_t idesc(int mm, int nn, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(nn >> 3) << 17) | ((uint32_t)(mm >> 4) << 24);
}

__device__ __forceinline__ bool mbar_try_sleep(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(kSuspendNs) : "memory");
    return ok != 0;
}

struct Waiter {
    volatile int* abort_flag;
    unsigned long long limit_ns;
    // true when the phase completed; false when the CTA is aborting or the wait expired
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, unsigned code,
                                               bool honour_abort = true) const {
        if (mbar_try_cluster(bar, parity)) return true;
        const uint64_t t0 = gtimer();
        while (true) {
            if (mbar_try_sleep(bar, parity)) return true;
            if (honour_abort && *abort_flag) return false;
            if (gtimer() - t0 > limit_ns) {
                atomicOr(&g_linear_status, code);
                *abort_flag = 1;
                return false;
            }
        }
    }
};

__device__ __forceinline__ void pause_ns(unsigned long long ns) {
    const uint64_t t0 = gtimer();
    while (gtimer() - t0 < ns) __nanosleep(1000);
}

// ---- CTA-pair forms
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id,
                                         uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate) : "memory");
}
// one arrival on the barrier at this offset in both CTAs, once the MMAs issued so far have completed
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"((uint16_t)3) : "memory");
}
// load into this CTA's shared memory, completing on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int c0,
                                              int c1) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// the descriptor of K16 step k of an operand's rows
template <bool MN>
__device__ __forceinline__ uint64_t step_desc(uint32_t base, int k) {
    return MN ? sw128_desc_mn(base + k * 2048, BLK, 1024) : sw128_desc(base + k * 32);
}

struct Maps {
    CUtensorMap a, b;
};

struct Epilogue {
    const float* bias;
    const bf16* residual;
    bf16* D;
    bf16* z;
    int act;
    int vec;                             // rows of D, z and residual are 16-byte aligned
};

// ------------------------------------------------------------------------- the pair kernel

template <int BN>
struct PairCfg {
    static constexpr int A_BYTES = 128 * ROW, B_BYTES = BN / 2 * ROW, STAGE = A_BYTES + B_BYTES;
    static constexpr int NS = 196608 / STAGE;                  // 6 stages at BN = 256, 8 at BN = 128
    static constexpr int OUT = EPI * 32 * ROW;                 // a 32 x 64 bf16 block per epilogue warp
    static constexpr int SMEM = NS * STAGE + OUT + 1024;       // + alignment slack
    static constexpr int TMEM_COLS = 512;                      // all of it, so both CTAs hold column 0
    static_assert(SMEM <= 232448 - 512, "shared memory");
    static_assert(2 * BN <= TMEM_COLS, "two accumulators");
};

// Tiles in an order that keeps the operands of those in flight in L2: bands of 8 tile rows, each
// walked column by column.
__device__ __forceinline__ void tile_at(int64_t i, int mt, int nt, int& m, int& n) {
    constexpr int BAND = 8;
    const int64_t per = (int64_t)BAND * nt;
    const int band = (int)(i / per);
    const int rows = mt - band * BAND < BAND ? mt - band * BAND : BAND;
    const int j = (int)(i - band * per);
    m = band * BAND + j % rows;
    n = j / rows;
}

template <int BN, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
gemm_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue ep, int64_t M, int64_t N, int ksteps, int mt,
                 int nt, unsigned long long wait_ns) {
    using C = PairCfg<BN>;
    constexpr int NS = C::NS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t bars[2 * NS + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    auto full = [&](int s) { return smem_u32(&bars[s]); };           // first CTA: both CTAs' loads landed
    auto empty = [&](int s) { return smem_u32(&bars[NS + s]); };     // the stage's MMAs are done
    auto accf = [&](int b) { return smem_u32(&bars[2 * NS + b]); };  // accumulator complete
    auto acce = [&](int b) { return smem_u32(&bars[2 * NS + 2 + b]); };   // first CTA: read by both CTAs
    const uint32_t drained = smem_u32(&bars[2 * NS + 4]);
    const Waiter wait{&abort_flag, wait_ns};
    const Waiter drain{&abort_flag, wait_ns > kDrainNs ? wait_ns : kDrainNs};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 2 * EPI);
        }
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    const int64_t tiles = (int64_t)mt * nt;
    const int64_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int64_t i = first; ok && i < tiles; i += stride) {
                int m, n;
                tile_at(i, mt, nt, m, n);
                const int m0 = m * 256 + (int)rank * 128, n0 = n * BN + (int)rank * (BN / 2);
                for (int ks = 0; ks < ksteps; ++ks, ++it) {
                    const int s = it % NS;
                    if (it >= NS && !(ok = wait(empty(s), (uint32_t)(it / NS - 1) & 1u, E_STAGE))) break;
                    if (rank == 0) mbar_arrive_tx(full(s), 2 * C::STAGE);
                    const uint32_t bar = mapa(full(s), 0);
                    const uint32_t a = smem_u32(sm + s * C::STAGE), b = a + C::A_BYTES;
                    if constexpr (A_MN) {
                        tma_load_pair(a, &maps.a, bar, m0, ks * BK);
                        tma_load_pair(a + BLK, &maps.a, bar, m0 + 64, ks * BK);
                    } else {
                        tma_load_pair(a, &maps.a, bar, ks * BK, m0);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int j = 0; j < BN / 128; ++j)
                            tma_load_pair(b + j * BLK, &maps.b, bar, n0 + 64 * j, ks * BK);
                    } else {
                        tma_load_pair(b, &maps.b, bar, ks * BK, n0);
                    }
                }
            }
            // the last stages' MMAs have signalled this CTA too before it may exit
            for (int j = it < NS ? 0 : it - NS; ok && j < it; ++j)
                ok = wait(empty(j % NS), (uint32_t)(j / NS) & 1u, E_STAGE);
            if (!ok) pause_ns(kLandNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t ID = idesc(256, BN, A_MN, B_MN);
            int it = 0, tc = 0;
            bool ok = true;
            for (int64_t i = first; ok && i < tiles; i += stride, ++tc) {
                const int buf = tc & 1;
                if (tc >= 2 && !(ok = wait(acce(buf), (uint32_t)((tc >> 1) - 1) & 1u, E_ACC))) break;
                tc_fence_after();
                for (int ks = 0; ks < ksteps; ++ks, ++it) {
                    const int s = it % NS;
                    if (!(ok = wait(full(s), (uint32_t)(it / NS) & 1u, E_STAGE))) break;
                    tc_fence_after();
                    const uint32_t a = smem_u32(sm + s * C::STAGE), b = a + C::A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_pair(tm + buf * BN, step_desc<A_MN>(a, k), step_desc<B_MN>(b, k), ID,
                                 (ks > 0 || k > 0) ? 1u : 0u);
                    mma_commit_pair(empty(s));
                }
                if (ok) mma_commit_pair(accf(buf));
            }
            if (!ok) {
                // every MMA issued so far: TMEM must be idle before it is freed
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             :: "r"(drained) : "memory");
                drain(drained, 0u, E_DRAIN, false);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, h = (warp - 2) >> 2;
        const uint32_t tq = tm + ((uint32_t)(32 * q) << 16);
        unsigned char* out = sm + NS * C::STAGE + (warp - 2) * 32 * ROW;
        const uint32_t acce_first[2] = {mapa(acce(0), 0), mapa(acce(1), 0)};
        int tc = 0;
        for (int64_t i = first; i < tiles; i += stride, ++tc) {
            const int buf = tc & 1;
            int m, n;
            tile_at(i, mt, nt, m, n);
            const int64_t r0 = (int64_t)m * 256 + rank * 128 + 32 * q;
            if (!__all_sync(0xffffffffu, wait(accf(buf), (uint32_t)(tc >> 1) & 1u, E_ACC))) break;
            tc_fence_after();
            for (int cc = 0; cc < BN / 2; cc += 64) {
                const int64_t c0 = (int64_t)n * BN + h * (BN / 2) + cc;
                float v[64];
                tmem_ld32(tq + buf * BN + h * (BN / 2) + cc, reinterpret_cast<float(&)[32]>(v[0]));
                tmem_ld32(tq + buf * BN + h * (BN / 2) + cc + 32, reinterpret_cast<float(&)[32]>(v[32]));
                if (c0 >= N || r0 >= M) continue;
                // this warp's 32 x 64 block between registers (a row per lane) and memory (128 bytes
                // of a row per eight lanes), through shared memory swizzled by 16-byte chunks
                auto lane_chunk = [&](int j) {
                    return reinterpret_cast<uint4*>(out + lane * ROW + ((j ^ (lane & 7)) << 4));
                };
                auto put = [&](bf16* dst) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) *lane_chunk(j) = Vec16<bf16>::pack(v + 8 * j);
                    __syncwarp();
                    if (ep.vec) {
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const int r = 4 * p + (lane >> 3), j = lane & 7;
                            if (r0 + r < M && c0 + 8 * j < N)
                                st_v4(dst + (r0 + r) * N + c0 + 8 * j,
                                      *reinterpret_cast<const uint4*>(out + r * ROW + ((j ^ (r & 7)) << 4)));
                        }
                    } else {
                        for (int r = 0; r < 32 && r0 + r < M; ++r)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int c = lane + 32 * u;
                                if (c0 + c < N)
                                    dst[(r0 + r) * N + c0 + c] = *reinterpret_cast<const bf16*>(
                                        out + r * ROW + (((c >> 3) ^ (r & 7)) << 4) + 2 * (c & 7));
                            }
                    }
                    __syncwarp();
                };
                if (ep.bias) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] += c0 + j < N ? __ldg(ep.bias + c0 + j) : 0.f;
                }
                if (ep.z) put(ep.z);
                with_act(ep.act, [&](auto kind) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) v[j] = act_value<kind(), true>(v[j]);
                });
                if (ep.residual) {
                    if (ep.vec) {
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            const int r = 4 * p + (lane >> 3), j = lane & 7;
                            if (r0 + r < M && c0 + 8 * j < N)
                                *reinterpret_cast<uint4*>(out + r * ROW + ((j ^ (r & 7)) << 4)) =
                                    ld_stream_v4(ep.residual + (r0 + r) * N + c0 + 8 * j);
                        }
                    } else {
                        for (int r = 0; r < 32 && r0 + r < M; ++r)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int c = lane + 32 * u;
                                if (c0 + c < N)
                                    *reinterpret_cast<bf16*>(out + r * ROW + (((c >> 3) ^ (r & 7)) << 4) +
                                                             2 * (c & 7)) = ep.residual[(r0 + r) * N + c0 + c];
                            }
                    }
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float f[8];
                        Vec16<bf16>::unpack(*lane_chunk(j), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[8 * j + e] += f[e];
                    }
                    __syncwarp();
                }
                put(ep.D);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(acce_first[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tm, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------- the split kernel

template <int BN>
struct SplitCfg {
    static constexpr int A_BYTES = 128 * ROW, B_BYTES = BN * ROW, STAGE = A_BYTES + B_BYTES;
    static constexpr int NS = 110592 / STAGE;                  // two CTAs per SM
    static constexpr int SMEM = NS * STAGE + 1024;
    static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
    static_assert(NS * STAGE >= BN * 128 * 4, "the partial tile fits the stages");
};

// D[c][r] = sum_k A(r, k) B(c, k), c < Nc, r < Mr, rows of Mr elements: A's side is the contiguous
// one.  bias belongs to r.
template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(THREADS, 2)
gemm_split_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue ep, int64_t Mr, int64_t Nc, int ksteps, int mt,
                  int S, unsigned long long wait_ns) {
    using C = SplitCfg<BN>;
    constexpr int NS = C::NS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t bars[2 * NS + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[NS + s]); };
    const uint32_t accf = smem_u32(&bars[2 * NS]), drained = smem_u32(&bars[2 * NS + 1]);
    const Waiter wait{&abort_flag, wait_ns};
    const Waiter drain{&abort_flag, wait_ns > kDrainNs ? wait_ns : kDrainNs};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / S;
    const int m0 = (tile % mt) * 128, n0 = (tile / mt) * BN;
    const int k_lo = (int)((int64_t)ksteps * rank / S), k_hi = (int)((int64_t)ksteps * (rank + 1) / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(accf, 1);
        mbar_init(drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    bool done = true;                    // the warp's wait completed

    if (warp == 0) {
        if (lane == 0) {
            bool ok = true;
            for (int ks = k_lo; ks < k_hi; ++ks) {
                const int it = ks - k_lo, s = it % NS;
                if (it >= NS && !(ok = wait(empty(s), (uint32_t)(it / NS - 1) & 1u, E_STAGE))) break;
                mbar_arrive_tx(full(s), C::STAGE);
                const uint32_t a = smem_u32(sm + s * C::STAGE), b = a + C::A_BYTES;
                if constexpr (A_MN) {
                    tma_load_2d(a, &maps.a, full(s), m0, ks * BK);
                    tma_load_2d(a + BLK, &maps.a, full(s), m0 + 64, ks * BK);
                } else {
                    tma_load_2d(a, &maps.a, full(s), ks * BK, m0);
                }
                if constexpr (B_MN) {
#pragma unroll
                    for (int j = 0; j < BN / 64; ++j) tma_load_2d(b + j * BLK, &maps.b, full(s), n0 + 64 * j, ks * BK);
                } else {
                    tma_load_2d(b, &maps.b, full(s), ks * BK, n0);
                }
            }
            if (!ok) pause_ns(kLandNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t ID = idesc(128, BN, A_MN, B_MN);
            bool ok = true;
            for (int ks = k_lo; ks < k_hi; ++ks) {
                const int it = ks - k_lo, s = it % NS;
                if (!(ok = wait(full(s), (uint32_t)(it / NS) & 1u, E_STAGE))) break;
                tc_fence_after();
                const uint32_t a = smem_u32(sm + s * C::STAGE), b = a + C::A_BYTES;
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                    mma_bf16(tm, step_desc<A_MN>(a, k), step_desc<B_MN>(b, k), ID, (it > 0 || k > 0) ? 1u : 0u);
                mma_commit(empty(s));
            }
            mma_commit(ok ? accf : drained);
            if (!ok) drain(drained, 0u, E_DRAIN, false);
        }
        __syncwarp();
    } else {
        done = __all_sync(0xffffffffu, wait(accf, 0u, E_ACC));
        tc_fence_after();
    }

    const int q = warp & 3, h = (warp - 2) >> 2;
    const int64_t r = (int64_t)m0 + 32 * q + lane;
    const uint32_t tq = tm + ((uint32_t)(32 * q) << 16);
    const float bias = warp >= 2 && ep.bias && r < Mr ? __ldg(ep.bias + r) : 0.f;
    // the outputs of columns c .. c + n - 1 (n <= 16) from their sums
    auto emit = [&](int c, int n, float (&v)[16]) {
        if (r >= Mr) return;
        if (ep.z) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < n && n0 + c + j < Nc) store_elem(ep.z + (n0 + (int64_t)c + j) * Mr + r, v[j] + bias);
        }
        with_act(ep.act, [&](auto kind) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (j < n && n0 + c + j < Nc) {
                    const int64_t at = (n0 + (int64_t)c + j) * Mr + r;
                    float o = act_value<kind(), true>(v[j] + bias);
                    if (ep.residual) o += to_f32(__ldg(ep.residual + at));
                    store_elem(ep.D + at, o);
                }
        });
    };
    constexpr int HALF = BN / 2, STEP = HALF < 16 ? HALF : 16;      // columns of a warp, and per TMEM load
    if (S == 1) {
        if (warp >= 2 && done) {
            for (int c = h * HALF; c < (h + 1) * HALF; c += STEP) {
                if (n0 + c >= Nc) break;
                float v[16];
                if constexpr (STEP == 16) {
                    tmem_ld16(tq + c, v);
                } else {
                    const uint4 lo = tmem_ld4(tq + c), hi = tmem_ld4(tq + c + 4);
                    v[0] = __uint_as_float(lo.x); v[1] = __uint_as_float(lo.y); v[2] = __uint_as_float(lo.z);
                    v[3] = __uint_as_float(lo.w); v[4] = __uint_as_float(hi.x); v[5] = __uint_as_float(hi.y);
                    v[6] = __uint_as_float(hi.z); v[7] = __uint_as_float(hi.w);
                }
                emit(c, STEP, v);
            }
        }
    } else {
        // the partial tile over the stages (their loads have been consumed), [column][128 rows]
        float* part = reinterpret_cast<float*>(sm);
        if (warp >= 2 && done) {
            for (int c = h * HALF; c < (h + 1) * HALF; c += STEP) {
                float v[16];
                if constexpr (STEP == 16) {
                    tmem_ld16(tq + c, v);
                } else {
                    const uint4 lo = tmem_ld4(tq + c), hi = tmem_ld4(tq + c + 4);
                    v[0] = __uint_as_float(lo.x); v[1] = __uint_as_float(lo.y); v[2] = __uint_as_float(lo.z);
                    v[3] = __uint_as_float(lo.w); v[4] = __uint_as_float(hi.x); v[5] = __uint_as_float(hi.y);
                    v[6] = __uint_as_float(hi.z); v[7] = __uint_as_float(hi.w);
                }
#pragma unroll
                for (int j = 0; j < STEP; ++j) part[(c + j) * 128 + 32 * q + lane] = v[j];
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (warp >= 2 && done) {
            // this CTA's BN / S columns, half of them per warp of a lane quarter
            const int per = BN / S / 2, c_lo = rank * 2 * per + h * per;
            for (int c = c_lo; c < c_lo + per; c += 16) {
                const int n = per < 16 ? per : 16;
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0.f;
                for (int p = 0; p < S; ++p) {
                    const uint32_t at = mapa(smem_u32(part + c * 128 + 32 * q + lane), (uint32_t)p);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (j < n) v[j] += ld_cluster_f32(at + j * 512);
                }
                emit(c, n, v);
            }
        }
        __syncwarp();
        cluster_sync_all();              // no CTA leaves while its partial tile is read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        cudaGetLastError();
    });
    return fn;
}

// An operand of `rows` rows (M or N side) and K: boxes of 64 along the contiguous index and
// `box_rows` rows (K contiguous) or 64 of K (rows contiguous).
bool make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t K, int64_t ld, bool mn, int box_rows) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(mn ? rows : K), (cuuint64_t)(mn ? K : rows)};
    const cuuint64_t str[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)(mn ? 64 : box_rows)};
    const cuuint32_t e1[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, str, box, e1,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<unsigned long long> g_wait_ns{kWaitNs};

template <typename K>
cudaError_t allow_smem(K kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

Epilogue epilogue_of(const GemmArgs& g) {
    Epilogue ep;
    ep.bias = g.bias;
    ep.residual = static_cast<const bf16*>(g.residual);
    ep.D = static_cast<bf16*>(g.D);
    ep.z = static_cast<bf16*>(g.z);
    ep.act = g.act;
    ep.vec = g.N % 8 == 0 && (uintptr_t)g.D % 16 == 0 && (uintptr_t)g.z % 16 == 0 && (uintptr_t)g.residual % 16 == 0;
    return ep;
}

template <int BN, bool A_MN, bool B_MN>
cudaError_t pair_launch(const GemmArgs& g, int sms) {
    using C = PairCfg<BN>;
    auto kern = gemm_pair_kernel<BN, A_MN, B_MN>;
    cudaError_t e = allow_smem(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    Maps maps;
    if (!make_map(&maps.a, g.A, g.M, g.K, g.lda, A_MN, 128) || !make_map(&maps.b, g.B, g.N, g.K, g.ldb, B_MN, BN / 2))
        return cudaErrorInvalidValue;
    const int mt = (int)((g.M + 255) / 256), nt = (int)((g.N + BN - 1) / BN);
    const int64_t tiles = (int64_t)mt * nt, pairs = sms / 2;
    const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
    kern<<<grid, THREADS, C::SMEM, g.stream>>>(maps, epilogue_of(g), g.M, g.N, (int)((g.K + BK - 1) / BK), mt, nt,
                                               g_wait_ns.load());
    return cudaGetLastError();
}

template <int BN>
cudaError_t pair_layout(const GemmArgs& g, int sms) {
    if (g.a_mn) return g.b_mn ? pair_launch<BN, true, true>(g, sms) : cudaErrorInvalidValue;
    return g.b_mn ? pair_launch<BN, false, true>(g, sms) : pair_launch<BN, false, false>(g, sms);
}

template <int BN, bool A_MN, bool B_MN>
cudaError_t split_launch(const GemmArgs& g, int S) {
    using C = SplitCfg<BN>;
    auto kern = gemm_split_kernel<BN, A_MN, B_MN>;
    cudaError_t e = allow_smem(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    Maps maps;                           // the product's B side on the MMA rows
    if (!make_map(&maps.a, g.B, g.N, g.K, g.ldb, A_MN, 128) || !make_map(&maps.b, g.A, g.M, g.K, g.lda, B_MN, BN))
        return cudaErrorInvalidValue;
    const int mt = (int)((g.N + 127) / 128);
    const int64_t tiles = (int64_t)mt * ((g.M + BN - 1) / BN);
    if (tiles * S > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * S));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = g.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, maps, epilogue_of(g), g.N, g.M, (int)((g.K + BK - 1) / BK), mt, S,
                              g_wait_ns.load());
}

template <int BN>
cudaError_t split_layout(const GemmArgs& g, int S) {
    if (g.a_mn) {
        if constexpr (BN >= 64) return g.b_mn ? split_launch<BN, true, true>(g, S) : cudaErrorInvalidValue;
        return cudaErrorInvalidValue;
    }
    return g.b_mn ? split_launch<BN, true, false>(g, S) : split_launch<BN, false, false>(g, S);
}

}  // namespace lintc

bool gemm_tc_ok(const GemmArgs& g) {
    const int64_t lim = ((int64_t)1 << 31) - 1024;
    return g.dt == BF16 && g.lda % 8 == 0 && g.ldb % 8 == 0 && (uintptr_t)g.A % 16 == 0 && (uintptr_t)g.B % 16 == 0 &&
           g.M < lim && g.N < lim && g.K < lim;
}

cudaError_t launch_gemm_tc(const GemmArgs& g) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const int64_t big = ((g.M + 255) / 256) * ((g.N + 255) / 256);
    if (2 * big >= di.sm_count) return lintc::pair_layout<256>(g, di.sm_count);
    // a narrow MMA N for few tokens; a product over tokens (rows contiguous) has boxes of 64
    const int bn = g.a_mn ? (g.M <= 64 ? 64 : 128) : g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
    const int64_t tiles = ((g.N + 127) / 128) * ((g.M + bn - 1) / bn), steps = (g.K + 63) / 64;
    int S = 1;
    while (S < 8 && tiles * S * 2 <= 2 * di.sm_count && steps >= S * 4) S *= 2;
    switch (bn) {
        case 16: return lintc::split_layout<16>(g, S);
        case 32: return lintc::split_layout<32>(g, S);
        case 64: return lintc::split_layout<64>(g, S);
        default: return lintc::split_layout<128>(g, S);
    }
}

cudaError_t linear_tc_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_linear_status, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    if (clear && *out) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_linear_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace mhc
