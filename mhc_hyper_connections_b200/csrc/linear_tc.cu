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
//     under the MMAs of the next.  The tiles of the last round, where they leave pairs idle, may be
//     shared by several pairs along K (Work); join_kernel adds their parts up (T = 700, 8192 -> 1100:
//     15 tiles in 4 parts each).  Warp roles: 0 TMA, 1 MMA issue (first CTA of the pair), 2-17 epilogue.
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

#include <algorithm>
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

constexpr int BK = 64;                  // K of a block: one 128-byte row
constexpr int ROW = 128;                // bytes
constexpr int BLK = 64 * ROW;           // a 64 x 64 box of an operand whose M / N index is contiguous
constexpr int EPI = 8;                  // epilogue warps of the split kernel: two per TMEM lane quarter
constexpr int THREADS = 32 * (2 + EPI);
// The pair kernels have four per lane quarter: an activation's chains of dependent operations need
// more warps than that to cover (T = 4096, 1024 -> 4096 with GELU, 8 warps: 56 us, 28 of them without it)
constexpr int PAIR_EPI = 16;
constexpr int CW = 32;                  // columns of outputs that a warp of theirs forms at a time
constexpr int PAIR_THREADS = 32 * (2 + PAIR_EPI);
// Clusters that a pair kernel's work is laid out for, one per two SMs of a 148-SM device.  The layout is
// part of the workspace's size, so it does not follow the device; a smaller one takes more rounds.
constexpr int PAIRS = 74;
constexpr unsigned long long kWaitNs = 1000000000ull;    // 1 s per wait
// more for a wait on a whole accumulator, per K block (0.3 us at most, measured): the sum over 2^31 tokens takes
// 1.4 s, in which every stage comes in time
constexpr unsigned long long kBlockNs = 4000ull;
constexpr unsigned long long kDrainNs = 2000000000ull;   // 2 s for the drains at exit
constexpr unsigned long long kLandNs = 2000000ull;       // after a failed wait: loads in flight land

enum : unsigned { E_STAGE = 1u, E_ACC = 2u, E_DRAIN = 4u };

// instruction descriptor, kind::f16: D fp32, A and B bf16
__host__ __device__ constexpr uint32_t idesc(int mm, int nn, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(nn >> 3) << 17) | ((uint32_t)(mm >> 4) << 24);
}

struct Waiter {
    volatile int* abort_flag;
    unsigned long long limit_ns;
    __device__ __forceinline__ Waiter over(int blocks) const { return Waiter{abort_flag, limit_ns + blocks * kBlockNs}; }
    // true when the phase completed; false when the CTA is aborting or the wait expired
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, unsigned code,
                                               bool honour_abort = true) const {
        // the timer is read only after tries that no healthy wait needs: reading it costs more than
        // a pipeline step
        for (int i = 0; i < 256; ++i) {
            if (mbar_try(bar, parity)) return true;
            if (honour_abort && *abort_flag) return false;
        }
        const uint64_t t0 = gtimer();
        while (true) {
            if (mbar_try(bar, parity)) return true;
            if (honour_abort && *abort_flag) return false;
            if (gtimer() - t0 > limit_ns) {
                atomicOr(&g_linear_status, code);
                *abort_flag = 1;
                return false;
            }
        }
    }
    // the whole warp's answer, with every lane past the wait
    __device__ __forceinline__ bool warp(uint32_t bar, uint32_t parity, unsigned code, bool honour_abort = true) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity, code, honour_abort));
    }
};

// Position in a ring of NS stages: the slot, and the parity of the slot's current round.  Waiting
// for the opposite parity is waiting for the previous round, which before the first one is over.
template <int NS>
struct Ring {
    int s = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++s == NS) {
            s = 0;
            parity ^= 1u;
        }
    }
};

// One lane of a converged warp.  The issue loops below are walked by whole warps and only the
// instructions that start asynchronous work sit under this predicate: the compiler then keeps
// descriptors and addresses in uniform registers.  Walked by one lane alone, a K step of the MMA
// loop took 620 cycles to issue, more than its MMAs take to run.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

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
__device__ __forceinline__ void tma_load_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int c0,
                                                 int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The descriptor of an operand's rows in stage 0, and the descriptor units (16 bytes) from one K16
// step to the next: 32 bytes along a row, or 16 rows of a box whose rows run along M / N.
template <bool MN>
__device__ __forceinline__ uint64_t base_desc(uint32_t base) {
    return MN ? sw128_desc_mn(base, BLK, 1024) : sw128_desc(base);
}
template <bool MN> constexpr uint32_t K16 = MN ? 2048 / 16 : 32 / 16;

// 32 lanes x 8 consecutive 32-bit columns, waiting for the load
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&f)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr) : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 :: "l"(map), "r"(c0), "r"(c1), "r"(src) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// operands, the outputs D and z of a pair kernel (where their rows are 16-byte aligned), and the parts of
// its shared tiles
struct Maps {
    CUtensorMap a, b, d, z, p;
};

// The wait limit, and the failure-path test hook: stages after which a CTA stops loading (< 0: never)
struct Limits {
    unsigned long long wait_ns;
    int stop;
};

template <typename T>
struct Epilogue {
    const float* bias;
    const T* residual;
    T* D;
    T* z;
    int act;
    int vec;                             // rows of D, z and residual are 16-byte aligned
};

// A warp's 32 rows x `cols` columns of the residual on their way to L2, while their tile is formed (a row
// per lane; T = 4096, 1024 -> 4096 with a residual from HBM: see finish_block's loads)
template <typename T>
__device__ __forceinline__ void prefetch_residual(const Epilogue<T>& ep, int64_t r0, int64_t c0, int cols, int64_t M,
                                                  int64_t N, int lane) {
    if (!ep.residual || r0 + lane >= M) return;
    for (int c = 0; c < cols && c0 + c < N; c += CW)
        asm volatile("prefetch.global.L2 [%0];" :: "l"(ep.residual + (r0 + lane) * N + c0 + c));
}

// The outputs of a warp's 32 rows x CW columns at (r0, c0) from their sums, a row per lane:
// v = act(v + bias) + residual, and z.  Between registers and memory the block goes through the warp's
// shared memory, swizzled by 16-byte chunks as TMA stores of 64- and 128-byte rows expect them: written
// by the lanes instead, dW of T = 64, 4096 -> 16384 (134 MB out) took 50 us, 21 of them in the stores.
// lane 0 has the stores in flight; whoever ends the kernel waits for them.
template <typename T>
__device__ __forceinline__ void finish_block(const Epilogue<T>& ep, const Maps& maps, float (&v)[CW],
                                             unsigned char* out, int64_t r0, int64_t c0, int64_t M, int64_t N,
                                             int lane) {
    constexpr int VEC = Vec16<T>::VEC, CPR = CW / VEC;          // 16-byte chunks per row: 4 or 8
    auto at = [&](int r, int j) { return out + (r * CPR + (j ^ (CPR == 8 ? r & 7 : (r >> 1) & 3))) * 16; };
    // vector loads: lane's chunk lane % CPR of rows lane / CPR + (32 / CPR) p, p < CPR
    constexpr int STEP = 32 / CPR;
    const int lr = lane / CPR, lc = lane % CPR;
    const int64_t mine = (r0 + lr) * N + c0 + VEC * lc;
    const int rows = c0 + VEC * lc < N ? (M - r0 < 32 ? (int)(M - r0) : 32) - lr : 0;
    auto free_block = [&] {              // the last store has read it
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
    };
    auto put = [&](T* dst, const CUtensorMap& map) {
#pragma unroll
        for (int j = 0; j < CPR; ++j) *reinterpret_cast<uint4*>(at(lane, j)) = Vec16<T>::pack(v + VEC * j);
        if (ep.vec) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tma_store_2d(&map, smem_u32(out), (int)c0, (int)r0);
            return;
        }
        __syncwarp();
#pragma unroll 2
        for (int r = 0; r < 32 && r0 + r < M; ++r)
            if (c0 + lane < N)
                dst[(r0 + r) * N + c0 + lane] = reinterpret_cast<const T*>(at(r, lane / VEC))[lane % VEC];
        __syncwarp();
    };
    if (ep.bias) {
        if (c0 + CW <= N && (uintptr_t)ep.bias % 16 == 0) {
#pragma unroll
            for (int j = 0; j < CW; j += 4) {
                const float4 b = __ldg(reinterpret_cast<const float4*>(ep.bias + c0 + j));
                v[j] += b.x; v[j + 1] += b.y; v[j + 2] += b.z; v[j + 3] += b.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < CW; ++j) v[j] += c0 + j < N ? __ldg(ep.bias + c0 + j) : 0.f;
        }
    }
    free_block();
    if (ep.z) put(ep.z, maps.z);
    if (ep.residual) {
        if (ep.z) free_block();
        if (ep.vec) {
#pragma unroll
            for (int p = 0; p < CPR; ++p)
                if (STEP * p < rows)
                    *reinterpret_cast<uint4*>(at(STEP * p + lr, lc)) = ld_stream_v4(ep.residual + mine + p * STEP * N);
        } else {
#pragma unroll 2
            for (int r = 0; r < 32 && r0 + r < M; ++r)
                if (c0 + lane < N)
                    reinterpret_cast<T*>(at(r, lane / VEC))[lane % VEC] = ep.residual[(r0 + r) * N + c0 + lane];
        }
        __syncwarp();
    }
    with_act(ep.act, [&](auto kind) {
#pragma unroll
        for (int j = 0; j < CW; ++j) v[j] = act_value<kind(), sizeof(T) == 2>(v[j]);
    });
    if (ep.residual) {
#pragma unroll
        for (int j = 0; j < CPR; ++j) {
            float f[VEC];
            Vec16<T>::unpack(*reinterpret_cast<uint4*>(at(lane, j)), f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[VEC * j + e] += f[e];
        }
    }
    if (ep.z && !ep.residual) free_block();
    put(ep.D, maps.d);                   // a lane overwrites its own row of the residual
}

// A warp's 32 rows x CW columns of a shared tile's part, as they are, in two halves of 64-byte rows
__device__ __forceinline__ void store_part(const CUtensorMap& map, const float (&v)[CW], unsigned char* out, int c0,
                                           int64_t r0, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<float4*>(out + (lane * 4 + (j ^ ((lane >> 1) & 3))) * 16) =
                make_float4(v[16 * h + 4 * j], v[16 * h + 4 * j + 1], v[16 * h + 4 * j + 2], v[16 * h + 4 * j + 3]);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tma_store_2d(&map, smem_u32(out), c0 + 16 * h, (int)r0);
    }
}

// ------------------------------------------------------------------------- the pair kernel

template <int BN>
struct PairCfg {
    static constexpr int A_BYTES = 128 * ROW, B_BYTES = BN / 2 * ROW, BLOCK = A_BYTES + B_BYTES;
    // Blocks per stage: a stage's waits and commits take about as long to issue as 8 MMAs of N = 128
    // (T = 256, 16384 -> 4096 at BN = 128: 67 us with one block per stage, 54 with two); at N = 256 the
    // MMAs of one block cover them, and finer stages are refilled sooner (79 us with one, 83 with two)
    static constexpr int KS = BN == 256 ? 1 : 2;
    static constexpr int STAGE = KS * BLOCK;
    static constexpr int NS = 196608 / STAGE;                  // 6 stages at BN = 256, 4 at BN = 128
    static constexpr int OUT = PAIR_EPI * 32 * CW * 2;         // a block of outputs per epilogue warp
    static constexpr int SMEM = NS * STAGE + OUT + 1024;       // + alignment slack
    static constexpr int TMEM_COLS = 512;                      // all of it, so both CTAs hold column 0
    static_assert(SMEM <= 232448 - 512, "shared memory");
    static_assert(2 * BN <= TMEM_COLS, "two accumulators");
    static_assert(BN / 4 % CW == 0, "whole blocks per epilogue warp");
};

// What the pairs of a launch do, in this order: tiles 0 .. full - 1 whole, and the others in S parts each
// along K, which are left in blocks of 256 x BN floats.
struct Work {
    int mt, nt, kblocks, S;
    int64_t full, items;
};

struct Item {
    int m, n, k0, k1;
    int64_t block;                       // of a part, or -1
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

__device__ __forceinline__ Item item_at(int64_t i, const Work& w) {
    Item it;
    it.k0 = 0;
    it.k1 = w.kblocks;
    it.block = -1;
    if (i >= w.full) {
        it.block = i - w.full;
        const int part = (int)(it.block % w.S);
        i = w.full + it.block / w.S;
        it.k0 = (int)((int64_t)w.kblocks * part / w.S);
        it.k1 = (int)((int64_t)w.kblocks * (part + 1) / w.S);
    }
    tile_at(i, w.mt, w.nt, it.m, it.n);
    return it;
}

// The outputs of the shared tiles from their parts, added in order: four columns of a row per thread.  The
// parts were written moments before and come from L2.
template <typename T, int BN>
__global__ void __launch_bounds__(256)
join_kernel(const float* __restrict__ part, const __grid_constant__ Epilogue<T> ep, int64_t M, int64_t N, Work w) {
    constexpr int ROWS = 256 / (BN / 4);
    pdl_launch_next();
    pdl_wait();
    const int r = blockIdx.x * ROWS + threadIdx.x / (BN / 4), c = threadIdx.x % (BN / 4) * 4;
    int m, n;
    tile_at(w.full + blockIdx.y, w.mt, w.nt, m, n);
    const int64_t row = (int64_t)m * 256 + r, col = (int64_t)n * BN + c;
    if (row >= M || col >= N) return;
    const float* p = part + ((int64_t)blockIdx.y * w.S * 256 + r) * BN + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = 0; k < w.S; ++k) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(p + (int64_t)k * 256 * BN));
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    }
    const int64_t at = row * N + col;
    const int left = N - col < 4 ? (int)(N - col) : 4;
    float res[4] = {0.f, 0.f, 0.f, 0.f};
    auto put = [&](T* dst) {
        if (ep.vec) {                    // N is a multiple of four
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint2*>(dst + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            else
                *reinterpret_cast<float4*>(dst + at) = make_float4(v[0], v[1], v[2], v[3]);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) store_elem(dst + at + e, v[e]);
    };
    if (ep.residual) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) res[e] = to_f32(__ldg(ep.residual + at + e));
    }
    if (ep.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < left) v[e] += __ldg(ep.bias + col + e);
    }
    if (ep.z) put(ep.z);
    with_act(ep.act, [&](auto kind) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = act_value<kind(), sizeof(T) == 2>(v[e]);
    });
    if (ep.residual) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += res[e];
    }
    put(ep.D);
}

template <int BN, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
gemm_pair_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue<bf16> ep, int64_t M, int64_t N,
                 const __grid_constant__ Work work, Limits lim) {
    using C = PairCfg<BN>;
    constexpr int NS = C::NS, KS = C::KS;
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
    const Waiter wait{&abort_flag, lim.wait_ns};
    const Waiter drain{&abort_flag, lim.wait_ns > kDrainNs ? lim.wait_ns : kDrainNs};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), base = smem_u32(sm);

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 2 * PAIR_EPI);
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
    // The next kernel may set itself up from here on, not before: a CTA of it that took this one's
    // TMEM would wait for this kernel's end.  What the previous one wrote is there after the wait.
    pdl_launch_next();
    pdl_wait();
    const uint32_t tm = tmem_slot;
    const int64_t items = work.items;
    const int64_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;

    if (warp == 0) {
        Ring<NS> ring;
        bool ok = true;
        int left = lim.stop;
        for (int64_t i = first; ok && left != 0 && i < items; i += stride) {
            const Item it = item_at(i, work);
            const int m0 = it.m * 256 + (int)rank * 128, n0 = it.n * BN + (int)rank * (BN / 2);
            for (int kb = it.k0; kb < it.k1 && left != 0; kb += KS, ring.next(), --left) {
                const int s = ring.s;
                if (!(ok = wait.warp(empty(s), ring.parity ^ 1u, E_STAGE))) break;
                if (elect_one()) {
                    const int nb = it.k1 - kb < KS ? it.k1 - kb : KS;
                    if (rank == 0) mbar_arrive_tx(full(s), 2 * C::BLOCK * nb);
                    const uint32_t bar = mapa(full(s), 0);
#pragma unroll
                    for (int u = 0; u < KS; ++u) {
                        if (u >= nb) break;
                        const uint32_t a = base + s * C::STAGE + u * C::BLOCK, b = a + C::A_BYTES;
                        const int k = (kb + u) * BK;
                        if constexpr (A_MN) {
                            tma_load_pair(a, &maps.a, bar, m0, k);
                            tma_load_pair(a + BLK, &maps.a, bar, m0 + 64, k);
                        } else {
                            tma_load_pair(a, &maps.a, bar, k, m0);
                        }
                        if constexpr (B_MN) {
#pragma unroll
                            for (int j = 0; j < BN / 128; ++j) tma_load_pair(b + j * BLK, &maps.b, bar, n0 + 64 * j, k);
                        } else {
                            tma_load_pair(b, &maps.b, bar, k, n0);
                        }
                    }
                }
                __syncwarp();
            }
        }
        // the last stages' MMAs have signalled this CTA too before it may exit (a stage never used
        // counts as free)
        for (int j = 0; ok && j < NS; ++j, ring.next()) ok = wait.warp(empty(ring.s), ring.parity ^ 1u, E_STAGE);
        if (!ok) pause_ns(kLandNs);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t ID = idesc(256, BN, A_MN, B_MN);
            const uint64_t da0 = base_desc<A_MN>(base), db0 = base_desc<B_MN>(base + C::A_BYTES);
            Ring<NS> ring;
            int tc = 0;
            bool ok = true;
            for (int64_t i = first; ok && i < items; i += stride, ++tc) {
                const Item it = item_at(i, work);
                const int buf = tc & 1;
                if (!(ok = wait.warp(acce(buf), ((uint32_t)(tc >> 1) & 1u) ^ 1u, E_ACC))) break;
                tc_fence_after();
                for (int kb = it.k0; kb < it.k1; kb += KS, ring.next()) {
                    const int s = ring.s;
                    if (!(ok = wait.warp(full(s), ring.parity, E_STAGE))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int u = 0; u < KS; ++u) {
                            if (kb + u >= it.k1) break;
                            const uint32_t off = (uint32_t)(s * (C::STAGE >> 4) + u * (C::BLOCK >> 4));
#pragma unroll
                            for (int k = 0; k < BK / 16; ++k)
                                mma_pair(tm + buf * BN, da0 + off + k * K16<A_MN>, db0 + off + k * K16<B_MN>, ID,
                                         (kb > it.k0 || u > 0 || k > 0) ? 1u : 0u);
                        }
                        mma_commit_pair(empty(s));
                        if (kb + KS >= it.k1) mma_commit_pair(accf(buf));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                // every MMA issued so far: TMEM must be idle before it is freed
                if (elect_one())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                                 :: "r"(drained) : "memory");
                drain.warp(drained, 0u, E_DRAIN, false);
            }
        }
        __syncwarp();
    } else {
        // a warp has BN / 4 columns of its lane quarter
        const int q = warp & 3, h = (warp - 2) >> 2;
        const uint32_t tq = tm + ((uint32_t)(32 * q) << 16) + h * (BN / 4);
        unsigned char* out = sm + NS * C::STAGE + (warp - 2) * 32 * CW * 2;
        const uint32_t acce_first[2] = {mapa(acce(0), 0), mapa(acce(1), 0)};
        int tc = 0;
        for (int64_t i = first; i < items; i += stride, ++tc) {
            const int buf = tc & 1;
            const Item it = item_at(i, work);
            const int64_t r0 = (int64_t)it.m * 256 + rank * 128 + 32 * q, c0 = (int64_t)it.n * BN + h * (BN / 4);
            if (it.block < 0) prefetch_residual(ep, r0, c0, BN / 4, M, N, lane);
            if (!wait.over(it.k1 - it.k0).warp(accf(buf), (uint32_t)(tc >> 1) & 1u, E_ACC)) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < BN / 4; c += CW) {
                if (c0 + c >= N || r0 >= M) continue;
                float v[CW];
                tmem_ld32(tq + buf * BN + c, v);
                if (it.block < 0)
                    finish_block<bf16>(ep, maps, v, out, r0, c0 + c, M, N, lane);
                else
                    store_part(maps.p, v, out, h * (BN / 4) + c, it.block * 256 + rank * 128 + 32 * q, lane);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_cluster(buf ? acce_first[1] : acce_first[0]);
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tm, C::TMEM_COLS);
    }
}

// ------------------------------------------------------------------------- fp32 operands
//
// An fp32 value is the sum of three bf16 ones, h + m + l, 8 significant bits each.  Of the nine products
// of two such sums the six above 2^-24 of the whole are formed; the products of a chunk of K add up in
// TMEM, the chunks in registers.  The tensor core's additions drop the bits below its accumulator
// instead of rounding, an error of one sign that grows with the number of additions.  So a chunk is
// short (CHUNK blocks of 64), and the five small products have an accumulator of their own, where the
// dropped bits are 2^-8 of those of h h (one accumulator for all six: a relative error of 1.5e-6 at
// any K; see linear.cu for when this kernel runs).
//
// The parts are those of the values times 2^16 (SplitJob), so the sums are 2^32 times what they stand for.
// One of 2^126 or more (2^94, 2e28, of the product's) has overflowed on the way or may have: it sets *over,
// and the CUDA-core kernel behind this one forms the product.

struct F32Cfg {
    static constexpr int BN = 128;
    static constexpr int A_PLANE = 128 * ROW, B_PLANE = BN / 2 * ROW;      // one of the three parts
    static constexpr int STAGE = 3 * (A_PLANE + B_PLANE);                  // 64 of K
    static constexpr int NS = 2;
    static constexpr int OUT = PAIR_EPI * 32 * CW * 4;
    static constexpr int SMEM = NS * STAGE + OUT + 1024;
    static constexpr int TMEM_COLS = 512;
    static constexpr int CHUNK = 4;
    static constexpr float UNSCALE = 0x1p-32f, OVER = 0x1p126f;
    static_assert(SMEM <= 232448 - 512, "shared memory");
    static_assert(BN == 4 * CW, "a block per epilogue warp");
};

// The maps cover the planes as a third dimension and bring the three parts of a box together: rows
// along K as [part][row], others as [64 rows][part][64 of K].
template <bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PAIR_THREADS, 1)
gemm_f32_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue<float> ep, int64_t M, int64_t N,
                const __grid_constant__ Work work, Limits lim, int* __restrict__ over) {
    using C = F32Cfg;
    constexpr int NS = C::NS, BN = C::BN;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t bars[2 * NS + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[NS + s]); };
    auto accf = [&](int b) { return smem_u32(&bars[2 * NS + b]); };
    auto acce = [&](int b) { return smem_u32(&bars[2 * NS + 2 + b]); };
    const uint32_t drained = smem_u32(&bars[2 * NS + 4]);
    const Waiter wait{&abort_flag, lim.wait_ns};
    const Waiter drain{&abort_flag, lim.wait_ns > kDrainNs ? lim.wait_ns : kDrainNs};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), base = smem_u32(sm);

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf(b), 1);
            mbar_init(acce(b), 2 * PAIR_EPI);
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
    pdl_launch_next();                   // as in the pair kernel
    pdl_wait();
    const uint32_t tm = tmem_slot;
    const int64_t items = work.items;
    const int64_t first = blockIdx.x >> 1, stride = gridDim.x >> 1;

    if (warp == 0) {
        Ring<NS> ring;
        bool ok = true;
        int left = lim.stop;
        for (int64_t i = first; ok && left != 0 && i < items; i += stride) {
            const Item it = item_at(i, work);
            const int m0 = it.m * 256 + (int)rank * 128, n0 = it.n * BN + (int)rank * (BN / 2);
            for (int kb = it.k0; kb < it.k1 && left != 0; ++kb, ring.next(), --left) {
                const int s = ring.s;
                if (!(ok = wait.warp(empty(s), ring.parity ^ 1u, E_STAGE))) break;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_tx(full(s), 2 * C::STAGE);
                    const uint32_t bar = mapa(full(s), 0);
                    const uint32_t a = base + s * C::STAGE, b = a + 3 * C::A_PLANE;
                    const int k = kb * BK;
                    if constexpr (A_MN) {
                        tma_load_pair_3d(a, &maps.a, bar, m0, k, 0);
                        tma_load_pair_3d(a + 3 * BLK, &maps.a, bar, m0 + 64, k, 0);
                    } else {
                        tma_load_pair_3d(a, &maps.a, bar, k, m0, 0);
                    }
                    if constexpr (B_MN) {
                        tma_load_pair_3d(b, &maps.b, bar, n0, k, 0);
                    } else {
                        tma_load_pair_3d(b, &maps.b, bar, k, n0, 0);
                    }
                }
                __syncwarp();
            }
        }
        for (int j = 0; ok && j < NS; ++j, ring.next()) ok = wait.warp(empty(ring.s), ring.parity ^ 1u, E_STAGE);
        if (!ok) pause_ns(kLandNs);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t ID = idesc(256, BN, A_MN, B_MN);
            // parts of A and B in each product, smallest products first
            constexpr int PA[6] = {2, 0, 1, 1, 0, 0}, PB[6] = {0, 2, 1, 0, 1, 0};
            constexpr uint32_t AP = (A_MN ? BLK : C::A_PLANE) >> 4, BP = (B_MN ? BLK : C::B_PLANE) >> 4;
            const uint64_t da0 = A_MN ? sw128_desc_mn(base, 3 * BLK, 1024) : sw128_desc(base);
            const uint64_t db0 = base_desc<B_MN>(base + 3 * C::A_PLANE);
            Ring<NS> ring;
            int tc = 0;
            bool ok = true;
            for (int64_t i = first; ok && i < items; i += stride) {
                const Item it = item_at(i, work);
                for (int kb = it.k0; ok && kb < it.k1; ++tc) {
                    const int buf = tc & 1;
                    if (!(ok = wait.warp(acce(buf), ((uint32_t)(tc >> 1) & 1u) ^ 1u, E_ACC))) break;
                    tc_fence_after();
                    const int end = kb + C::CHUNK < it.k1 ? kb + C::CHUNK : it.k1;
                    for (bool fresh = true; kb < end; ++kb, fresh = false, ring.next()) {
                        const int s = ring.s;
                        if (!(ok = wait.warp(full(s), ring.parity, E_STAGE))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t off = (uint32_t)(s * (C::STAGE >> 4));
#pragma unroll
                            for (int p = 0; p < 6; ++p)
#pragma unroll
                                for (int k = 0; k < BK / 16; ++k)
                                    mma_pair(tm + buf * 2 * BN + (p < 5 ? BN : 0), da0 + off + PA[p] * AP + k * K16<A_MN>,
                                             db0 + off + PB[p] * BP + k * K16<B_MN>, ID,
                                             (!fresh || (p > 0 && p < 5) || k > 0) ? 1u : 0u);
                            mma_commit_pair(empty(s));
                            if (kb == end - 1) mma_commit_pair(accf(buf));
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok) {
                if (elect_one())
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                                 :: "r"(drained) : "memory");
                drain.warp(drained, 0u, E_DRAIN, false);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, h = (warp - 2) >> 2;
        const uint32_t tq = tm + ((uint32_t)(32 * q) << 16) + h * CW;
        unsigned char* out = sm + NS * C::STAGE + (warp - 2) * 32 * CW * 4;
        const uint32_t acce_first[2] = {mapa(acce(0), 0), mapa(acce(1), 0)};
        int tc = 0;
        bool ok = true;
        for (int64_t i = first; ok && i < items; i += stride) {
            const Item it = item_at(i, work);
            const int64_t r0 = (int64_t)it.m * 256 + rank * 128 + 32 * q, c0 = (int64_t)it.n * BN + h * CW;
            if (it.block < 0) prefetch_residual(ep, r0, c0, CW, M, N, lane);
            float sum[CW] = {};
            for (int kb = it.k0; kb < it.k1; kb += C::CHUNK, ++tc) {
                const int buf = tc & 1;
                if (!(ok = wait.warp(accf(buf), (uint32_t)(tc >> 1) & 1u, E_ACC))) break;
                tc_fence_after();
                float v[CW], w[CW];
                tmem_ld32(tq + buf * 2 * BN, v);
                tmem_ld32(tq + buf * 2 * BN + BN, w);
#pragma unroll
                for (int j = 0; j < CW; ++j) sum[j] += v[j] + w[j];
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(buf ? acce_first[1] : acce_first[0]);
            }
            if (!ok) break;
            if (c0 >= N || r0 >= M) continue;
            bool large = false;
#pragma unroll
            for (int j = 0; j < CW; ++j) {
                large |= !(fabsf(sum[j]) < C::OVER);
                sum[j] *= C::UNSCALE;
            }
            if (large) *over = 1;
            if (it.block < 0)
                finish_block<float>(ep, maps, sum, out, r0, c0, M, N, lane);
            else
                store_part(maps.p, sum, out, h * CW, it.block * 256 + rank * 128 + 32 * q, lane);
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
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
    static constexpr int A_BYTES = 128 * ROW, B_BYTES = BN * ROW, BLOCK = A_BYTES + B_BYTES;
    // two CTAs per SM up to BN = 64, one above; two blocks per stage where three such stages fit
    static constexpr int PER_SM = BN > 64 ? 1 : 2;
    static constexpr int ROOM = 221184 / PER_SM;
    static constexpr int KS = 6 * BLOCK <= ROOM ? 2 : 1;
    static constexpr int STAGE = KS * BLOCK;
    static constexpr int NS = ROOM / STAGE;
    static constexpr int SMEM = NS * STAGE + 1024;
    static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
    static_assert(NS * STAGE >= BN * 128 * 4, "the partial tile fits the stages");
};

// D[c][r] = sum_k A(r, k) B(c, k), c < Nc, r < Mr, rows of Mr elements: A's side is the contiguous
// one.  bias belongs to r.
template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(THREADS, SplitCfg<BN>::PER_SM)
gemm_split_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Epilogue<bf16> ep, int64_t Mr, int64_t Nc, int kblocks, int mt,
                  int S, Limits lim) {
    using C = SplitCfg<BN>;
    constexpr int NS = C::NS, KS = C::KS;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t bars[2 * NS + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[NS + s]); };
    const uint32_t accf = smem_u32(&bars[2 * NS]), drained = smem_u32(&bars[2 * NS + 1]);
    const Waiter wait{&abort_flag, lim.wait_ns};
    const Waiter drain{&abort_flag, lim.wait_ns > kDrainNs ? lim.wait_ns : kDrainNs};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const uint32_t base = smem_u32(sm);
    const int tile = blockIdx.x / S;
    const int m0 = (tile % mt) * 128, n0 = (tile / mt) * BN;
    const int k_lo = (int)((int64_t)kblocks * rank / S), k_hi = (int)((int64_t)kblocks * (rank + 1) / S);

    // Warp 0 sets up the barriers and goes on to load at once; the others meet after TMEM is there.
    // As in the pair kernel, the next kernel may start once this CTA holds its TMEM.
    if (warp == 0) {
        if (lane == 0) {
            for (int s = 0; s < NS; ++s) {
                mbar_init(full(s), 1);
                mbar_init(empty(s), 1);
            }
            mbar_init(accf, 1);
            mbar_init(drained, 1);
            abort_flag = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("bar.arrive 1, %0;" :: "n"(THREADS) : "memory");
    } else {
        if (warp == 1) {
            tmem_alloc(smem_u32(&tmem_slot), C::TMEM_COLS);
            pdl_launch_next();
        }
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" :: "n"(THREADS) : "memory");
        tc_fence_after();
    }
    const uint32_t tm = warp == 0 ? 0u : tmem_slot;
    pdl_wait();                          // what the previous kernel wrote is there
    bool done = true;                    // the warp's wait completed

    if (warp == 0) {
        Ring<NS> ring;
        bool ok = true;
        int left = lim.stop;
        for (int kb = k_lo; kb < k_hi && left != 0; kb += KS, ring.next(), --left) {
            const int s = ring.s;
            if (!(ok = wait.warp(empty(s), ring.parity ^ 1u, E_STAGE))) break;
            if (elect_one()) {
                const int nb = k_hi - kb < KS ? k_hi - kb : KS;
                mbar_arrive_tx(full(s), C::BLOCK * nb);
#pragma unroll
                for (int u = 0; u < KS; ++u) {
                    if (u >= nb) break;
                    const uint32_t a = base + s * C::STAGE + u * C::BLOCK, b = a + C::A_BYTES;
                    const int k = (kb + u) * BK;
                    if constexpr (A_MN) {
                        tma_load_2d(a, &maps.a, full(s), m0, k);
                        tma_load_2d(a + BLK, &maps.a, full(s), m0 + 64, k);
                    } else {
                        tma_load_2d(a, &maps.a, full(s), k, m0);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int j = 0; j < BN / 64; ++j) tma_load_2d(b + j * BLK, &maps.b, full(s), n0 + 64 * j, k);
                    } else {
                        tma_load_2d(b, &maps.b, full(s), k, n0);
                    }
                }
            }
            __syncwarp();
        }
        if (!ok) pause_ns(kLandNs);
        __syncwarp();
    } else if (warp == 1) {
        constexpr uint32_t ID = idesc(128, BN, A_MN, B_MN);
        const uint64_t da0 = base_desc<A_MN>(base), db0 = base_desc<B_MN>(base + C::A_BYTES);
        Ring<NS> ring;
        bool ok = true;
        for (int kb = k_lo; kb < k_hi; kb += KS, ring.next()) {
            const int s = ring.s;
            if (!(ok = wait.warp(full(s), ring.parity, E_STAGE))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int u = 0; u < KS; ++u) {
                    if (kb + u >= k_hi) break;
                    const uint32_t off = (uint32_t)(s * (C::STAGE >> 4) + u * (C::BLOCK >> 4));
#pragma unroll
                    for (int k = 0; k < BK / 16; ++k)
                        mma_bf16(tm, da0 + off + k * K16<A_MN>, db0 + off + k * K16<B_MN>, ID,
                                 (kb > k_lo || u > 0 || k > 0) ? 1u : 0u);
                }
                mma_commit(empty(s));
                if (kb + KS >= k_hi) mma_commit(accf);
            }
            __syncwarp();
        }
        if (!ok) {
            // every MMA issued so far: TMEM must be idle before it is freed
            if (elect_one()) mma_commit(drained);
            drain.warp(drained, 0u, E_DRAIN, false);
        }
        __syncwarp();
    }

    const int q = warp & 3, h = (warp - 2) >> 2;
    const int64_t r = (int64_t)m0 + 32 * q + lane;
    const uint32_t tq = tm + ((uint32_t)(32 * q) << 16);
    const float bias = warp >= 2 && ep.bias && r < Mr ? __ldg(ep.bias + r) : 0.f;
    constexpr int HALF = BN / 2;
    // a whole tile's residual, on its way while the sums are formed
    bf16 res[HALF];
    if (warp >= 2) {
        if (S == 1 && ep.residual) {
#pragma unroll
            for (int c = 0; c < HALF; ++c)
                if (n0 + h * HALF + c < Nc && r < Mr) res[c] = __ldg(ep.residual + (n0 + (int64_t)h * HALF + c) * Mr + r);
        }
        done = wait.over(k_hi - k_lo).warp(accf, 0u, E_ACC);
        tc_fence_after();
    }
    if (S == 1) {
        // a thread owns a row; its stores and those of its warp's other lanes are contiguous
        if (warp >= 2 && done) {
            const int c_lo = h * HALF, c_hi = c_lo + HALF < Nc - n0 ? c_lo + HALF : (int)(Nc - n0);
            with_act(ep.act, [&](auto kind) {
#pragma unroll
                for (int i = 0; i < HALF; i += 8) {
                    const int c = c_lo + i;
                    if (c >= c_hi) break;
                    float v[8];
                    tmem_ld8(tq + c, v);
                    int64_t at = (n0 + (int64_t)c) * Mr + r;
#pragma unroll
                    for (int j = 0; j < 8; ++j, at += Mr)
                        if (c + j < c_hi && r < Mr) {
                            const float z = v[j] + bias;
                            if (ep.z) store_elem(ep.z + at, z);
                            float o = act_value<kind(), true>(z);
                            if (ep.residual) o += to_f32(res[i + j]);
                            store_elem(ep.D + at, o);
                        }
                }
            });
        }
    } else {
        // The partial tile goes over the stages (their loads have been consumed), [column][128 rows].
        // In that order CTA r adds up the r-th part of it, four rows of a column per thread: 16-byte
        // reads of the other CTAs' shared memory, several times the rate of 4-byte ones.
        float* part = reinterpret_cast<float*>(sm);
        if (warp >= 2 && done) {
#pragma unroll 1
            for (int c = h * HALF; c < (h + 1) * HALF; c += 8) {
                float v[8];
                tmem_ld8(tq + c, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) part[(c + j) * 128 + 32 * q + lane] = v[j];
            }
        }
        __syncwarp();
        cluster_sync_all();
        if (warp >= 2 && done) {
            const int share = BN * 32 / S;             // groups of four rows
            with_act(ep.act, [&](auto kind) {
#pragma unroll 1
                for (int i = threadIdx.x - 64; i < share; i += 32 * EPI) {
                    const int g = rank * share + i, c = g / 32;
                    const int64_t r4 = (int64_t)m0 + 4 * (g % 32);
                    if (n0 + c >= Nc || r4 >= Mr) continue;
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
                    for (int p = 0; p < S; ++p) {
                        const float4 f = ld_cluster_v4(mapa(base + 16 * g, (uint32_t)p));
                        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
                    }
                    const int64_t at = (n0 + (int64_t)c) * Mr + r4;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (r4 + j < Mr) {
                            const float z = v[j] + (ep.bias ? __ldg(ep.bias + r4 + j) : 0.f);
                            if (ep.z) store_elem(ep.z + at + j, z);
                            float o = act_value<kind(), true>(z);
                            if (ep.residual) o += to_f32(__ldg(ep.residual + at + j));
                            store_elem(ep.D + at + j, o);
                        }
                }
            });
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

// An output of M rows of N elements, stored in blocks of 32 x CW
template <typename T>
bool make_map_out(CUtensorMap* map, void* p, int64_t M, int64_t N) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
    const cuuint64_t str[1] = {(cuuint64_t)N * sizeof(T)};
    const cuuint32_t box[2] = {CW, 32};
    const cuuint32_t e1[2] = {1, 1};
    return enc(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p, dims, str,
               box, e1, CU_TENSOR_MAP_INTERLEAVE_NONE,
               sizeof(T) == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a pair kernel's outputs, where it stores through them
template <typename T>
bool output_maps(Maps* maps, const Epilogue<T>& ep, int64_t M, int64_t N) {
    return !ep.vec || (make_map_out<T>(&maps->d, ep.D, M, N) && (!ep.z || make_map_out<T>(&maps->z, ep.z, M, N)));
}

// The three planes of an fp32 operand, `plane` elements apart: boxes of 64 x (box_rows or 64) x 3
bool make_map_planes(CUtensorMap* map, const void* p, int64_t rows, int64_t K, int64_t ld, int64_t plane, bool mn,
                     int box_rows) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)(mn ? rows : K), (cuuint64_t)(mn ? K : rows), 3};
    const cuuint64_t str[2] = {(cuuint64_t)ld * 2, (cuuint64_t)plane * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)(mn ? 64 : box_rows), 3};
    const cuuint32_t e1[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, str, box, e1,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<unsigned long long> g_wait_ns{kWaitNs};
std::atomic<int> g_stop{-1};

Limits limits() { return Limits{g_wait_ns.load(), g_stop.load()}; }

template <typename K>
cudaError_t allow_smem(K kern, int bytes) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T>
Epilogue<T> epilogue_of(const GemmArgs& g) {
    Epilogue<T> ep;
    ep.bias = g.bias;
    ep.residual = static_cast<const T*>(g.residual);
    ep.D = static_cast<T*>(g.D);
    ep.z = static_cast<T*>(g.z);
    ep.act = g.act;
    ep.vec = g.N % Vec16<T>::VEC == 0 && (uintptr_t)g.D % 16 == 0 && (uintptr_t)g.z % 16 == 0 &&
             (uintptr_t)g.residual % 16 == 0;
    return ep;
}

// The blocks of 256 x BN floats that hold the parts of shared tiles, stored in boxes of 32 x 16
bool make_map_parts(CUtensorMap* map, void* p, int64_t blocks, int bn) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)bn, (cuuint64_t)(256 * blocks)};
    const cuuint64_t str[1] = {(cuuint64_t)bn * 4};
    const cuuint32_t box[2] = {16, 32};
    const cuuint32_t e1[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p, dims, str, box, e1, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Work work_of(int64_t M, int64_t N, int64_t K, int bn, int S) {
    Work w{};
    w.mt = (int)((M + 255) / 256);
    w.nt = (int)((N + bn - 1) / bn);
    w.kblocks = (int)((K + BK - 1) / BK);
    w.S = S;
    const int64_t tiles = (int64_t)w.mt * w.nt;
    w.full = S > 1 ? tiles / PAIRS * PAIRS : tiles;
    w.items = w.full + (tiles - w.full) * S;
    return w;
}

// The pair kernel on its work, and the sums of the shared tiles after it
template <typename T, int BN, typename K, typename... More>
cudaError_t launch_pairs(K kern, int smem, Maps& maps, const GemmArgs& g, int S, int sms, More... more) {
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    const Epilogue<T> ep = epilogue_of<T>(g);
    const Work w = work_of(g.M, g.N, g.K, BN, S);
    const int64_t shared = w.items - w.full, pairs = sms / 2;
    if (!output_maps(&maps, ep, g.M, g.N) || (shared && !make_map_parts(&maps.p, g.part, shared, BN)))
        return cudaErrorInvalidValue;
    const unsigned grid = 2u * (unsigned)(w.items < pairs ? w.items : pairs);
    e = launch_pdl(kern, dim3(grid), dim3(PAIR_THREADS), (size_t)smem, g.stream, maps, ep, g.M, g.N, w, limits(),
                   more...);
    if (e != cudaSuccess || !shared) return e;
    return launch_pdl(join_kernel<T, BN>, dim3(BN / 4, (unsigned)(shared / S)), dim3(256), 0, g.stream,
                      static_cast<const float*>(g.part), ep, g.M, g.N, w);
}

template <int BN, bool A_MN, bool B_MN>
cudaError_t pair_launch(const GemmArgs& g, int S, int sms) {
    Maps maps{};
    if (!make_map(&maps.a, g.A, g.M, g.K, g.lda, A_MN, 128) || !make_map(&maps.b, g.B, g.N, g.K, g.ldb, B_MN, BN / 2))
        return cudaErrorInvalidValue;
    return launch_pairs<bf16, BN>(gemm_pair_kernel<BN, A_MN, B_MN>, PairCfg<BN>::SMEM, maps, g, S, sms);
}

template <int BN>
cudaError_t pair_layout(const GemmArgs& g, int S, int sms) {
    if (g.a_mn) return g.b_mn ? pair_launch<BN, true, true>(g, S, sms) : cudaErrorInvalidValue;
    return g.b_mn ? pair_launch<BN, false, true>(g, S, sms) : pair_launch<BN, false, false>(g, S, sms);
}

template <bool A_MN, bool B_MN>
cudaError_t f32_launch(const GemmArgs& g, const F32Planes& f, int S, int sms) {
    constexpr int BN = F32Cfg::BN;
    Maps maps{};
    if (!make_map_planes(&maps.a, f.A, g.M, g.K, f.lda, f.a_plane, A_MN, 128) ||
        !make_map_planes(&maps.b, f.B, g.N, g.K, f.ldb, f.b_plane, B_MN, BN / 2))
        return cudaErrorInvalidValue;
    return launch_pairs<float, BN>(gemm_f32_kernel<A_MN, B_MN>, F32Cfg::SMEM, maps, g, S, sms, f.over);
}

template <int BN, bool A_MN, bool B_MN>
cudaError_t split_launch(const GemmArgs& g, int S) {
    using C = SplitCfg<BN>;
    auto kern = gemm_split_kernel<BN, A_MN, B_MN>;
    cudaError_t e = allow_smem(kern, C::SMEM);
    if (e != cudaSuccess) return e;
    Maps maps{};                         // the product's B side on the MMA rows
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
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)S;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, epilogue_of<bf16>(g), g.N, g.M, (int)((g.K + BK - 1) / BK), mt, S,
                              limits());
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

namespace {

// Which kernel runs a product.
struct Plan {
    int pair_bn;                         // 256 or 128: the pair kernel; 0: the split kernel
    int bn, S;                           // of the split kernel; S: clusters per tile, of the pair kernel's last round
};

constexpr int SMS = 2 * lintc::PAIRS;

// The time, in us, of a pair kernel whose K blocks take `per_kb` each and whose tiles at least `least`, and the
// best number S of pairs for a tile of its last round.  Sharing takes a second kernel (3 us) and the traffic of
// the parts (rem S blocks of bn x 1 KB).  A shared tile adds up K in another order than a whole one, so a product
// whose rows are tokens shares all its tiles or none: equal tokens of a call get equal bits.  (a_mn: rows are
// channels.)
double pair_time(int64_t M, int64_t N, int64_t K, bool a_mn, int bn, double per_kb, double least, int* S) {
    const int64_t kb = (K + 63) / 64, tiles = ((M + 255) / 256) * ((N + bn - 1) / bn);
    const int64_t full = tiles / lintc::PAIRS, rem = tiles % lintc::PAIRS;
    const double tile = std::max(per_kb * kb, least);
    *S = 1;
    if (!rem) return full * tile;
    if (full && !a_mn) return (full + 1) * tile;
    double last = tile;
    for (int s = 2; s <= 16 && rem * s <= lintc::PAIRS && kb >= 4 * s; ++s) {
        const double t = std::max(per_kb * ((kb + s - 1) / s), least) + 3.0 + 0.06 * rem * s * bn / 256;
        if (t < last) {
            last = t;
            *S = s;
        }
    }
    return full * tile + last;
}

// Up to 64 rows of A, the split kernel with the narrowest MMA N that holds them, and K split until two
// CTAs per SM stream the other operand.  Above that, the smallest of these times, in us, with kb
// blocks of 64 along K and w rounds of tiles over the device; measured with the operands in L2 (T from
// 100 to 8192, K and N from 256 to 16384), each within a fifth of its kernel's time:
//   pair, 256 x 256   w max(0.30 kb, 2.9)      28 at T = 1024, 4096 -> 4096 (256 x 128: 31, split: 43)
//   pair, 256 x 128   w max(0.185 kb, 2.0)     8.0 at T = 512, 1024 -> 1024 (256 x 256: 11, split: 9.4)
//   split by S        w (0.23 kb / S + 3.5) - 3, and 3 more to join the parts
//                                              17 at T = 333, 8192 -> 1000 with S = 4 (pair: 29)
Plan plan(int64_t M, int64_t N, int64_t K, bool a_mn) {
    Plan p{};
    const int64_t kb = (K + 63) / 64, rows = (N + 127) / 128;
    auto rounds = [](int64_t tiles, int64_t at_once) { return (double)((tiles + at_once - 1) / at_once); };
    if (M <= 64) {
        p.bn = a_mn || M > 32 ? 64 : M > 16 ? 32 : 16;    // a product over tokens has boxes of 64
        const int64_t tiles = rows;
        p.S = 1;
        while (p.S < 8 && tiles * p.S * 2 <= 2 * SMS && kb >= p.S * 4) p.S *= 2;
        return p;
    }
    int s256, s128;
    double best = pair_time(M, N, K, a_mn, 256, 0.30, 2.9, &s256);
    const double half = pair_time(M, N, K, a_mn, 128, 0.185, 2.0, &s128);
    p.pair_bn = 256;
    p.S = s256;
    if (half < best) {
        best = half;
        p.pair_bn = 128;
        p.S = s128;
    }
    p.bn = 128;
    for (int S = 1; S <= 8 && kb >= 2 * S - 1; S *= 2) {
        // clusters at once: a GPC of 16 to 20 SMs holds two clusters of 8
        const int64_t at_once = S == 8 ? SMS * 3 / 32 : SMS / S;
        const double t = rounds(rows * ((M + 127) / 128), at_once) * (0.23 * kb / S + 3.5 + (S > 1 ? 3.0 : 0.0)) - 3.0;
        if (t < best) {
            best = t;
            p.pair_bn = 0;
            p.S = S;
        }
    }
    return p;
}

double f32_time(int64_t M, int64_t N, int64_t K, bool a_mn, int* S) {
    return pair_time(M, N, K, a_mn, lintc::F32Cfg::BN, 1.1, 4.0, S);
}

size_t part_bytes(int64_t M, int64_t N, int64_t K, int bn, int S) {
    const lintc::Work w = lintc::work_of(M, N, K, bn, S);
    return (size_t)(w.items - w.full) * 256 * bn * 4;
}

}  // namespace

size_t gemm_tc_part_bytes(int64_t M, int64_t N, int64_t K, bool a_mn) {
    const Plan p = plan(M, N, K, a_mn);
    return p.pair_bn ? part_bytes(M, N, K, p.pair_bn, p.S) : 0;
}

size_t gemm_f32_part_bytes(int64_t M, int64_t N, int64_t K, bool a_mn) {
    int S;
    f32_time(M, N, K, a_mn, &S);
    return part_bytes(M, N, K, lintc::F32Cfg::BN, S);
}

double gemm_f32_time(int64_t M, int64_t N, int64_t K, bool a_mn) {
    int S;
    return f32_time(M, N, K, a_mn, &S);
}

cudaError_t launch_gemm_tc(const GemmArgs& g) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    const Plan p = plan(g.M, g.N, g.K, g.a_mn);
    if (p.pair_bn == 256) return lintc::pair_layout<256>(g, p.S, di.sm_count);
    if (p.pair_bn == 128) return lintc::pair_layout<128>(g, p.S, di.sm_count);
    switch (p.bn) {
        case 16: return lintc::split_layout<16>(g, p.S);
        case 32: return lintc::split_layout<32>(g, p.S);
        case 64: return lintc::split_layout<64>(g, p.S);
        default: return lintc::split_layout<128>(g, p.S);
    }
}

cudaError_t launch_gemm_f32(const GemmArgs& g, const F32Planes& f) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    int S;
    f32_time(g.M, g.N, g.K, g.a_mn, &S);
    if (g.a_mn) return g.b_mn ? lintc::f32_launch<true, true>(g, f, S, di.sm_count) : cudaErrorInvalidValue;
    return g.b_mn ? lintc::f32_launch<false, true>(g, f, S, di.sm_count)
                  : lintc::f32_launch<false, false>(g, f, S, di.sm_count);
}

void linear_tc_set_stop(int stop, unsigned long long wait_ns) {
    lintc::g_stop.store(stop);
    lintc::g_wait_ns.store(wait_ns);
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
