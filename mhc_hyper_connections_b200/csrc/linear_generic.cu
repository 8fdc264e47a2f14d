// linear_generic.cu -- D[m][n] = act(sum_k A(m, k) B(n, k) + bias[n]) + residual[m][n] on CUDA
// cores: any size, alignment and storage type, with either index of A and B contiguous.  It runs
// the fp32 products of few tokens or few operations, those with values that the tensor-core form has
// no parts for, and the bf16 products whose addresses the tensor-core kernels refuse.
//
// 2 M N K operations against 128 FMAs per SM and clock bound it (few tokens: the larger operand's
// bytes).  A block forms a BM x BN tile, a thread TM x TN of it in registers (in groups of up to four
// consecutive rows and columns, so that shared memory is read in vectors without conflicts); operands
// go through shared memory as fp32, k-major, 16 deep, with the next step's elements already in
// registers.  Where the tiles leave SMs idle, a cluster of S blocks splits K: each leaves its partial
// tile in its shared memory and adds up its share of the rows over the cluster in rank order.
#include "activation.cuh"
#include "tc_ptx.cuh"

namespace mhc {
namespace {

constexpr int BK = 16;
constexpr int THREADS = 256;

// Four elements along the contiguous index: a vector where rows are 16-byte aligned fp32 and all four
// are inside
template <typename T>
__device__ __forceinline__ void load4(const T* p, int64_t left, bool vec, float (&f)[4]) {
    if constexpr (sizeof(T) == 4) {
        if (vec && left >= 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p));
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = e < left ? to_f32(__ldg(p + e)) : 0.f;
}

// A thread's share of a ROWS x BK operand tile, and its place in shared memory
template <typename T, int ROWS, bool MN>
struct Loader {
    static constexpr int PER = ROWS * BK / THREADS, VECS = PER / 4;
    static constexpr int PITCH = ROWS + 4;
    float f[PER];

    __device__ __forceinline__ void fetch(const T* p, int64_t ld, int64_t row0, int64_t rows, int64_t k0, int64_t k1,
                                          bool vec) {
        if constexpr (VECS == 0) {
            const int r = MN ? threadIdx.x % ROWS : threadIdx.x / BK, k = MN ? threadIdx.x / ROWS : threadIdx.x % BK;
            const bool in = row0 + r < rows && k0 + k < k1;
            f[0] = in ? to_f32(__ldg(p + (MN ? (k0 + k) * ld + row0 + r : (row0 + r) * ld + k0 + k))) : 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                const int v = threadIdx.x + j * THREADS;
                float (&g)[4] = *reinterpret_cast<float(*)[4]>(f + 4 * j);
                const int r = MN ? v % (ROWS / 4) * 4 : v / (BK / 4), k = MN ? v / (ROWS / 4) : v % (BK / 4) * 4;
                const int64_t row = row0 + r, kk = k0 + k;
                if (MN ? kk < k1 : row < rows)
                    load4(p + (MN ? kk * ld + row : row * ld + kk), MN ? rows - row : k1 - kk, vec, g);
                else
                    g[0] = g[1] = g[2] = g[3] = 0.f;
            }
        }
    }
    __device__ __forceinline__ void store(float (*sm)[PITCH]) const {
        if constexpr (VECS == 0) {
            const int r = MN ? threadIdx.x % ROWS : threadIdx.x / BK, k = MN ? threadIdx.x / ROWS : threadIdx.x % BK;
            sm[k][r] = f[0];
        } else {
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                const int v = threadIdx.x + j * THREADS;
                if constexpr (MN) {
                    *reinterpret_cast<float4*>(&sm[v / (ROWS / 4)][v % (ROWS / 4) * 4]) =
                        make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) sm[v % (BK / 4) * 4 + e][v / (BK / 4)] = f[4 * j + e];
                }
            }
        }
    }
};

// N consecutive floats of shared memory
template <int N>
__device__ __forceinline__ void read_n(const float* p, float* f) {
    if constexpr (N == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x; f[1] = v.y;
    }
}

// Tiles: 128 x 128 (8 x 8 per thread), 64 x 64 (4 x 4), and 16 x 128 (2 x 4) for few rows of A.
// ONLY_IF: does nothing unless one of only_if_n words is set.
template <typename T, int BM, int BN, int TM, int TN, bool A_MN, bool B_MN, bool ONLY_IF>
__global__ void __launch_bounds__(THREADS)
gemm_kernel(const T* __restrict__ A, const T* __restrict__ B, int64_t lda, int64_t ldb, int64_t M, int64_t N,
            int64_t K, const float* __restrict__ bias, const T* __restrict__ residual, int act, T* __restrict__ D,
            T* __restrict__ z, int S, bool veca, bool vecb, bool vecd, const int* __restrict__ only_if, int only_if_n) {
    constexpr int GX = BN / TN;                        // threads along n; THREADS / GX along m
    constexpr int VM = TM < 4 ? TM : 4, VN = 4;        // consecutive rows and columns of a thread
    static_assert(GX * (BM / TM) == THREADS, "threads cover the tile");
    using LA = Loader<T, BM, A_MN>;
    using LB = Loader<T, BN, B_MN>;
    constexpr int SM_FLOATS = BK * (LA::PITCH + LB::PITCH);
    constexpr bool SPLITS = BM * BN <= 64 * 64;        // the partial tile fits
    __shared__ __align__(16) float smem[SPLITS && BM * BN > SM_FLOATS ? BM * BN : SM_FLOATS];
    float (*As)[LA::PITCH] = reinterpret_cast<float (*)[LA::PITCH]>(smem);
    float (*Bs)[LB::PITCH] = reinterpret_cast<float (*)[LB::PITCH]>(smem + BK * LA::PITCH);
    const int tid = threadIdx.x, tx = tid % GX, ty = tid / GX;
    const int rank = SPLITS && S > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int64_t mt = (M + BM - 1) / BM, tile = blockIdx.x / S;
    const int64_t m0 = tile % mt * BM, n0 = tile / mt * BN;
    const int64_t steps = (K + BK - 1) / BK;
    const int64_t kb = steps * rank / S * BK, ke = steps * (rank + 1) / S * BK < K ? steps * (rank + 1) / S * BK : K;
    pdl_launch_next();
    pdl_wait();
    if constexpr (ONLY_IF) {
        int any = 0;
        for (int i = tid; i < only_if_n; i += THREADS) any |= only_if[i];
        if (!__syncthreads_or(any)) return;            // the same answer in every block
    }

    float acc[TM][TN] = {};
    LA la;
    LB lb;
    auto fetch = [&](int64_t k) {
        la.fetch(A, lda, m0, M, k, ke, veca);
        lb.fetch(B, ldb, n0, N, k, ke, vecb);
    };
    // row i (column j) of this thread within the tile
    auto row = [&](int i) { return (i / VM) * (BM * VM / TM) + ty * VM + i % VM; };
    auto col = [&](int j) { return (j / VN) * (BN * VN / TN) + tx * VN + j % VN; };
    fetch(kb);
    for (int64_t k0 = kb; k0 < ke; k0 += BK) {
        la.store(As);
        lb.store(Bs);
        __syncthreads();
        if (k0 + BK < ke) fetch(k0 + BK);
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; i += VM) read_n<VM>(&As[k][row(i)], a + i);
#pragma unroll
            for (int j = 0; j < TN; j += VN) read_n<VN>(&Bs[k][col(j)], b + j);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    auto finish = [&](auto kind, int64_t m, int64_t n, float v) {
        if (bias) v += __ldg(bias + n);
        if (z) store_elem(z + m * N + n, v);
        float o = act_value<kind(), sizeof(T) == 2>(v);
        if (residual) o += to_f32(__ldg(residual + m * N + n));
        store_elem(D + m * N + n, o);
    };
    if constexpr (SPLITS) {
        if (S > 1) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) smem[row(i) * BN + col(j)] = acc[i][j];
            ptx::cluster_sync_all();
            with_act(act, [&](auto kind) {
                for (int e = rank * (BM * BN / S) + tid; e < (rank + 1) * (BM * BN / S); e += THREADS) {
                    const int64_t m = m0 + e / BN, n = n0 + e % BN;
                    if (m >= M || n >= N) continue;
                    float v = 0.f;
#pragma unroll 8
                    for (int p = 0; p < S; ++p) {
                        float f;
                        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                     : "=f"(f) : "r"(ptx::mapa(ptx::smem_u32(smem + e), (uint32_t)p)) : "memory");
                        v += f;
                    }
                    finish(kind, m, n, v);
                }
            });
            ptx::cluster_sync_all();                   // no block leaves while its part is read
            return;
        }
    }
    with_act(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + row(i);
            if (m >= M) continue;
#pragma unroll
            for (int j = 0; j < TN; j += VN) {
                const int64_t n = n0 + col(j);
                if constexpr (sizeof(T) == 4) {
                    if (vecd) {                        // N a multiple of 4: all four columns, or none
                        if (n >= N) continue;
                        float v[4], r[4] = {0.f, 0.f, 0.f, 0.f};
                        if (residual) Vec16<float>::unpack(ld_stream_v4(residual + m * N + n), r);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = acc[i][j + e] + (bias ? __ldg(bias + n + e) : 0.f);
                        if (z) st_v4(z + m * N + n, Vec16<float>::pack(v));
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = act_value<kind(), false>(v[e]) + r[e];
                        st_v4(D + m * N + n, Vec16<float>::pack(v));
                        continue;
                    }
                }
#pragma unroll
                for (int e = 0; e < VN; ++e)
                    if (n + e < N) finish(kind, m, n + e, acc[i][j + e]);
            }
        }
    });
}

template <typename T, int BM, int BN, int TM, int TN, bool A_MN, bool B_MN, bool ONLY_IF>
cudaError_t launch(const GemmArgs& g, int S, const int* only_if, int only_if_n) {
    const int64_t tiles = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
    if (tiles * S > INT32_MAX) return cudaErrorInvalidValue;
    auto vec = [](const void* p, int64_t ld) { return sizeof(T) == 4 && ld % 4 == 0 && (uintptr_t)p % 16 == 0; };
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * S));
    cfg.blockDim = dim3(THREADS);
    cfg.stream = g.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)S;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<T, BM, BN, TM, TN, A_MN, B_MN, ONLY_IF>, static_cast<const T*>(g.A),
                              static_cast<const T*>(g.B), g.lda, g.ldb, g.M, g.N, g.K, g.bias,
                              static_cast<const T*>(g.residual), (int)g.act, static_cast<T*>(g.D),
                              static_cast<T*>(g.z), S, vec(g.A, g.lda), vec(g.B, g.ldb),
                              vec(g.D, g.N) && vec(g.z, g.N) && vec(g.residual, g.N), only_if, only_if_n);
}

// 128 x 128 tiles reuse each loaded element twice as often as 64 x 64 ones, which run where the large tiles would
// leave SMs without one; up to 16 rows of A, tiles of 16.  S: blocks that share a tile.
struct Tiling {
    int rows, S;
    int64_t tiles;
};
Tiling tiling(int64_t M, int64_t N, int64_t K, int sms) {
    auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
    if (M > 16 && tiles(128, 128) >= sms) return Tiling{128, 1, tiles(128, 128)};
    Tiling t{M > 16 ? 64 : 16, 1, M > 16 ? tiles(64, 64) : tiles(16, 128)};
    while (t.S < 8 && t.tiles * t.S * 2 <= 4 * sms && K >= 128 * t.S) t.S *= 2;      // up to four blocks per SM, 64 of K each
    return t;
}

template <typename T, bool A_MN, bool B_MN>
cudaError_t pick(const GemmArgs& g, const int* only_if, int only_if_n) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    if constexpr (sizeof(T) == 4) {
        if (only_if) return launch<T, 128, 128, 8, 8, A_MN, B_MN, true>(g, 1, only_if, only_if_n);
    }
    const Tiling t = tiling(g.M, g.N, g.K, di.sm_count);
    if (t.rows == 128) return launch<T, 128, 128, 8, 8, A_MN, B_MN, false>(g, 1, nullptr, 0);
    return t.rows == 64 ? launch<T, 64, 64, 4, 4, A_MN, B_MN, false>(g, t.S, nullptr, 0)
                        : launch<T, 16, 128, 2, 4, A_MN, B_MN, false>(g, t.S, nullptr, 0);
}

template <typename T>
cudaError_t pick_layout(const GemmArgs& g, const int* o, int n) {
    if (g.a_mn) return g.b_mn ? pick<T, true, true>(g, o, n) : cudaErrorInvalidValue;
    return g.b_mn ? pick<T, false, true>(g, o, n) : pick<T, false, false>(g, o, n);
}

}  // namespace

// Measured over T = 9 to 2048, K and N = 256 to 4096, all three layouts (operands in L2): a step of 16 of K takes
// longer the more blocks an SM has.  Off by a seventh (rms).  148 SMs whatever the device: the workspace's size
// follows from it.
double gemm_generic_time(int64_t M, int64_t N, int64_t K) {
    const Tiling t = tiling(M, N, K, 148);
    const double steps = (double)(((K + BK - 1) / BK + t.S - 1) / t.S), more = (double)((t.tiles * t.S + 147) / 148 - 1);
    if (t.rows == 16) return 3.7 + steps * (0.63 + 0.77 * more);
    return t.rows == 64 ? 3.2 + steps * (1.2 + 0.45 * more) : 7.0 + steps * (1.15 + 2.2 * more);
}

cudaError_t launch_gemm_generic(const GemmArgs& g, const int* only_if, int only_if_n) {
    return g.dt == BF16 ? pick_layout<__nv_bfloat16>(g, only_if, only_if_n) : pick_layout<float>(g, only_if, only_if_n);
}

}  // namespace mhc
