// linear_thin.cu -- the products of linear_generic.cu for up to 8 rows of A: a few tokens against a
// weight matrix.  The matrix B is read once, in the storage's own width; A's few rows come from L1.
// Bound by B's bytes.
//
//   * B's rows run along K (the forward product): thin_dot_kernel.  A warp forms COLS columns at once,
//     its lanes 16 bytes of K each; the warps of a block split K, and their lanes' sums are added by
//     shuffles and then in shared memory.
//   * B's rows run along N (dx = dz W): thin_axpy_kernel.  A lane owns 16 bytes of columns; the warps
//     of a block and the blocks of a cluster split K, and add their sums up in warp and rank order.
#include "activation.cuh"
#include "tc_ptx.cuh"

namespace mhc {
namespace {

constexpr int WARPS = 8;
constexpr int COLS = 4;

// VEC elements from element `at` of an array of `total`; elements past `left` read as zero
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, int64_t at, int64_t total, int64_t left, bool vec, float* f) {
    constexpr int VEC = Vec16<T>::VEC;
    if (left <= 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 0.f;
    } else if (vec && left >= VEC) {
        Vec16<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p + at)), f);
    } else if constexpr (sizeof(T) == 2) {
        Vec16<T>::unpack(ld_shifted_v4(p, at, total), f);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if (e >= left) f[e] = 0.f;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = e < left ? __ldg(p + at + e) : 0.f;
    }
}

template <typename T>
struct Out {
    const float* bias;
    const T* residual;
    T* D;
    T* z;
    int act;
};

template <typename T>
__device__ __forceinline__ void finish(const Out<T>& o, int64_t at, int64_t n, float v) {
    if (o.bias) v += __ldg(o.bias + n);
    if (o.z) store_elem(o.z + at, v);
    with_act(o.act, [&](auto kind) {
        float y = act_value<kind(), sizeof(T) == 2>(v);
        if (o.residual) y += to_f32(__ldg(o.residual + at));
        store_elem(o.D + at, y);
    });
}

template <typename T, int MT>
__global__ void __launch_bounds__(32 * WARPS)
thin_dot_kernel(const T* __restrict__ A, const T* __restrict__ B, int64_t lda, int64_t ldb, int M, int64_t N, int64_t K,
                const __grid_constant__ Out<T> out, bool veca, bool vecb) {
    constexpr int VEC = Vec16<T>::VEC;
    __shared__ float sm[WARPS][MT * COLS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n0 = (int64_t)blockIdx.x * COLS;
    pdl_launch_next();
    pdl_wait();
    float acc[MT][COLS] = {};
#pragma unroll 2
    for (int64_t k = (int64_t)(warp * 32 + lane) * VEC; k < K; k += WARPS * 32 * VEC) {
        float b[COLS][VEC];
#pragma unroll
        for (int c = 0; c < COLS; ++c)
            load_vec(B, (n0 + c) * ldb + k, N * ldb, n0 + c < N ? K - k : 0, vecb, b[c]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m >= M) break;
            float a[VEC];
            load_vec(A, m * lda + k, M * lda, K - k, veca, a);
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[m][c] = fmaf(a[e], b[c][e], acc[m][c]);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            float v = acc[m][c];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) sm[warp][m * COLS + c] = v;
        }
    __syncthreads();
    if (threadIdx.x < MT * COLS) {
        const int m = threadIdx.x / COLS;
        const int64_t n = n0 + threadIdx.x % COLS;
        if (m < M && n < N) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += sm[w][threadIdx.x];
            finish(out, m * N + n, n, v);
        }
    }
}

template <typename T, int MT>
__global__ void __launch_bounds__(32 * WARPS)
thin_axpy_kernel(const T* __restrict__ A, const T* __restrict__ B, int64_t lda, int64_t ldb, int M, int64_t N,
                 int64_t K, const __grid_constant__ Out<T> out, bool vecb, int S) {
    constexpr int VEC = Vec16<T>::VEC, COLUMNS = 32 * VEC, U = 4;
    __shared__ float sm[WARPS][MT * COLUMNS / 4];      // a quarter of the columns at a time
    __shared__ float part[MT * COLUMNS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = S > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int64_t n0 = (int64_t)(blockIdx.x / S) * COLUMNS, n = n0 + lane * VEC;
    const int64_t kb = K * rank / S, ke = K * (rank + 1) / S;
    pdl_launch_next();
    pdl_wait();
    float acc[MT][VEC] = {};
    for (int64_t k = kb + warp; k < ke; k += WARPS * U) {
        float b[U][VEC], a[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t kk = k + u * WARPS;
            load_vec(B, kk * ldb + n, K * ldb, kk < ke ? N - n : 0, vecb, b[u]);
#pragma unroll
            for (int m = 0; m < MT; ++m) a[u][m] = m < M && kk < ke ? to_f32(__ldg(A + m * lda + kk)) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (k + u * WARPS >= ke) break;            // 0 * inf would be NaN
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[m][e] = fmaf(a[u][m], b[u][e], acc[m][e]);
        }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {                      // lanes 8 p .. 8 p + 7 own the p-th quarter
        if (lane / 8 == p)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < VEC; ++e) sm[warp][m * (COLUMNS / 4) + lane % 8 * VEC + e] = acc[m][e];
        __syncthreads();
        for (int i = threadIdx.x; i < MT * COLUMNS / 4; i += 32 * WARPS) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) v += sm[w][i];
            part[i / (COLUMNS / 4) * COLUMNS + p * (COLUMNS / 4) + i % (COLUMNS / 4)] = v;
        }
        __syncthreads();
    }
    if (S > 1) ptx::cluster_sync_all();
    for (int i = rank * (MT * COLUMNS / S) + threadIdx.x; i < (rank + 1) * (MT * COLUMNS / S); i += 32 * WARPS) {
        const int m = i / COLUMNS;
        const int64_t c = n0 + i % COLUMNS;
        if (m >= M || c >= N) continue;
        float v = 0.f;
        if (S > 1) {
#pragma unroll 8
            for (int p = 0; p < S; ++p) {
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(f) : "r"(ptx::mapa(ptx::smem_u32(part + i), (uint32_t)p)) : "memory");
                v += f;
            }
        } else {
            v = part[i];
        }
        finish(out, m * N + c, c, v);
    }
    if (S > 1) ptx::cluster_sync_all();                // no block leaves while its part is read
}

template <typename T, int MT>
cudaError_t launch(const GemmArgs& g, int sms) {
    constexpr int VEC = Vec16<T>::VEC;
    auto vec = [](const void* p, int64_t ld) { return ld % VEC == 0 && (uintptr_t)p % 16 == 0; };
    const Out<T> out{g.bias, static_cast<const T*>(g.residual), static_cast<T*>(g.D), static_cast<T*>(g.z), (int)g.act};
    const T* A = static_cast<const T*>(g.A);
    const T* B = static_cast<const T*>(g.B);
    const bool vb = vec(g.B, g.ldb);
    if (!g.b_mn)
        return launch_pdl(thin_dot_kernel<T, MT>, dim3((unsigned)((g.N + COLS - 1) / COLS)), dim3(32 * WARPS), 0,
                          g.stream, A, B, g.lda, g.ldb, (int)g.M, g.N, g.K, out, vec(g.A, g.lda), vb);
    const int64_t tiles = (g.N + 32 * VEC - 1) / (32 * VEC);
    int S = 1;                                         // four blocks per SM, four rows of B per warp
    while (S < 8 && tiles * S * 2 <= 4 * sms && g.K >= 2 * S * WARPS * 4) S *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * S));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.stream = g.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)S;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, thin_axpy_kernel<T, MT>, A, B, g.lda, g.ldb, (int)g.M, g.N, g.K, out, vb, S);
}

template <typename T>
cudaError_t pick(const GemmArgs& g, int sms) {
    if (g.M <= 1) return launch<T, 1>(g, sms);
    if (g.M <= 2) return launch<T, 2>(g, sms);
    if (g.M <= 4) return launch<T, 4>(g, sms);
    return launch<T, 8>(g, sms);
}

}  // namespace

bool gemm_thin_ok(const GemmArgs& g) { return g.M <= 8 && !g.a_mn; }

cudaError_t launch_gemm_thin(const GemmArgs& g) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    return g.dt == BF16 ? pick<__nv_bfloat16>(g, di.sm_count) : pick<float>(g, di.sm_count);
}

}  // namespace mhc
