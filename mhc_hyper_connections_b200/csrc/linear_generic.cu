// linear_generic.cu -- D[m][n] = act(sum_k A(m, k) B(n, k) + bias[n]) + residual[m][n] on CUDA
// cores: any size, alignment and storage type, with either index of A and B contiguous.  It runs
// the fp32 products, whose 24 significant bits the tensor cores do not keep in one pass, and the
// bf16 ones that the tensor-core kernel refuses.
//
// 2 M N K operations against 128 FMAs per SM and clock bound it.  A block forms a BM x BN tile, a
// thread TM x TM of it in registers (rows and columns TX apart in groups of four, so that shared
// memory is read in 16-byte vectors without conflicts); operands go through shared memory as fp32,
// k-major, 16 deep, with the next step's elements already in registers.
#include "activation.cuh"

namespace mhc {
namespace {

constexpr int BK = 16;
constexpr int THREADS = 256;

// TM = 8: 128 x 128 tiles; TM = 4: 64 x 64 tiles, for products with few tiles
template <typename T, int TM, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(THREADS)
gemm_kernel(const T* __restrict__ A, const T* __restrict__ B, int64_t lda, int64_t ldb, int64_t M, int64_t N,
            int64_t K, const float* __restrict__ bias, const T* __restrict__ residual, int act, T* __restrict__ D,
            T* __restrict__ z) {
    constexpr int BM = 16 * TM;                    // the tile is BM x BM
    constexpr int LD = BM * BK / THREADS;          // elements of A (and of B) a thread loads per step
    constexpr int PITCH = BM + 4;
    __shared__ __align__(16) float As[BK][PITCH], Bs[BK][PITCH];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int64_t mt = (M + BM - 1) / BM;
    const int64_t m0 = (int64_t)(blockIdx.x % mt) * BM, n0 = (int64_t)(blockIdx.x / mt) * BM;

    pdl_launch_next();
    pdl_wait();

    float acc[TM][TM] = {};
    float ra[LD], rb[LD];
    // element j of this thread: (row, k) within the tile, consecutive threads along the contiguous index
    auto place = [&](bool mn, int j, int& row, int& k) {
        const int e = tid + j * THREADS;
        row = mn ? e % BM : e / BK;
        k = mn ? e / BM : e % BK;
    };
    auto fetch = [&](int64_t k0) {
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            int r, k;
            place(A_MN, j, r, k);
            const int64_t m = m0 + r, ka = k0 + k;
            ra[j] = m < M && ka < K ? to_f32(__ldg(A + (A_MN ? ka * lda + m : m * lda + ka))) : 0.f;
            place(B_MN, j, r, k);
            const int64_t n = n0 + r, kb = k0 + k;
            rb[j] = n < N && kb < K ? to_f32(__ldg(B + (B_MN ? kb * ldb + n : n * ldb + kb))) : 0.f;
        }
    };
    fetch(0);
    for (int64_t k0 = 0; k0 < K; k0 += BK) {
#pragma unroll
        for (int j = 0; j < LD; ++j) {
            int r, k;
            place(A_MN, j, r, k);
            As[k][r] = ra[j];
            place(B_MN, j, r, k);
            Bs[k][r] = rb[j];
        }
        __syncthreads();
        if (k0 + BK < K) fetch(k0 + BK);
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float a[TM], b[TM];
#pragma unroll
            for (int h = 0; h < TM; h += 4) {
                const float4 va = *reinterpret_cast<const float4*>(&As[k][16 * h + 4 * ty]);
                const float4 vb = *reinterpret_cast<const float4*>(&Bs[k][16 * h + 4 * tx]);
                a[h] = va.x; a[h + 1] = va.y; a[h + 2] = va.z; a[h + 3] = va.w;
                b[h] = vb.x; b[h + 1] = vb.y; b[h + 2] = vb.z; b[h + 3] = vb.w;
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
    }
    with_act(act, [&](auto kind) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + 16 * (i & ~3) + 4 * ty + (i & 3);
            if (m >= M) continue;
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int64_t n = n0 + 16 * (j & ~3) + 4 * tx + (j & 3);
                if (n >= N) continue;
                const float v = acc[i][j] + (bias ? __ldg(bias + n) : 0.f);
                if (z) store_elem(z + m * N + n, v);
                float o = act_value<kind(), sizeof(T) == 2>(v);
                if (residual) o += to_f32(__ldg(residual + m * N + n));
                store_elem(D + m * N + n, o);
            }
        }
    });
}

template <typename T, int TM, bool A_MN, bool B_MN>
cudaError_t launch(const GemmArgs& g) {
    constexpr int BM = 16 * TM;
    const int64_t tiles = ((g.M + BM - 1) / BM) * ((g.N + BM - 1) / BM);
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(gemm_kernel<T, TM, A_MN, B_MN>, dim3((unsigned)tiles), dim3(THREADS), 0, g.stream,
                      static_cast<const T*>(g.A), static_cast<const T*>(g.B), g.lda, g.ldb, g.M, g.N, g.K, g.bias,
                      static_cast<const T*>(g.residual), (int)g.act, static_cast<T*>(g.D), static_cast<T*>(g.z));
}

template <typename T, bool A_MN, bool B_MN>
cudaError_t pick(const GemmArgs& g) {
    DeviceInfo di;
    const cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    // 128 x 128 tiles reuse each loaded element twice as often; 64 x 64 ones where the large tiles
    // would leave SMs without one
    const int64_t big = ((g.M + 127) / 128) * ((g.N + 127) / 128);
    return big >= di.sm_count ? launch<T, 8, A_MN, B_MN>(g) : launch<T, 4, A_MN, B_MN>(g);
}

template <typename T>
cudaError_t pick_layout(const GemmArgs& g) {
    if (g.a_mn) return g.b_mn ? pick<T, true, true>(g) : cudaErrorInvalidValue;
    return g.b_mn ? pick<T, false, true>(g) : pick<T, false, false>(g);
}

}  // namespace

cudaError_t launch_gemm_generic(const GemmArgs& g) {
    return g.dt == BF16 ? pick_layout<__nv_bfloat16>(g) : pick_layout<float>(g);
}

}  // namespace mhc
