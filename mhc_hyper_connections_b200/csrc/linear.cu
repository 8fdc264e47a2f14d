// linear.cu -- the linear product with its epilogue, forward and backward: which kernel runs, and
// the backward's elementwise step.
//
//   forward    z = x W^T + bias          y = act(z) + residual
//   backward   dz = dy act'(z)           dx = dz W     dW = dz^T x     dbias = sum_t dz
//
// The elementwise step reads dy and z once, writes dz in the storage type (the operand both
// products read) and sums its columns from the fp32 values: each block walks a run of tokens, adds
// its eight rows of threads in shared memory and leaves one row of sums; a second kernel adds the
// blocks' rows in order.  It is bound by HBM (3 T N elements).  Without an activation dz is dy, and
// the step only sums columns.
#include <algorithm>

#include "activation.cuh"

namespace mhc {
namespace {

constexpr int DZ_COLS = 32;            // threads along a row
constexpr int DZ_ROWS = 8;             // rows a block takes at a time
constexpr int DZ_BLOCKS = 8 * 148;     // blocks wanted, eight per SM of a 148-SM device

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// runs of tokens of the elementwise step, each with a row of column sums
int64_t dz_runs(int64_t T, int N) {
    const int64_t col_blocks = ((int64_t)N + 255) / 256;
    const int64_t want = std::max<int64_t>(1, DZ_BLOCKS / col_blocks);
    return std::min(want, (T + DZ_ROWS - 1) / DZ_ROWS);
}

// A thread takes VEC columns and four tokens at a time (their loads are in flight together).  dz
// null: column sums only; part null: no sums.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(DZ_COLS* DZ_ROWS)
dz_kernel(const T* __restrict__ dy, const T* __restrict__ z, int64_t Tn, int N, int64_t run, T* __restrict__ dz,
          int64_t ld, float* __restrict__ part) {
    constexpr int U = 4;
    __shared__ float sm[DZ_ROWS][DZ_COLS * VEC + 1];
    const int tx = threadIdx.x % DZ_COLS, ty = threadIdx.x / DZ_COLS;
    const int64_t c = ((int64_t)blockIdx.x * DZ_COLS + tx) * VEC;
    const int64_t t0 = (int64_t)blockIdx.y * run, t1 = t0 + run < Tn ? t0 + run : Tn;
    float s[VEC] = {};
    if (c < N) {
        for (int64_t t = t0 + ty; t < t1; t += DZ_ROWS * U) {
            float g[U][VEC], zf[U][VEC];
            if constexpr (VEC > 1) {
                uint4 rg[U], rz[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t tu = t + u * DZ_ROWS;
                    rg[u] = rz[u] = make_uint4(0, 0, 0, 0);
                    if (tu < t1) {
                        rg[u] = ld_stream_v4(dy + tu * N + c);
                        if constexpr (ACT != ACT_NONE) rz[u] = ld_stream_v4(z + tu * N + c);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    Vec16<T>::unpack(rg[u], g[u]);
                    Vec16<T>::unpack(rz[u], zf[u]);
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t tu = t + u * DZ_ROWS;
                    g[u][0] = zf[u][0] = 0.f;
                    if (tu < t1) {
                        g[u][0] = to_f32(__ldg(dy + tu * N + c));
                        if constexpr (ACT != ACT_NONE) zf[u][0] = to_f32(__ldg(z + tu * N + c));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t tu = t + u * DZ_ROWS;
                if (tu >= t1) break;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    // rounded as a product whether or not dz is stored, so that the sums are the same bits
                    if constexpr (ACT != ACT_NONE)
                        g[u][e] = __fmul_rn(g[u][e], act_slope<ACT, sizeof(T) == 2>(zf[u][e]));
                    s[e] += g[u][e];
                }
                if (dz) {
                    if constexpr (VEC > 1) {
                        st_v4(dz + tu * ld + c, Vec16<T>::pack(g[u]));
                    } else {
                        store_elem(dz + tu * ld + c, g[u][0]);
                    }
                }
            }
        }
    }
    if (!part) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) sm[ty][tx * VEC + e] = s[e];
    __syncthreads();
    for (int i = threadIdx.x; i < DZ_COLS * VEC; i += DZ_COLS * DZ_ROWS) {
        const int64_t col = (int64_t)blockIdx.x * DZ_COLS * VEC + i;
        if (col >= N) continue;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < DZ_ROWS; ++r) v += sm[r][i];
        part[(int64_t)blockIdx.y * N + col] = v;
    }
}

// out[c] = sum over P rows of part, in a fixed order
__global__ void __launch_bounds__(256)
sum_rows_kernel(const float* __restrict__ part, int64_t P, int N, float* __restrict__ out) {
    __shared__ float sm[8][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < N)
        for (int64_t p = warp; p < P; p += 8) s += part[p * N + c];
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < N) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sm[k][lane];
        out[c] = s;
    }
}

template <typename T, int VEC>
void start_dz(const LinearArgs& a, void* dz, int64_t ld, int64_t run, int64_t rows, float* sums) {
    const int cols = DZ_COLS * VEC;
    const dim3 grid((unsigned)((a.N + (int64_t)cols - 1) / cols), (unsigned)rows);
    auto go = [&](auto kern) {
        kern<<<grid, DZ_COLS * DZ_ROWS, 0, a.stream>>>(static_cast<const T*>(a.dy), static_cast<const T*>(a.z), a.T,
                                                       a.N, run, static_cast<T*>(dz), ld, sums);
    };
    switch (a.act) {
        case ACT_RELU: go(dz_kernel<T, VEC, ACT_RELU>); break;
        case ACT_GELU: go(dz_kernel<T, VEC, ACT_GELU>); break;
        case ACT_GELU_TANH: go(dz_kernel<T, VEC, ACT_GELU_TANH>); break;
        case ACT_SILU: go(dz_kernel<T, VEC, ACT_SILU>); break;
        default: go(dz_kernel<T, VEC, ACT_NONE>); break;
    }
}

template <typename T>
cudaError_t launch_dz(const LinearArgs& a, void* dz, int64_t ld, float* part) {
    constexpr int V = Vec16<T>::VEC;
    const int64_t runs = dz_runs(a.T, a.N);
    const int64_t run = ((a.T + runs - 1) / runs + DZ_ROWS - 1) / DZ_ROWS * DZ_ROWS;
    const int64_t rows = (a.T + run - 1) / run;      // runs that hold tokens
    float* sums = a.dbias ? (rows == 1 ? a.dbias : part) : nullptr;
    if (a.N % V == 0 && ld % V == 0 && (uintptr_t)a.dy % 16 == 0 && (uintptr_t)a.z % 16 == 0)
        start_dz<T, V>(a, dz, ld, run, rows, sums);
    else
        start_dz<T, 1>(a, dz, ld, run, rows, sums);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && a.dbias && rows > 1)
        e = launch_pdl(sum_rows_kernel, dim3((unsigned)((a.N + (int64_t)31) / 32)), dim3(256), 0, a.stream, part,
                       rows, a.N, a.dbias);
    return e;
}

cudaError_t product(const GemmArgs& g) { return gemm_tc_ok(g) ? launch_gemm_tc(g) : launch_gemm_generic(g); }

// regions of the backward's workspace, in bytes
struct BackwardLayout {
    size_t dz, part, total;
    int64_t ld;                        // elements per row of dz: 16-byte rows
};

BackwardLayout backward_regions(int64_t T, int K, int N, DType dt) {
    BackwardLayout L{};
    const size_t es = dt == BF16 ? 2 : 4;
    const int64_t v = 16 / es;
    (void)K;
    L.ld = ((int64_t)N + v - 1) / v * v;
    L.dz = 0;
    L.part = round256((size_t)T * L.ld * es);
    L.total = L.part + round256((size_t)dz_runs(T, N) * N * 4);
    return L;
}

}  // namespace

size_t linear_workspace(int64_t T, int K, int N, DType dt) {
    (void)T; (void)K; (void)N; (void)dt;
    return 0;
}

size_t linear_backward_workspace(int64_t T, int K, int N, DType dt) { return backward_regions(T, K, N, dt).total; }

cudaError_t launch_linear(const LinearArgs& a) {
    GemmArgs g{};
    g.A = a.x; g.lda = a.K; g.B = a.W; g.ldb = a.K;
    g.M = a.T; g.N = a.N; g.K = a.K;
    g.bias = a.bias; g.residual = a.residual; g.act = a.act; g.D = a.y; g.z = a.z;
    g.dt = a.dt; g.stream = a.stream;
    return product(g);
}

cudaError_t launch_linear_backward(const LinearArgs& a) {
    const BackwardLayout L = backward_regions(a.T, a.K, a.N, a.dt);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    const bool products = a.dx || a.dW;
    // dz is dy itself without an activation
    void* dz = a.act != ACT_NONE && products ? ws + L.dz : nullptr;
    cudaError_t e = cudaSuccess;
    if (dz || a.dbias) {
        float* part = reinterpret_cast<float*>(ws + L.part);
        e = a.dt == BF16 ? launch_dz<__nv_bfloat16>(a, dz, L.ld, part) : launch_dz<float>(a, dz, L.ld, part);
    }
    GemmArgs g{};
    g.A = dz ? dz : a.dy;
    g.lda = dz ? L.ld : a.N;
    g.dt = a.dt; g.stream = a.stream; g.act = ACT_NONE;
    g.b_mn = true;
    if (e == cudaSuccess && a.dx) {          // dx[t][k] = sum_n dz[t][n] W[n][k]
        g.B = a.W; g.ldb = a.K;
        g.M = a.T; g.N = a.K; g.K = a.N;
        g.D = a.dx;
        e = product(g);
    }
    if (e == cudaSuccess && a.dW) {          // dW[n][k] = sum_t dz[t][n] x[t][k]
        g.a_mn = true;
        g.B = a.x; g.ldb = a.K;
        g.M = a.N; g.N = a.K; g.K = a.T;
        g.D = a.dW;
        e = product(g);
    }
    return e;
}

}  // namespace mhc
