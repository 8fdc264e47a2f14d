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
constexpr int DZ_BLOCKS = 16 * 148;    // blocks wanted, sixteen per SM of a 148-SM device

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// Runs of tokens of the elementwise step, each with a row of column sums: two tokens per thread at least
// (one: T = 4096, N = 1024 11.4 us against 7.9, T = 16384, N = 256 15.5 against 11.2; four: no gain but
// without an activation, T = 1000, N = 4096 9.2 against 7.4)
int64_t dz_runs(int64_t T, int N) {
    const int64_t col_blocks = ((int64_t)N + 255) / 256;
    const int64_t want = std::max<int64_t>(1, DZ_BLOCKS / col_blocks);
    return std::min(want, (T + 2 * DZ_ROWS - 1) / (2 * DZ_ROWS));
}

// Loads of VEC columns at (t, c): 16-byte rows, or bf16 rows wherever they lie (SHIFT)
template <typename T, int VEC, bool SHIFT>
__device__ __forceinline__ void dz_load(const T* __restrict__ p, int64_t t, int64_t c, int64_t Tn, int N, float* f) {
    if constexpr (SHIFT) {
        Vec16<T>::unpack(ld_shifted_v4(p, t * N + c, Tn * N), f);
    } else if constexpr (VEC > 1) {
        Vec16<T>::unpack(ld_stream_v4(p + t * N + c), f);
    } else {
        f[0] = to_f32(__ldg(p + t * N + c));
    }
}

// A thread takes VEC columns of a token at a time: its two loads, and many blocks per SM in place of
// more of them (T = N = 16384 with GELU: four tokens at a time took 510 us, one 300, 5.4 TB/s; the
// sums alone, without dz, 216).  dz null: column sums only; part null: no sums.
template <typename T, int VEC, int ACT, bool SHIFT>
__global__ void __launch_bounds__(DZ_COLS* DZ_ROWS)
dz_kernel(const T* __restrict__ dy, const T* __restrict__ z, int64_t Tn, int N, int64_t run, T* __restrict__ dz,
          int64_t ld, float* __restrict__ part) {
    __shared__ float sm[DZ_ROWS][DZ_COLS * VEC + 1];
    pdl_launch_next();
    pdl_wait();
    const int tx = threadIdx.x % DZ_COLS, ty = threadIdx.x / DZ_COLS;
    const int64_t c = ((int64_t)blockIdx.x * DZ_COLS + tx) * VEC;
    const int64_t t0 = (int64_t)blockIdx.y * run, t1 = t0 + run < Tn ? t0 + run : Tn;
    float s[VEC] = {};
    if (c < N) {
        for (int64_t t = t0 + ty; t < t1; t += DZ_ROWS) {
            float g[VEC], zf[VEC];
            dz_load<T, VEC, SHIFT>(dy, t, c, Tn, N, g);
            if constexpr (ACT != ACT_NONE) dz_load<T, VEC, SHIFT>(z, t, c, Tn, N, zf);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // rounded as a product whether or not dz is stored, so that the sums are the same bits
                if constexpr (ACT != ACT_NONE) g[e] = __fmul_rn(g[e], act_slope<ACT, sizeof(T) == 2>(zf[e]));
                s[e] += g[e];
            }
            if (dz) {
                if constexpr (VEC > 1) {
                    st_v4(dz + t * ld + c, Vec16<T>::pack(g));      // may fill up the row's padding
                } else {
                    store_elem(dz + t * ld + c, g[0]);
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

// out[c] = sum over P rows of part, in a fixed order: 32 columns per block, a 32nd of the rows per warp,
// eight of them in flight
__global__ void __launch_bounds__(1024)
sum_rows_kernel(const float* __restrict__ part, int64_t P, int N, float* __restrict__ out) {
    constexpr int U = 8;
    __shared__ float sm[32][33];
    pdl_launch_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < N)
        for (int64_t p = warp; p < P; p += 32 * U) {
            float v[U];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = p + 32 * j < P ? __ldcg(part + (p + 32 * j) * N + c) : 0.f;
#pragma unroll
            for (int j = 0; j < U; ++j) s += v[j];
        }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < N) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += sm[k][lane];
        out[c] = s;
    }
}

template <typename T, int VEC, bool SHIFT>
cudaError_t start_dz(const LinearArgs& a, void* dz, int64_t ld, int64_t run, int64_t rows, float* sums) {
    const int cols = DZ_COLS * VEC;
    const dim3 grid((unsigned)((a.N + (int64_t)cols - 1) / cols), (unsigned)rows);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) {
        e = launch_pdl(kern, grid, dim3(DZ_COLS * DZ_ROWS), 0, a.stream, static_cast<const T*>(a.dy),
                       static_cast<const T*>(a.z), a.T, a.N, run, static_cast<T*>(dz), ld, sums);
    };
    switch (a.act) {
        case ACT_RELU: go(dz_kernel<T, VEC, ACT_RELU, SHIFT>); break;
        case ACT_GELU: go(dz_kernel<T, VEC, ACT_GELU, SHIFT>); break;
        case ACT_GELU_TANH: go(dz_kernel<T, VEC, ACT_GELU_TANH, SHIFT>); break;
        case ACT_SILU: go(dz_kernel<T, VEC, ACT_SILU, SHIFT>); break;
        default: go(dz_kernel<T, VEC, ACT_NONE, SHIFT>); break;
    }
    return e;
}

template <typename T>
cudaError_t launch_dz(const LinearArgs& a, void* dz, int64_t ld, float* part) {
    constexpr int V = Vec16<T>::VEC;
    const int64_t runs = dz_runs(a.T, a.N);
    const int64_t run = ((a.T + runs - 1) / runs + DZ_ROWS - 1) / DZ_ROWS * DZ_ROWS;
    const int64_t rows = (a.T + run - 1) / run;      // runs that hold tokens
    float* sums = a.dbias ? (rows == 1 ? a.dbias : part) : nullptr;
    cudaError_t e;
    if (a.N % V == 0 && (uintptr_t)a.dy % 16 == 0 && (uintptr_t)a.z % 16 == 0)
        e = start_dz<T, V, false>(a, dz, ld, run, rows, sums);
    else if constexpr (sizeof(T) == 2)
        e = start_dz<T, V, true>(a, dz, ld, run, rows, sums);
    else
        e = start_dz<T, 1, false>(a, dz, ld, run, rows, sums);
    if (e == cudaSuccess && a.dbias && rows > 1)
        e = launch_pdl(sum_rows_kernel, dim3((unsigned)((a.N + (int64_t)31) / 32)), dim3(1024), 0, a.stream, part,
                       rows, a.N, a.dbias);
    return e;
}

// A copy of bf16 rows with each row on a 16-byte boundary, for the tensor-core products of operands
// whose row length is not a multiple of 16 bytes.  Even 8 tokens gain by it (4095 -> 4096: 19 us, 45
// with gemm_thin on the rows as they lie).
struct PadJob {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    int64_t rows, ld;                  // ld: elements per row of dst, the row length rounded up to 8
    int cols;
};

__global__ void __launch_bounds__(256) pad_rows_kernel(const __grid_constant__ PadJob a, const __grid_constant__ PadJob b) {
    const PadJob& j = blockIdx.y ? b : a;
    pdl_launch_next();
    pdl_wait();
    const int64_t per = j.ld / 8, total = j.rows * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per, c = (i - row * per) * 8;
        st_v4(j.dst + row * j.ld + c, ld_shifted_v4(j.src, row * j.cols + c, j.rows * j.cols));
    }
}

cudaError_t pad_rows(const PadJob& a, const PadJob& b, cudaStream_t s) {
    const int64_t n = std::max(a.rows * a.ld, b.rows * b.ld) / 8;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 8 * 148);
    return launch_pdl(pad_rows_kernel, dim3(blocks, b.rows ? 2 : 1), dim3(256), 0, s, a, b);
}

int64_t padded(int64_t cols) { return (cols + 7) / 8 * 8; }

cudaError_t product(const GemmArgs& g) {
    if (gemm_tc_ok(g)) return launch_gemm_tc(g);
    return gemm_thin_ok(g) ? launch_gemm_thin(g) : launch_gemm_generic(g);
}

// The bf16 parts h + m + l of fp32 rows times 2^16, in three planes of rows on 16-byte boundaries.  The
// scale makes the parts exact for small values too: fp32's last place is never below 2^-149, bf16's smallest
// number is 2^-133 (without it values below 2^-110 lost bits: a relative error of 2.7e-5 at 1e-36).  A value
// that is not finite, or whose h would not be (from 2^112 on), has no such parts: its block sets its word of
// `odd`, and the CUDA-core kernel forms the product instead.
struct SplitJob {
    const float* src;
    __nv_bfloat16* dst;
    int* odd;                          // SPLIT_BLOCKS words
    int* clear;                        // a word to set to 0: F32Planes::over of a product of these rows
    int64_t rows, ld;                  // ld: elements per row of a plane, a multiple of 8
    int cols;
};
constexpr int SPLIT_BLOCKS = 4 * 148;

__global__ void __launch_bounds__(256) split_rows_kernel(const __grid_constant__ SplitJob a, const __grid_constant__ SplitJob b) {
    const SplitJob& j = blockIdx.y ? b : a;
    pdl_launch_next();
    pdl_wait();
    const int64_t per = j.ld / 8, total = j.rows * per, plane = j.rows * j.ld;
    const bool vec = j.cols % 4 == 0 && (uintptr_t)j.src % 16 == 0;
    int odd = 0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        const int c = (int)(i - row * per) * 8;
        const float* s = j.src + row * j.cols + c;
        float f[8];
        if (vec && c + 8 <= j.cols) {
            Vec16<float>::unpack(ld_stream_v4(s), f);
            Vec16<float>::unpack(ld_stream_v4(s + 4), f + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = c + e < j.cols ? __ldg(s + e) : 0.f;
        }
        float h[8], m[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] *= 65536.0f;
            h[e] = __bfloat162float(__float2bfloat16_rn(f[e]));
            odd |= !(fabsf(h[e]) <= 3.4028234e38f);
            f[e] -= h[e];                              // exact, as is the next difference
            m[e] = __bfloat162float(__float2bfloat16_rn(f[e]));
            f[e] -= m[e];
        }
        __nv_bfloat16* d = j.dst + row * j.ld + c;
        st_v4(d, Vec16<__nv_bfloat16>::pack(h));
        st_v4(d + plane, Vec16<__nv_bfloat16>::pack(m));
        st_v4(d + 2 * plane, Vec16<__nv_bfloat16>::pack(f));
    }
    odd = __syncthreads_or(odd);
    if (threadIdx.x == 0) {
        j.odd[blockIdx.x] = odd;
        if (blockIdx.x == 0) *j.clear = 0;
    }
}

// every block writes its word, so all SPLIT_BLOCKS of them are set afterwards
cudaError_t split_rows(const SplitJob& a, const SplitJob& b, cudaStream_t s) {
    return launch_pdl(split_rows_kernel, dim3(SPLIT_BLOCKS, b.rows ? 2 : 1), dim3(256), 0, s, a, b);
}

// fp32 products that go to the tensor cores: those whose time on CUDA cores exceeds that of the parts and their
// products, by these models in us (measured, operands in L2).  The parts: 10 bytes per element at 7.5 TB/s, at
// 2.9 past 64 MB, and 8.5 us for their launch and the one that forms values without parts, 9 more in a backward
// call, which decides for its two products together.  Up to 16 tokens CUDA cores are faster throughout.  Parts
// and CUDA cores, forward: T = 24, 4096 -> 1024 28 and 42, 1024 -> 4096 28 and 22; T = 64, 4096 -> 4096 94 and 77;
// T = 65 94 and 149; T = 512, 512 -> 512 17 and 14; backward: T = 24, 1024 -> 4096 50 and 88, 4096 -> 1024 49 and
// 41.  Of 260 calls (gemm_generic_time's shapes) three take the slower form by more than a tenth, all backward:
// T = 64, 4096 -> 1024 58 for 50; 512 -> 2048, T = 48 40 for 35, T = 24 38 for 34.
bool parts_pay(int64_t T, int K, int N, bool backward) {
    if (T <= 16 || T >= ((int64_t)1 << 31) - 1024) return false;
    const double bytes = 10.0 * ((double)T * K + (double)N * K + (backward ? (double)T * N : 0.0));
    const double split = bytes / 7.5e6 + std::max(0.0, bytes - 64e6) / 4.6e6 + 8.5;
    if (!backward) return split + gemm_f32_time(T, N, K, false) < gemm_generic_time(T, N, K);
    return split + 9.0 + gemm_f32_time(T, K, N, false) + gemm_f32_time(N, K, T, true) <
           gemm_generic_time(T, K, N) + gemm_generic_time(N, K, T);
}

// Regions of the workspaces, in bytes.  bf16 rows of K elements that are not a multiple of 16 bytes
// are copied to padded ones (x and W); fp32 operands of the tensor cores are held in parts.
struct Regions {
    size_t x, W, dz, part, odd, dzp, tiles, total;
    int64_t ldk, ldn;                  // elements per row of the copies of x and W, and of dz
    bool pad, parts;
};

Regions regions(int64_t T, int K, int N, DType dt, bool backward) {
    Regions L{};
    const size_t es = dt == BF16 ? 2 : 4;
    L.pad = dt == BF16 && K % 8 != 0;
    L.parts = dt == F32 && parts_pay(T, K, N, backward);
    L.ldk = L.pad || L.parts ? padded(K) : K;
    L.ldn = dt == BF16 || L.parts ? padded(N) : N;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t at = off; off += round256(bytes); return at; };
    if (L.pad || L.parts) {
        L.x = take((size_t)T * L.ldk * (L.parts ? 6 : 2));
        L.W = take((size_t)N * L.ldk * (L.parts ? 6 : 2));
    }
    if (L.parts) L.odd = take((size_t)(3 * SPLIT_BLOCKS + 2) * 4);
    if (backward) {
        L.dz = take((size_t)T * (dt == BF16 ? L.ldn : N) * es);
        L.part = take((size_t)dz_runs(T, N) * N * 4);
        if (L.parts) L.dzp = take((size_t)T * L.ldn * 6);
    }
    // parts of tiles that the tensor-core kernels share, of one product at a time
    auto shared = [&](int64_t M, int64_t n, int64_t k, bool a_mn) {
        return dt == BF16 ? gemm_tc_part_bytes(M, n, k, a_mn) : L.parts ? gemm_f32_part_bytes(M, n, k, a_mn) : 0;
    };
    L.tiles = take(backward ? std::max(shared(T, K, N, false), shared(N, K, T, true)) : shared(T, N, K, false));
    L.total = off;
    return L;
}

}  // namespace

size_t linear_workspace(int64_t T, int K, int N, DType dt) { return regions(T, K, N, dt, false).total; }

size_t linear_backward_workspace(int64_t T, int K, int N, DType dt) { return regions(T, K, N, dt, true).total; }

cudaError_t launch_linear(const LinearArgs& a) {
    const Regions L = regions(a.T, a.K, a.N, a.dt, false);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    GemmArgs g{};
    g.A = a.x; g.B = a.W;
    g.lda = g.ldb = a.K;
    g.M = a.T; g.N = a.N; g.K = a.K;
    g.bias = a.bias; g.residual = a.residual; g.act = a.act; g.D = a.y; g.z = a.z;
    g.part = reinterpret_cast<float*>(ws + L.tiles);
    g.dt = a.dt; g.stream = a.stream;
    __nv_bfloat16* xc = reinterpret_cast<__nv_bfloat16*>(ws + L.x);
    __nv_bfloat16* wc = reinterpret_cast<__nv_bfloat16*>(ws + L.W);
    if (L.parts) {
        int* over = reinterpret_cast<int*>(ws + L.odd);      // and the words of x and W after it
        int* odd = over + 1;
        const SplitJob x{static_cast<const float*>(a.x), xc, odd, over, a.T, L.ldk, a.K};
        const SplitJob w{static_cast<const float*>(a.W), wc, odd + SPLIT_BLOCKS, over, a.N, L.ldk, a.K};
        cudaError_t e = split_rows(x, w, a.stream);
        if (e == cudaSuccess)
            e = launch_gemm_f32(g, F32Planes{xc, wc, L.ldk, L.ldk, a.T * L.ldk, a.N * L.ldk, over});
        return e == cudaSuccess ? launch_gemm_generic(g, over, 1 + 2 * SPLIT_BLOCKS) : e;
    }
    if (L.pad) {
        const PadJob x{static_cast<const __nv_bfloat16*>(a.x), xc, a.T, L.ldk, a.K};
        const PadJob w{static_cast<const __nv_bfloat16*>(a.W), wc, a.N, L.ldk, a.K};
        const cudaError_t e = pad_rows(x, w, a.stream);
        if (e != cudaSuccess) return e;
        g.A = xc; g.B = wc;
        g.lda = g.ldb = L.ldk;
    }
    return product(g);
}

cudaError_t launch_linear_backward(const LinearArgs& a) {
    const Regions L = regions(a.T, a.K, a.N, a.dt, true);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    const bool products = a.dx || a.dW;
    // dz is dy itself without an activation, unless the tensor cores need its rows on 16-byte boundaries
    const bool copy = a.act != ACT_NONE || (a.dt == BF16 && (a.N % 8 != 0 || (uintptr_t)a.dy % 16 != 0));
    void* dz = copy && products ? ws + L.dz : nullptr;
    const int64_t ldz = dz && a.dt == BF16 ? L.ldn : a.N;
    cudaError_t e = cudaSuccess;
    if (dz || a.dbias) {
        float* part = reinterpret_cast<float*>(ws + L.part);
        e = a.dt == BF16 ? launch_dz<__nv_bfloat16>(a, dz, ldz, part) : launch_dz<float>(a, dz, ldz, part);
    }
    if (e != cudaSuccess || !products) return e;
    __nv_bfloat16* xc = reinterpret_cast<__nv_bfloat16*>(ws + L.x);
    __nv_bfloat16* wc = reinterpret_cast<__nv_bfloat16*>(ws + L.W);
    __nv_bfloat16* zc = reinterpret_cast<__nv_bfloat16*>(ws + L.dzp);
    // the words of dx's product: its over, W's, dz's; and of dW's: dz's, x's, its over
    int* const words = reinterpret_cast<int*>(ws + L.odd);
    int *const odd = words + 1, *const over_dW = odd + 3 * SPLIT_BLOCKS;
    if (L.parts) {
        int* const over_z = a.dx ? words : over_dW;      // also cleared with the other operand's rows
        const SplitJob jw{static_cast<const float*>(a.W), wc, odd, words, a.N, L.ldk, a.K};
        const SplitJob jz{static_cast<const float*>(dz ? dz : a.dy), zc, odd + SPLIT_BLOCKS, over_z, a.T, L.ldn, a.N};
        const SplitJob jx{static_cast<const float*>(a.x), xc, odd + 2 * SPLIT_BLOCKS, over_dW, a.T, L.ldk, a.K};
        e = split_rows(jz, a.dx ? jw : jx, a.stream);
        if (e == cudaSuccess && a.dx && a.dW) e = split_rows(jx, SplitJob{}, a.stream);
    } else if (L.pad) {
        const PadJob jw{static_cast<const __nv_bfloat16*>(a.W), wc, a.N, L.ldk, a.K};
        const PadJob jx{static_cast<const __nv_bfloat16*>(a.x), xc, a.T, L.ldk, a.K};
        e = pad_rows(a.dx ? jw : jx, a.dx && a.dW ? jx : PadJob{}, a.stream);
    }
    if (e != cudaSuccess) return e;
    GemmArgs g{};
    g.A = dz ? dz : a.dy;
    g.lda = ldz;
    g.part = reinterpret_cast<float*>(ws + L.tiles);
    g.dt = a.dt; g.stream = a.stream; g.act = ACT_NONE;
    g.b_mn = true;
    g.ldb = L.pad ? L.ldk : a.K;
    // one of the two products, with the words of its operands
    auto run = [&](const void* B, const __nv_bfloat16* parts, int64_t b_rows, const int* first, int* over) {
        g.B = L.pad ? parts : B;
        if (!L.parts) return product(g);
        cudaError_t r = launch_gemm_f32(g, F32Planes{zc, parts, L.ldn, L.ldk, a.T * L.ldn, b_rows * L.ldk, over});
        if (r == cudaSuccess) r = launch_gemm_generic(g, first, 1 + 2 * SPLIT_BLOCKS);
        return r;
    };
    if (a.dx) {                              // dx[t][k] = sum_n dz[t][n] W[n][k]
        g.M = a.T; g.N = a.K; g.K = a.N;
        g.D = a.dx;
        e = run(a.W, wc, a.N, words, words);
    }
    if (e == cudaSuccess && a.dW) {          // dW[n][k] = sum_t dz[t][n] x[t][k]
        g.a_mn = true;
        g.M = a.N; g.N = a.K; g.K = a.T;
        g.D = a.dW;
        e = run(a.x, xc, a.T, odd + SPLIT_BLOCKS, over_dW);
    }
    return e;
}

}  // namespace mhc
