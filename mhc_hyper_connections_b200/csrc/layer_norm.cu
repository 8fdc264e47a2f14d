// layer_norm.cu -- layer norm over the channels of a token, forward and backward.
//
//   forward    mean = sum_c x_c / d     var = sum_c (x_c - mean)^2 / d     rstd = 1 / sqrt(var + eps)
//              y_c  = (x_c - mean) rstd w_c + b_c
//   backward   xh_c = (x_c - mean) rstd     g_c = dy_c w_c
//              dx_c = rstd (g_c - sum(g) / d - xh_c sum(g xh) / d)
//              dw_c = sum_t dy_c xh_c       db_c = sum_t dy_c
//
// Both are bound by HBM: 2 T d elements forward, 3 T d backward, a few operations each.  So each
// row is read once and kept in registers, packed as it was stored, between its reduction and its
// output; sums are fp32, and the variance is summed around the mean (a second walk over the
// registers), which a mean far from zero does not spoil.
//
// A row belongs to one warp (WARP, rows of up to 4 vectors per lane) or to one thread block.  A
// thread owns the same NV vectors of VEC columns in every row it sees, so w and b are loaded once
// and the backward's column sums stay in registers until the thread's last row.  A group takes R
// rows at a time: their loads are in flight together and they share each reduction's barrier.
// Column sums are added up in a fixed order: over a group's rows, over a block's warps in shared
// memory, and over the blocks by a second kernel that reads one fp32 row pair per block.
#include "common.cuh"
#include "launch.cuh"

namespace mhc {
namespace {

// blocks that write column-sum rows for the second kernel: three per SM of a 148-SM device
constexpr int BWD_BLOCKS = 444;
constexpr int WARPS = 8;               // warps per block where a row belongs to a warp

// VEC elements as they lie in memory: 16 bytes, or one element where rows are not 16-byte aligned
template <typename T, int VEC> struct Pack;
template <typename T> struct Pack<T, 1> {
    using raw = T;
    __device__ __forceinline__ static raw zero() { return T(0.f); }
    __device__ __forceinline__ static raw load(const T* p) { return __ldg(p); }
    __device__ __forceinline__ static void unpack(raw v, float* f) { f[0] = to_f32(v); }
    __device__ __forceinline__ static void store(T* p, const float* f) { store_elem(p, f[0]); }
};
template <typename T, int VEC> struct Pack {
    using raw = uint4;
    static_assert(VEC == Vec16<T>::VEC, "a pack is 16 bytes");
    __device__ __forceinline__ static raw zero() { return make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ static raw load(const T* p) { return ld_stream_v4(p); }
    __device__ __forceinline__ static void unpack(raw v, float* f) { Vec16<T>::unpack(v, f); }
    __device__ __forceinline__ static void store(T* p, const float* f) { st_v4(p, Vec16<T>::pack(f)); }
};

// Sum R values over the group (a warp, or the block); every thread gets the sums.  The block form
// alternates between two buffers, so one barrier per call is enough: a buffer is written again
// only after every thread has passed the barrier of the call in between.
template <int R, bool WARP>
__device__ __forceinline__ void group_sum(float (&v)[R], float* buf, int& phase) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    if constexpr (!WARP) {
        float* b = buf + phase * 32 * R;
        phase ^= 1;
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) b[warp * R + r] = v[r];
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = 0.f;
        for (int w = 0; w < nw; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += b[w * R + r];
    }
}

// threads of a block: a warp per row uses WARPS warps; a block per row as many threads as the row
// needs, up to 1024 with one vector each (few rows) and 512 with more, which the registers allow
template <int NV, bool WARP> constexpr int MAX_THREADS = WARP ? 32 * WARPS : (NV == 1 ? 1024 : 512);

template <typename T, int VEC, int NV, int R, bool WARP>
__global__ void __launch_bounds__(MAX_THREADS<NV, WARP>)
ln_fwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                              int64_t Tn, int d, float eps, T* __restrict__ y, float* __restrict__ mean_out,
                              float* __restrict__ rstd_out) {
    using P = Pack<T, VEC>;
    __shared__ float buf[WARP ? 1 : 64 * R];
    int phase = 0;
    pdl_launch_next();
    pdl_wait();
    const int nthr = WARP ? 32 : blockDim.x;
    const int idx = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t groups = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t gid = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const float inv_d = 1.0f / (float)d;

    float wv[NV][VEC], bv[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nthr + idx) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wv[v][e] = w && c < d ? __ldg(w + c + e) : 1.f;
            bv[v][e] = b && c < d ? __ldg(b + c + e) : 0.f;
        }
    }

    for (int64_t row0 = gid; row0 < Tn; row0 += groups * R) {
        typename P::raw raw[R][NV];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * groups;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * nthr + idx) * VEC;
                raw[r][v] = row < Tn && c < d ? P::load(x + row * d + c) : P::zero();
            }
        }
        float s[R], mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[VEC];
                P::unpack(raw[r][v], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[r] += f[e];
            }
        }
        group_sum<R, WARP>(s, buf, phase);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = s[r] * inv_d;
            s[r] = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float f[VEC];
                P::unpack(raw[r][v], f);
                const bool in = (v * nthr + idx) * VEC < d;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float c = f[e] - mean[r];
                    if (in) s[r] = fmaf(c, c, s[r]);
                }
            }
        }
        group_sum<R, WARP>(s, buf, phase);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * groups;
            if (row >= Tn) break;
            const float rstd = 1.0f / sqrtf(fmaf(s[r], inv_d, eps));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * nthr + idx) * VEC;
                float f[VEC];
                P::unpack(raw[r][v], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = fmaf((f[e] - mean[r]) * rstd, wv[v][e], bv[v][e]);
                if (c < d) P::store(y + row * d + c, f);
            }
            if (idx == 0 && mean_out) {
                mean_out[row] = mean[r];
                rstd_out[row] = rstd;
            }
        }
    }
}

// Rows too long for the registers of one block: the block walks the row three times.
template <typename T>
__global__ void __launch_bounds__(1024)
ln_fwd_long_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                   const float* __restrict__ b, int64_t Tn, int d, float eps, T* __restrict__ y,
                                   float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float buf[64];
    int phase = 0;
    pdl_launch_next();
    pdl_wait();
    const float inv_d = 1.0f / (float)d;
    for (int64_t row = blockIdx.x; row < Tn; row += gridDim.x) {
        const T* xr = x + row * d;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < d; c += blockDim.x) s[0] += to_f32(__ldg(xr + c));
        group_sum<1, false>(s, buf, phase);
        const float mean = s[0] * inv_d;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float v = to_f32(__ldg(xr + c)) - mean;
            s[0] = fmaf(v, v, s[0]);
        }
        group_sum<1, false>(s, buf, phase);
        const float rstd = 1.0f / sqrtf(fmaf(s[0], inv_d, eps));
        for (int c = threadIdx.x; c < d; c += blockDim.x)
            store_elem(y + row * d + c, fmaf((to_f32(__ldg(xr + c)) - mean) * rstd, w ? __ldg(w + c) : 1.f,
                                             b ? __ldg(b + c) : 0.f));
        if (threadIdx.x == 0 && mean_out) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
    }
}

// part: one [2][d] row pair (dw, db) per block
template <typename T, int VEC, int NV, int R, bool WARP>
__global__ void __launch_bounds__(MAX_THREADS<NV, WARP>)
ln_bwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
                              const float* __restrict__ rstd, const T* __restrict__ dy, int64_t Tn, int d,
                              T* __restrict__ dx, float* __restrict__ part) {
    using P = Pack<T, VEC>;
    __shared__ float buf[WARP ? 1 : 64 * 2 * R];
    extern __shared__ float cols[];        // WARP: [2][d] column sums of the block
    int phase = 0;
    pdl_launch_next();
    pdl_wait();
    const int nthr = WARP ? 32 : blockDim.x;
    const int idx = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t groups = WARP ? (int64_t)gridDim.x * (blockDim.x >> 5) : gridDim.x;
    const int64_t gid = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    const float inv_d = 1.0f / (float)d;

    float wv[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nthr + idx) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wv[v][e] = w && c < d ? __ldg(w + c + e) : 1.f;
            dw[v][e] = db[v][e] = 0.f;
        }
    }

    for (int64_t row0 = gid; row0 < Tn; row0 += groups * R) {
        typename P::raw xr[R][NV], gr[R][NV];
        float mu[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * groups;
            mu[r] = row < Tn ? __ldg(mean + row) : 0.f;
            rs[r] = row < Tn ? __ldg(rstd + row) : 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * nthr + idx) * VEC;
                const bool in = row < Tn && c < d;
                xr[r][v] = in ? P::load(x + row * d + c) : P::zero();
                gr[r][v] = in ? P::load(dy + row * d + c) : P::zero();
            }
        }
        // sums[r] = sum g, sums[R + r] = sum g xh; columns past d and rows past Tn have dy = 0
        float sums[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sums[r] = sums[R + r] = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float xf[VEC], gf[VEC];
                P::unpack(xr[r][v], xf);
                P::unpack(gr[r][v], gf);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (xf[e] - mu[r]) * rs[r], g = gf[e] * wv[v][e];
                    dw[v][e] = fmaf(gf[e], xh, dw[v][e]);
                    db[v][e] += gf[e];
                    sums[r] += g;
                    sums[R + r] = fmaf(g, xh, sums[R + r]);
                }
            }
        }
        if (!dx) continue;
        group_sum<2 * R, WARP>(sums, buf, phase);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * groups;
            if (row >= Tn) break;
            const float a = sums[r] * inv_d, k = sums[R + r] * inv_d;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * nthr + idx) * VEC;
                float xf[VEC], gf[VEC];
                P::unpack(xr[r][v], xf);
                P::unpack(gr[r][v], gf);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (xf[e] - mu[r]) * rs[r];
                    gf[e] = rs[r] * (fmaf(gf[e], wv[v][e], -a) - xh * k);
                }
                if (c < d) P::store(dx + row * d + c, gf);
            }
        }
    }

    if (!part) return;
    float* pw = part + (int64_t)blockIdx.x * 2 * d;
    if constexpr (WARP) {
        // the block's warps add their sums in turn
        const int nw = blockDim.x >> 5;
        for (int k = 0; k < nw; ++k) {
            if ((int)(threadIdx.x >> 5) == k) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * nthr + idx) * VEC;
                    if (c < d)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            cols[c + e] = (k ? cols[c + e] : 0.f) + dw[v][e];
                            cols[d + c + e] = (k ? cols[d + c + e] : 0.f) + db[v][e];
                        }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) pw[c] = cols[c];
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nthr + idx) * VEC;
            if (c < d)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    pw[c + e] = dw[v][e];
                    pw[d + c + e] = db[v][e];
                }
        }
    }
}

// Rows too long for registers: the block's column sums live in its row pair of `part`, each
// entry read and written by one thread only.
template <typename T>
__global__ void __launch_bounds__(1024)
ln_bwd_long_kernel(const T* __restrict__ x, const float* __restrict__ w,
                                   const float* __restrict__ mean, const float* __restrict__ rstd,
                                   const T* __restrict__ dy, int64_t Tn, int d, T* __restrict__ dx, float* part) {
    __shared__ float buf[64 * 2];
    int phase = 0;
    pdl_launch_next();
    pdl_wait();
    const float inv_d = 1.0f / (float)d;
    float* pw = part ? part + (int64_t)blockIdx.x * 2 * d : nullptr;
    for (int64_t row = blockIdx.x; row < Tn; row += gridDim.x) {
        const T* xr = x + row * d;
        const T* gr = dy + row * d;
        const float mu = __ldg(mean + row), rs = __ldg(rstd + row);
        const bool first = row == blockIdx.x;
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float gy = to_f32(__ldg(gr + c)), xh = (to_f32(__ldg(xr + c)) - mu) * rs;
            const float g = gy * (w ? __ldg(w + c) : 1.f);
            s[0] += g;
            s[1] = fmaf(g, xh, s[1]);
            if (pw) {
                pw[c] = fmaf(gy, xh, first ? 0.f : pw[c]);
                pw[d + c] = gy + (first ? 0.f : pw[d + c]);
            }
        }
        if (!dx) continue;
        group_sum<2, false>(s, buf, phase);
        const float a = s[0] * inv_d, k = s[1] * inv_d;
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float xh = (to_f32(__ldg(xr + c)) - mu) * rs;
            store_elem(dx + row * d + c, rs * (fmaf(to_f32(__ldg(gr + c)), w ? __ldg(w + c) : 1.f, -a) - xh * k));
        }
    }
}

// out[c] = sum over the P blocks of part[p][c], c < 2 d: a block takes 32 columns, its 8 warps a
// strided share of the rows each, added in a fixed order
__global__ void __launch_bounds__(256)
ln_cols_kernel(const float* __restrict__ part, int P, int d, float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float sm[8][33];
    pdl_launch_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * (int64_t)d)
        for (int p = warp; p < P; p += 8) s += part[(int64_t)p * 2 * d + c];
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * (int64_t)d) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sm[k][lane];
        if (c < d) {
            if (dw) dw[c] = s;
        } else if (db) {
            db[c - d] = s;
        }
    }
}

bool rows16(const void* p) { return (uintptr_t)p % 16 == 0; }

// resident blocks of a kernel on the device, for a grid that walks its rows; not asked where the
// blocks wanted are no more than the SMs
template <typename K>
cudaError_t resident(K kern, int threads, size_t smem, int64_t want, int* blocks) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    *blocks = di.sm_count;
    if (want <= di.sm_count) return cudaSuccess;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem);
    *blocks = di.sm_count * (per_sm > 0 ? per_sm : 1);
    return e;
}

template <typename T, int VEC, int NV, int R, bool WARP>
cudaError_t fwd(const LnArgs& a) {
    const int chunks = (a.d + VEC - 1) / VEC;
    const int threads = WARP ? 32 * WARPS : ((chunks + NV - 1) / NV + 31) / 32 * 32;
    auto kern = ln_fwd_kernel<T, VEC, NV, R, WARP>;
    const int64_t want = WARP ? (a.T + WARPS - 1) / WARPS : a.T;
    int cap;
    const cudaError_t e = resident(kern, threads, 0, want, &cap);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(want < cap ? want : cap)), dim3(threads), 0, a.stream,
                      static_cast<const T*>(a.x), a.w, a.b, a.T, a.d, a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
}

template <typename T, int VEC, int NV, int R, bool WARP>
cudaError_t bwd(const LnArgs& a, int* blocks) {
    const int chunks = (a.d + VEC - 1) / VEC;
    const int threads = WARP ? 32 * WARPS : ((chunks + NV - 1) / NV + 31) / 32 * 32;
    const size_t smem = WARP ? (size_t)2 * a.d * 4 : 0;
    auto kern = ln_bwd_kernel<T, VEC, NV, R, WARP>;
    const int64_t want = WARP ? (a.T + WARPS - 1) / WARPS : a.T;
    int cap;
    const cudaError_t e = resident(kern, threads, smem, want, &cap);
    if (e != cudaSuccess) return e;
    if (cap > BWD_BLOCKS) cap = BWD_BLOCKS;
    *blocks = (int)(want < cap ? want : cap);
    return launch_pdl(kern, dim3((unsigned)*blocks), dim3(threads), smem, a.stream, static_cast<const T*>(a.x), a.w,
                      a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d, static_cast<T*>(a.dx), a.part);
}

// The layout of a row by its length in vectors: a warp up to 4 vectors per lane, a block with 2
// (then 4) vectors per thread above that, and element-wise access where rows are not 16-byte
// aligned.  Few rows (at most one block per SM) take one vector per thread: the row's latency counts.
template <typename T>
cudaError_t fwd_t(const LnArgs& a, int sms) {
    constexpr int V = Vec16<T>::VEC;
    if (a.d % V == 0 && rows16(a.x) && rows16(a.y)) {
        const int c = a.d / V;
        if (c <= 32) return fwd<T, V, 1, 4, true>(a);
        if (c <= 1024 && a.T <= sms) return fwd<T, V, 1, 1, false>(a);
        if (c <= 64) return fwd<T, V, 2, 2, true>(a);
        if (c <= 128) return fwd<T, V, 4, 1, true>(a);
        if (c <= 1024) return fwd<T, V, 2, 2, false>(a);
        if (c <= 2048) return fwd<T, V, 4, 1, false>(a);
    } else {
        if (a.d <= 256) return fwd<T, 1, 8, 2, true>(a);
        if (a.d <= 4096) return fwd<T, 1, 8, 2, false>(a);
        if (a.d <= 8192) return fwd<T, 1, 16, 1, false>(a);
    }
    int cap;
    cudaError_t e = resident(ln_fwd_long_kernel<T>, 1024, 0, a.T, &cap);
    if (e != cudaSuccess) return e;
    return launch_pdl(ln_fwd_long_kernel<T>, dim3((unsigned)(a.T < cap ? a.T : cap)), dim3(1024), 0, a.stream,
                      static_cast<const T*>(a.x), a.w, a.b, a.T, a.d, a.eps, static_cast<T*>(a.y), a.mean, a.rstd);
}

template <typename T>
cudaError_t bwd_t(const LnArgs& a, int* blocks) {
    constexpr int V = Vec16<T>::VEC;
    if (a.d % V == 0 && rows16(a.x) && rows16(a.dy) && rows16(a.dx)) {
        const int c = a.d / V;
        if (c <= 32) return bwd<T, V, 1, 2, true>(a, blocks);
        if (c <= 64) return bwd<T, V, 2, 1, true>(a, blocks);
        if (c <= 1024) return bwd<T, V, 2, 2, false>(a, blocks);
        if constexpr (V == 4) {
            if (c <= 2048) return bwd<T, V, 4, 1, false>(a, blocks);
        }
    } else {
        if (a.d <= 256) return bwd<T, 1, 8, 1, true>(a, blocks);
        if (a.d <= 4096) return bwd<T, 1, 8, 1, false>(a, blocks);
        if (a.d <= 8192) return bwd<T, 1, 16, 1, false>(a, blocks);
    }
    int cap;
    cudaError_t e = resident(ln_bwd_long_kernel<T>, 1024, 0, a.T, &cap);
    if (e != cudaSuccess) return e;
    if (cap > BWD_BLOCKS) cap = BWD_BLOCKS;
    *blocks = (int)(a.T < cap ? a.T : cap);
    return launch_pdl(ln_bwd_long_kernel<T>, dim3((unsigned)*blocks), dim3(1024), 0, a.stream,
                      static_cast<const T*>(a.x), a.w, a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d,
                      static_cast<T*>(a.dx), a.part);
}

}  // namespace

int64_t layer_norm_part_floats(int64_t T, int d) {
    const int64_t p = T < BWD_BLOCKS ? T : BWD_BLOCKS;
    return p * 2 * d;
}

cudaError_t launch_layer_norm(const LnArgs& a) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    return a.dt == BF16 ? fwd_t<__nv_bfloat16>(a, di.sm_count) : fwd_t<float>(a, di.sm_count);
}

cudaError_t launch_layer_norm_backward(const LnArgs& a) {
    int blocks = 0;
    cudaError_t e = a.dt == BF16 ? bwd_t<__nv_bfloat16>(a, &blocks) : bwd_t<float>(a, &blocks);
    if (e != cudaSuccess || !a.part) return e;
    const unsigned grid = (unsigned)((2 * (int64_t)a.d + 31) / 32);
    return launch_pdl(ln_cols_kernel, dim3(grid), dim3(256), 0, a.stream, a.part, blocks, a.d, a.dw, a.db);
}

}  // namespace mhc
