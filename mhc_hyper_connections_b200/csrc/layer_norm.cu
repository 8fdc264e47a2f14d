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
// registers), which a mean far from zero does not spoil.  Where the mean's own roundings would show, a third
// walk takes them off (off_centre).
//
// A row belongs to 8, 16 or 32 lanes or to a thread block.  A thread owns the same NV vectors of VEC
// columns in every row it sees, so w and b are loaded once and the backward's column sums stay in
// registers until the thread's last row.
//   * ring kernels, for aligned rows and more of them than SMs: bulk copies bring the next rows into a
//     ring in shared memory, so the loads in flight do not depend on what the warps are doing (without it
//     a block's reductions and stores left HBM idle: 86 us forward at T = 16384, d = 4096, bf16).  One
//     ring and a warp that fills it per block, or (forward, long rows) one per warp: 49 us, 5.5 TB/s.
//   * shift kernels, the same for rows that are not a multiple of 16 bytes;
//   * register kernels, for few rows (latency counts: one vector per thread, no ring to set up), and one
//     element at a time for unaligned rows that the shift kernels do not take;
//   * long kernels, for rows beyond the registers of a block: three walks over the row.
// Column sums are added up in a fixed order: over a group's rows, over a block's warps in shared
// memory, and over the blocks by a second kernel that reads one fp32 row pair per block; or, for few
// rows, by a kernel that reads the rows once more beside the first one, or by blocks of the same launch.
#include <atomic>

#include "common.cuh"
#include "launch.cuh"
#include "tc_ptx.cuh"

namespace mhc {

// 1 once a bounded wait of the ring kernels expired (mhc_device_status).
__device__ unsigned int g_layer_norm_status;

namespace {

// blocks that write column-sum rows for the second kernel: two per SM of a 148-SM device, and up to
// eight where rows are short (T = 16384, d = 1024, bf16: 39 us with two)
int bwd_blocks(int d) { return d >= 4096 ? 296 : d <= 1024 ? 1184 : 296 * 4096 / d; }
// Up to here the column sums come straight from the rows, read a second time from L2 while the row
// kernel runs; above it from the row kernel's registers through `part`.  d = 2560, bf16, T = 128: 3.5 us
// against 8.2, T = 500: 6.4 against 9.6, T = 1000: 14.4 against 11.5.
constexpr int FEW_ROWS = 512;
// Up to here both are one launch, where a block holds a row with one vector per thread: a call 9.5 us against
// 11.7, bound by the host.  In a graph, where the device's time counts, it gains with fewer rows or longer ones
// and loses with others (bf16, T = 64, d = 1024: 2.1 us against 3.6, T = 256, d = 4096: 5.9 and 6.6, fp32 7.6 and
// 7.4; T = 128, d = 515: 2.9 and 2.7, both types; T = 256, d = 512 and 515: 4.9 and 3.5), because its column blocks
// have half the warps.
constexpr int ONE_LAUNCH_ROWS = 256;
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

// Sum R values over the group (G lanes of a warp; G = 0: the first nthr threads of the block); every
// thread of it gets the sums.  The block form alternates between two buffers, so one barrier per call
// is enough: a buffer is written again only after every thread has passed the barrier of the call in
// between.
template <int R, int G>
__device__ __forceinline__ void group_sum(float (&v)[R], float* buf, int& phase, int nthr) {
#pragma unroll
    for (int o = (G ? G : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    if constexpr (G == 0) {
        float* b = buf + phase * 32 * R;
        phase ^= 1;
        const int warp = threadIdx.x >> 5, nw = nthr >> 5;
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) b[warp * R + r] = v[r];
        }
        asm volatile("bar.sync 1, %0;" :: "r"(nthr) : "memory");
#pragma unroll
        for (int r = 0; r < R; ++r) v[r] = 0.f;
        for (int w = 0; w < nw; ++w)
#pragma unroll
            for (int r = 0; r < R; ++r) v[r] += b[w * R + r];
    }
}

// The first mean carries the roundings of its sum.  In a row of nearly equal values far from zero they make up
// most of x - mean and of the variance (12345.678 throughout with eps = 1e-5 gave y = 0.3, and bf16 100
// throughout, d = 1000, eps = 1e-12, gave y = 1).  Such rows, |mean| above 64 standard deviations, are walked
// once more for the sum t of x - mean: the mean moves by t / d, and the sum of squares s falls by t^2 / d.  The
// division (not a product with 1 / d) makes both exact for a row of one value: y = b, rstd = 1 / sqrt(eps).
// Summing t for every row in the second walk took up to a tenth more time (T = 8192, d = 5000, bf16: 46.7 us,
// 41.8 without).
__device__ __forceinline__ bool off_centre(float mean, float s, float inv_d) {
    return mean * mean * 0x1p-12f > s * inv_d;           // false for rows that are not finite
}
__device__ __forceinline__ void centre(float& mean, float& s, float t, int d) {
    const float m1 = t / (float)d;
    mean += m1;
    s = fmaxf(fmaf(-t, m1, s), 0.f);
}
// Such a row in most kernels that hold many registers per thread: the walk over memory, not inlined, so that
// the loop around it keeps its registers (T = 8192, d = 8192, fp32: 83 us, 96 with a walk over registers).  Two
// of them are better off with the walk over registers: bf16, T = 1000, d = 12288 19 us against 26 (the call
// leaves 56 registers there), and odd d = 3453 9.8 against 12.3.  nthr threads share the row, VEC elements at a
// time, G as in group_sum (buf: 32 floats for G = 0).
template <typename T, int VEC, int G>
__device__ __noinline__ float2 recentre(const T* __restrict__ row, int d, int idx, int nthr, float mean, float s,
                                        float* buf) {
    float t = 0.f;
    for (int c = idx * VEC; c < d; c += nthr * VEC) {
        float f[VEC];
        Pack<T, VEC>::unpack(Pack<T, VEC>::load(row + c), f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) t += f[e] - mean;
    }
#pragma unroll
    for (int o = (G ? G : 32) / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if constexpr (G == 0) {
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = t;
        asm volatile("bar.sync 1, %0;" :: "r"(nthr) : "memory");
        t = 0.f;
        for (int w = 0; w < nthr >> 5; ++w) t += buf[w];
        asm volatile("bar.sync 1, %0;" :: "r"(nthr) : "memory");      // before it is written again
    }
    centre(mean, s, t, d);
    return make_float2(mean, s);
}

// threads of a block: a warp per row uses WARPS warps; a block per row as many threads as the row
// needs, up to 1024 with one vector each (few rows) and 512 with more, which the registers allow
// The wait for the kernels before this one: ahead of its reads, or (late) at its end, for a kernel
// launched behind one that reads the same inputs, that waited for them itself before it let this one
// start, and whose outputs this one does not touch.  Waiting at the end keeps the stream's order for what
// follows.
struct StreamOrder {
    bool late;
    __device__ __forceinline__ explicit StreamOrder(bool l) : late(l) {
        if (!late) pdl_wait();
    }
    __device__ __forceinline__ ~StreamOrder() {
        if (late) pdl_wait();
    }
};

template <int NV, bool WARP> constexpr int MAX_THREADS = WARP ? 32 * WARPS : (NV == 1 ? 1024 : 512);

template <typename T, int VEC, int NV, int R, bool WARP>
__global__ void __launch_bounds__(MAX_THREADS<NV, WARP>)
ln_fwd_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b,
                              int64_t Tn, int d, float eps, T* __restrict__ y, float* __restrict__ mean_out,
                              float* __restrict__ rstd_out) {
    using P = Pack<T, VEC>;
    __shared__ float buf[WARP ? 1 : 64 * R], far[WARP ? 1 : 64];
    int phase = 0, far_phase = 0;
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
        group_sum<R, WARP ? 32 : 0>(s, buf, phase, nthr);
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
        group_sum<R, WARP ? 32 : 0>(s, buf, phase, nthr);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!off_centre(mean[r], s[r], inv_d)) continue;      // the same in the whole group; rows past Tn are 0
            if constexpr (NV == 1 || (NV == 8 && !WARP && sizeof(T) == 2)) {
                float t[1] = {0.f};
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float f[VEC];
                    P::unpack(raw[r][v], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        if ((v * nthr + idx) * VEC < d) t[0] += f[e] - mean[r];
                }
                group_sum<1, WARP ? 32 : 0>(t, far, far_phase, nthr);
                centre(mean[r], s[r], t[0], d);
            } else {
                const float2 m = recentre<T, VEC, WARP ? 32 : 0>(x + (row0 + r * groups) * d, d, idx, nthr, mean[r],
                                                                 s[r], far);
                mean[r] = m.x;
                s[r] = m.y;
            }
        }
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
    __shared__ float buf[64], far[32];
    int phase = 0;
    pdl_launch_next();
    pdl_wait();
    const float inv_d = 1.0f / (float)d;
    for (int64_t row = blockIdx.x; row < Tn; row += gridDim.x) {
        const T* xr = x + row * d;
        float s[1] = {0.f};
        for (int c = threadIdx.x; c < d; c += blockDim.x) s[0] += to_f32(__ldg(xr + c));
        group_sum<1, 0>(s, buf, phase, blockDim.x);
        float mean = s[0] * inv_d;
        s[0] = 0.f;
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float v = to_f32(__ldg(xr + c)) - mean;
            s[0] = fmaf(v, v, s[0]);
        }
        group_sum<1, 0>(s, buf, phase, blockDim.x);
        if (off_centre(mean, s[0], inv_d)) {
            const float2 m = recentre<T, 1, 0>(xr, d, threadIdx.x, blockDim.x, mean, s[0], far);
            mean = m.x;
            s[0] = m.y;
        }
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
                              T* __restrict__ dx, float* __restrict__ part, bool late) {
    using P = Pack<T, VEC>;
    __shared__ float buf[WARP ? 1 : 64 * 2 * R];
    extern __shared__ float cols[];        // WARP: [2][d] column sums of the block
    int phase = 0;
    pdl_launch_next();
    const StreamOrder order(late);
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
        group_sum<2 * R, WARP ? 32 : 0>(sums, buf, phase, nthr);
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
                                   const T* __restrict__ dy, int64_t Tn, int d, T* __restrict__ dx, float* part,
                                   bool late) {
    __shared__ float buf[64 * 2];
    int phase = 0;
    pdl_launch_next();
    const StreamOrder order(late);
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
        group_sum<2, 0>(s, buf, phase, blockDim.x);
        const float a = s[0] * inv_d, k = s[1] * inv_d;
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            const float xh = (to_f32(__ldg(xr + c)) - mu) * rs;
            store_elem(dx + row * d + c, rs * (fmaf(to_f32(__ldg(gr + c)), w ? __ldg(w + c) : 1.f, -a) - xh * k));
        }
    }
}

// ---- ring kernels

constexpr int MAX_SLOTS = 8;
constexpr int WARP_SLOTS = 4;            // of a warp's own ring
constexpr unsigned long long kRingLandNs = 2000000ull;       // after a failed wait: copies in flight land

// A wait that expires sets the status word and the block's abort flag; after it no wait blocks, the
// loops run out and the outputs are incomplete.
__device__ __forceinline__ bool wait_until(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned long long limit_ns) {
    for (int i = 0; i < 256; ++i) {
        if (ptx::mbar_try(bar, parity)) return true;
        if (*abort_flag) return false;
    }
    const uint64_t t0 = ptx::gtimer();
    while (true) {
        if (ptx::mbar_try(bar, parity)) return true;
        if (*abort_flag) return false;
        if (ptx::gtimer() - t0 > limit_ns) {
            atomicOr(&g_layer_norm_status, 1u);
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void land() {
    const uint64_t t0 = ptx::gtimer();
    while (ptx::gtimer() - t0 < kRingLandNs) __nanosleep(1000);
}

// The wait limit, and the failure-path test hook: batches after which loading stops (< 0: never)
struct Limits {
    unsigned long long wait_ns;
    int stop;
};

// A ring of slots filled by the producer warp.
struct Ring {
    uint64_t* bars;                      // [2 MAX_SLOTS]: full, empty
    volatile int* abort_flag;
    int slots;
    Limits lim;
    int s = 0;
    uint32_t parity = 0;

    __device__ __forceinline__ uint32_t full() const { return ptx::smem_u32(bars + s); }
    __device__ __forceinline__ uint32_t empty() const { return ptx::smem_u32(bars + MAX_SLOTS + s); }
    __device__ __forceinline__ void next() {
        if (++s == slots) {
            s = 0;
            parity ^= 1u;
        }
    }
    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t par) const { return wait_until(bar, par, abort_flag, lim.wait_ns); }
};

// set up by thread 0; the caller synchronises the block
__device__ __forceinline__ void ring_init(uint64_t* bars, int* abort_flag, int slots, int readers) {
    for (int i = 0; i < slots; ++i) {
        ptx::mbar_init(ptx::smem_u32(bars + i), 1);
        ptx::mbar_init(ptx::smem_u32(bars + MAX_SLOTS + i), readers);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// The producer warp's loop: NT tensors' rows of each of the block's batches, side by side in a slot
template <int NT>
__device__ __forceinline__ void ring_produce(Ring ring, unsigned char* smem, const unsigned char* const (&src)[NT],
                                             int64_t Tn, int B, int64_t row_bytes, int64_t batches) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        int left = ring.lim.stop;
        for (int64_t i = blockIdx.x; i < batches && left != 0; i += gridDim.x, ring.next(), --left) {
            if (!(ok = ring.wait(ring.empty(), ring.parity ^ 1u))) break;
            const int64_t row = i * B;
            const uint32_t bytes = (uint32_t)((Tn - row < B ? Tn - row : B) * row_bytes);
            ptx::mbar_arrive_tx(ring.full(), NT * bytes);
            const uint32_t dst = ptx::smem_u32(smem) + (uint32_t)(ring.s * NT * B * row_bytes);
#pragma unroll
            for (int t = 0; t < NT; ++t)
                ptx::bulk_g2s(dst + (uint32_t)(t * B * row_bytes), src[t] + row * row_bytes, bytes, ring.full());
        }
        if (!ok) land();
    }
    __syncwarp();
}

// A 16-byte vector as fp32 pairs, and back: the arithmetic below is in pairs, which halves its
// instructions (at d = 4096 the forward kernel issued more than it loaded without)
__device__ __forceinline__ void pairs_of(uint4 v, float2 (&f)[4]) {
    f[0] = bf16x2_to_f32x2(v.x); f[1] = bf16x2_to_f32x2(v.y);
    f[2] = bf16x2_to_f32x2(v.z); f[3] = bf16x2_to_f32x2(v.w);
}
__device__ __forceinline__ void pairs_of(uint4 v, float2 (&f)[2]) {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint4 vector_of(const float2 (&f)[4]) {
    return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                      pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ uint4 vector_of(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// w (or b) of a thread's NV vectors of columns, or `none` where the caller gave no array.  In registers:
// re-read from L1 for every row (32-byte pieces per thread) they took longer than the row itself.
template <int NV, int HV>
__device__ __forceinline__ void load_columns(const float* __restrict__ p, int d, int nthr, int idx, float none,
                                             float2 (&f)[NV][HV]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (v * nthr + idx) * 2 * HV;
#pragma unroll
        for (int e = 0; e < HV; ++e)
            f[v][e] = p && c < d ? make_float2(__ldg(p + c + 2 * e), __ldg(p + c + 2 * e + 1)) : both(none);
    }
}

// Rows belong to groups of G lanes (G = 8, 16, 32), or to the block (G = 0).  A group takes R rows at
// a time, NV 16-byte vectors per thread and row; a slot holds the B rows that the block takes at a time.
// TH: the most threads that share a row and its registers; 224 leaves room for a second block on the SM.
template <typename T, int NV, int R, int G, int TH>
__global__ void __launch_bounds__(TH + 32, TH == 224 ? 2 : 0)
ln_fwd_ring_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, int64_t Tn, int d,
                   float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int slots,
                   Limits lim) {
    constexpr int VEC = Vec16<T>::VEC, HV = VEC / 2;
    constexpr int B = G ? WARPS * (32 / (G ? G : 32)) * R : R;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[2 * MAX_SLOTS];
    __shared__ int abort_flag;
    __shared__ __align__(16) float buf[G ? 1 : 64 * R], far[G ? 1 : 32];
    int phase = 0;
    const int consumers = blockDim.x - 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) ring_init(bars, &abort_flag, slots, consumers >> 5);
    __syncthreads();
    pdl_launch_next();
    pdl_wait();
    Ring ring{bars, &abort_flag, slots, lim};
    const int64_t batches = (Tn + B - 1) / B, row_bytes = (int64_t)d * sizeof(T);
    if (warp == consumers >> 5) {
        const unsigned char* const src[1] = {reinterpret_cast<const unsigned char*>(x)};
        ring_produce<1>(ring, smem, src, Tn, B, row_bytes, batches);
        return;
    }
    const int nthr = G ? G : consumers, idx = G ? lane % (G ? G : 32) : threadIdx.x;
    const int first = G ? (threadIdx.x / (G ? G : 32)) * R : 0;        // the group's first row of a batch
    const float inv_d = 1.0f / (float)d;
    float2 wv[NV][HV], bv[NV][HV];
    load_columns<NV, HV>(w, d, nthr, idx, 1.f, wv);
    load_columns<NV, HV>(b, d, nthr, idx, 0.f, bv);
    for (int64_t i = blockIdx.x; i < batches; i += gridDim.x, ring.next()) {
        ring.wait(ring.full(), ring.parity);
        const T* rows = reinterpret_cast<const T*>(smem + (int64_t)ring.s * B * row_bytes) + (int64_t)first * d;
        // rows past Tn hold what the slot held before; nothing of them is stored
        uint4 raw[R][NV];
        float s[R], mean[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 acc = both(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int c = (v * nthr + idx) * VEC;
                raw[r][v] = c < d ? *reinterpret_cast<const uint4*>(rows + (int64_t)r * d + c) : make_uint4(0, 0, 0, 0);
                float2 f[HV];
                pairs_of(raw[r][v], f);
#pragma unroll
                for (int e = 0; e < HV; ++e) acc = __fadd2_rn(acc, f[e]);
            }
            s[r] = acc.x + acc.y;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ring.empty());                 // the slot is in registers
        group_sum<R, G>(s, buf, phase, nthr);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = s[r] * inv_d;
            float2 acc = both(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if ((v * nthr + idx) * VEC >= d) continue;
                float2 f[HV];
                pairs_of(raw[r][v], f);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 c = __fadd2_rn(f[e], both(-mean[r]));
                    acc = __ffma2_rn(c, c, acc);
                }
            }
            s[r] = acc.x + acc.y;
        }
        group_sum<R, G>(s, buf, phase, nthr);
        if constexpr (G != 0 || TH == 512) {
            bool off = false;             // the same in the whole group
#pragma unroll
            for (int r = 0; r < R; ++r) off |= off_centre(mean[r], s[r], inv_d);
            if (G ? __any_sync(0xffffffffu, off) : off) {
                float t[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float2 acc = both(0.f);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        if ((v * nthr + idx) * VEC >= d) continue;
                        float2 f[HV];
                        pairs_of(raw[r][v], f);
#pragma unroll
                        for (int e = 0; e < HV; ++e) acc = __fadd2_rn(acc, __fadd2_rn(f[e], both(-mean[r])));
                    }
                    t[r] = acc.x + acc.y;
                }
                group_sum<R, G>(t, buf, phase, nthr);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (off_centre(mean[r], s[r], inv_d)) centre(mean[r], s[r], t[r], d);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t row = i * B + r;
                if (row < Tn && off_centre(mean[r], s[r], inv_d)) {
                    const float2 m = recentre<T, VEC, 0>(x + row * d, d, idx, nthr, mean[r], s[r], far);
                    mean[r] = m.x;
                    s[r] = m.y;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = i * B + first + r;
            s[r] = 1.0f / sqrtf(fmaf(s[r], inv_d, eps));               // rstd
            if (idx == 0 && mean_out && row < Tn) {
                mean_out[row] = mean[r];
                rstd_out[row] = s[r];
            }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nthr + idx) * VEC;
            if (c >= d) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t row = i * B + first + r;
                if (row >= Tn) break;
                float2 f[HV];
                pairs_of(raw[r][v], f);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 xh = __fmul2_rn(__fadd2_rn(f[e], both(-mean[r])), both(s[r]));
                    f[e] = __ffma2_rn(xh, wv[v][e], bv[v][e]);
                }
                st_v4(y + row * d + c, vector_of(f));
            }
        }
    }
}

// Forward, a row per warp in NV vectors per lane, with w and b in shared memory.  No barriers: the rows
// of an SM's warps are at different points, so loads, reductions and stores overlap, and each warp has
// a ring of its own that it refills as soon as a row is in registers.  The 32-byte pieces of w and b
// that go with a bf16 vector are stored as two planes of 16 bytes per lane, which reads without bank
// conflicts.
// blocks of 256 threads per SM, as many as the registers of a row per warp allow (bf16, 8 vectors, T = 16384:
// d = 2048 22.3 us with two and 25.2 with three, d = 1537 29.5 and 33.8; fp32, d = 1024 20.9 and 19.7)
template <typename T, int NV>
constexpr int WARP_BLOCKS = NV > 10 ? 1 : NV > 8 || (NV == 8 && sizeof(T) == 2) ? 2 : NV > 4 ? 3 : 4;

template <typename T, int NV>
__global__ void __launch_bounds__(256, WARP_BLOCKS<T, NV>)
ln_fwd_warp_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, int64_t Tn, int d,
                   float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int slots,
                   Limits lim) {
    constexpr int TH = 256;
    constexpr int VEC = Vec16<T>::VEC, HV = VEC / 2, PL = VEC / 4;
    extern __shared__ float4 wb[];      // [w, b][NV][PL][32], then the warps' slots
    __shared__ __align__(8) uint64_t bars[TH / 32][WARP_SLOTS];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < TH / 32 * WARP_SLOTS) ptx::mbar_init(ptx::smem_u32(&bars[0][0] + threadIdx.x), 1);
    if (threadIdx.x == 0) abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    pdl_launch_next();
    pdl_wait();
    const int row_bytes = d * (int)sizeof(T);
    const int64_t warps = (int64_t)gridDim.x * (TH / 32);
    int64_t row = (int64_t)warp * gridDim.x + blockIdx.x;      // the last, partial round goes to all blocks
    unsigned char* ring = reinterpret_cast<unsigned char*>(wb + 2 * NV * PL * 32) + (size_t)warp * slots * row_bytes;
    int left = lim.stop;
    auto load = [&](int64_t r, int s) {
        if (left == 0) return;
        --left;
        const uint32_t bar = ptx::smem_u32(&bars[warp][s]);
        ptx::mbar_arrive_tx(bar, row_bytes);
        ptx::bulk_g2s(ptx::smem_u32(ring) + s * row_bytes, x + r * d, row_bytes, bar);
    };
    if (lane == 0)
        for (int s = 0; s < slots; ++s)
            if (row + s * warps < Tn) load(row + s * warps, s);
    bool ok = true;
    int slot = 0;
    uint32_t parity = 0;
    auto four = [&](const float* p, int c, float none) {
        if (!p || c >= d) return make_float4(none, none, none, none);
        if ((uintptr_t)p % 16 == 0) return __ldg(reinterpret_cast<const float4*>(p + c));
        return make_float4(__ldg(p + c), __ldg(p + c + 1), __ldg(p + c + 2), __ldg(p + c + 3));
    };
#pragma unroll 2
    for (int i = threadIdx.x; i < NV * 32 * PL; i += TH) {
        const int at = (i / (32 * PL) * PL + i % PL) * 32 + i / PL % 32;
        wb[at] = four(w, 4 * i, 1.f);
        wb[NV * PL * 32 + at] = four(b, 4 * i, 0.f);
    }
    __syncthreads();
    const float inv_d = 1.0f / (float)d;
    for (; row < Tn; row += warps) {
        ok = wait_until(ptx::smem_u32(&bars[warp][slot]), parity, &abort_flag, lim.wait_ns) && ok;
        uint4 raw[NV];
        const T* xr = reinterpret_cast<const T*>(ring + (size_t)slot * row_bytes) + lane * VEC;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            raw[v] = (v * 32 + lane) * VEC < d ? *reinterpret_cast<const uint4*>(xr + v * 32 * VEC)
                                               : make_uint4(0, 0, 0, 0);
        __syncwarp();
        if (lane == 0 && row + slots * warps < Tn) load(row + slots * warps, slot);
        if (++slot == slots) {
            slot = 0;
            parity ^= 1u;
        }
        float2 a0 = both(0.f), a1 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int e = 0; e < HV; e += 2) {
                a0 = __fadd2_rn(a0, f[e]);
                a1 = __fadd2_rn(a1, f[e + 1]);
            }
        }
        float s = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        float mean = s * inv_d;
        a0 = a1 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if ((v * 32 + lane) * VEC >= d) continue;
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int e = 0; e < HV; e += 2) {
                const float2 c0 = __fadd2_rn(f[e], both(-mean)), c1 = __fadd2_rn(f[e + 1], both(-mean));
                a0 = __ffma2_rn(c0, c0, a0);
                a1 = __ffma2_rn(c1, c1, a1);
            }
        }
        s = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (off_centre(mean, s, inv_d)) {
            a0 = both(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if ((v * 32 + lane) * VEC >= d) continue;
                float2 f[HV];
                pairs_of(raw[v], f);
#pragma unroll
                for (int e = 0; e < HV; ++e) a0 = __fadd2_rn(a0, __fadd2_rn(f[e], both(-mean)));
            }
            float t = a0.x + a0.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            centre(mean, s, t, d);
        }
        const float rstd = 1.0f / sqrtf(fmaf(s, inv_d, eps));
        T* yr = y + row * d + lane * VEC;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int h = 0; h < PL; ++h) {
                const float4 wq = wb[(v * PL + h) * 32 + lane], bq = wb[((NV + v) * PL + h) * 32 + lane];
                const float2 x0 = __fmul2_rn(__fadd2_rn(f[2 * h], both(-mean)), both(rstd));
                const float2 x1 = __fmul2_rn(__fadd2_rn(f[2 * h + 1], both(-mean)), both(rstd));
                f[2 * h] = __ffma2_rn(x0, make_float2(wq.x, wq.y), make_float2(bq.x, bq.y));
                f[2 * h + 1] = __ffma2_rn(x1, make_float2(wq.z, wq.w), make_float2(bq.z, bq.w));
            }
            if ((v * 32 + lane) * VEC < d) st_v4(yr + v * 32 * VEC, vector_of(f));
        }
        if (lane == 0 && mean_out) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
    }
    if (!ok) land();
}

// the same; a slot holds B rows of x, then B rows of dy
template <typename T, int NV, int R, int G, int TH>
__global__ void __launch_bounds__(TH + 32, 1)
ln_bwd_ring_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
                   const float* __restrict__ rstd, const T* __restrict__ dy, int64_t Tn, int d, T* __restrict__ dx,
                   float* __restrict__ part, bool late, int slots, Limits lim) {
    constexpr int VEC = Vec16<T>::VEC, HV = VEC / 2;
    constexpr int GROUPS = G ? WARPS * (32 / (G ? G : 32)) : 1, B = GROUPS * R;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t bars[2 * MAX_SLOTS];
    __shared__ int abort_flag;
    __shared__ __align__(16) float buf[G ? 1 : 128 * R];
    int phase = 0;
    const int consumers = blockDim.x - 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) ring_init(bars, &abort_flag, slots, consumers >> 5);
    __syncthreads();
    pdl_launch_next();
    const StreamOrder order(late);
    Ring ring{bars, &abort_flag, slots, lim};
    const int64_t batches = (Tn + B - 1) / B, row_bytes = (int64_t)d * sizeof(T);
    if (warp == consumers >> 5) {
        const unsigned char* const src[2] = {reinterpret_cast<const unsigned char*>(x),
                                             reinterpret_cast<const unsigned char*>(dy)};
        ring_produce<2>(ring, smem, src, Tn, B, row_bytes, batches);
        return;
    }
    const int nthr = G ? G : consumers, idx = G ? lane % (G ? G : 32) : threadIdx.x;
    const int group = G ? threadIdx.x / (G ? G : 32) : 0, first = group * R;
    const float inv_d = 1.0f / (float)d;
    float2 wv[NV][HV], dw[NV][HV], db[NV][HV];
    load_columns<NV, HV>(w, d, nthr, idx, 1.f, wv);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < HV; ++e) dw[v][e] = db[v][e] = both(0.f);
    float mu_n[R], rs_n[R];              // the statistics of the group's rows, loaded one batch ahead
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = i * B + first + r;
            mu_n[r] = row < Tn ? __ldg(mean + row) : 0.f;
            rs_n[r] = row < Tn ? __ldg(rstd + row) : 0.f;
        }
    };
    fetch(blockIdx.x);
    for (int64_t i = blockIdx.x; i < batches; i += gridDim.x, ring.next()) {
        float mu[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = mu_n[r];
            rs[r] = rs_n[r];
        }
        fetch(i + gridDim.x);
        ring.wait(ring.full(), ring.parity);
        const T* xs = reinterpret_cast<const T*>(smem + (int64_t)ring.s * 2 * B * row_bytes) + (int64_t)first * d;
        const T* gs = xs + (int64_t)B * d;
        // x waits as it was stored, g as fp32: unpacking dy again costs more than the registers (T = 16384, d =
        // 4096: 81 us against 77)
        uint4 xr[R][NV];
        float2 gk[R][NV][HV];
        float2 sg[R], sx[R];                         // sums of g, of g xh
#pragma unroll
        for (int r = 0; r < R; ++r) sg[r] = sx[r] = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nthr + idx) * VEC;
            if (c >= d) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (i * B + first + r >= Tn) break;          // the slot's last contents
                xr[r][v] = *reinterpret_cast<const uint4*>(xs + (int64_t)r * d + c);
                const uint4 graw = *reinterpret_cast<const uint4*>(gs + (int64_t)r * d + c);
                float2 xf[HV], gf[HV];
                pairs_of(xr[r][v], xf);
                pairs_of(graw, gf);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 xh = __fmul2_rn(__fadd2_rn(xf[e], both(-mu[r])), both(rs[r]));
                    const float2 g = gk[r][v][e] = __fmul2_rn(gf[e], wv[v][e]);
                    dw[v][e] = __ffma2_rn(gf[e], xh, dw[v][e]);
                    db[v][e] = __fadd2_rn(db[v][e], gf[e]);
                    sg[r] = __fadd2_rn(sg[r], g);
                    sx[r] = __ffma2_rn(g, xh, sx[r]);
                }
            }
        }
        float sums[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sums[r] = sg[r].x + sg[r].y;
            sums[R + r] = sx[r].x + sx[r].y;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ring.empty());
        if (!dx) continue;
        group_sum<2 * R, G>(sums, buf, phase, nthr);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nthr + idx) * VEC;
            if (c >= d) continue;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t row = i * B + first + r;
                if (row >= Tn) break;
                // dx = rs g w - (rs q) xh - rs a
                const float2 a = both(-rs[r] * (sums[r] * inv_d)), q = both(-rs[r] * (sums[R + r] * inv_d) * rs[r]);
                float2 xf[HV], gf[HV];
                pairs_of(xr[r][v], xf);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 t = __ffma2_rn(__fadd2_rn(xf[e], both(-mu[r])), q, a);
                    gf[e] = __ffma2_rn(gk[r][v][e], both(rs[r]), t);
                }
                st_v4(dx + row * d + c, vector_of(gf));
            }
        }
    }
    if (!part) return;
    float* pw = part + (int64_t)blockIdx.x * 2 * d;
    if constexpr (G != 0) {
        // the block's groups add their sums in turn, over the ring (every row in it has been read)
        float* cols = reinterpret_cast<float*>(smem);
#pragma unroll 1
        for (int k = 0; k < GROUPS; ++k) {
            if (k % (32 / (G ? G : 32)) == 0) asm volatile("bar.sync 1, %0;" :: "r"(consumers) : "memory");
            __syncwarp();
            if (group == k) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int c = (v * nthr + idx) * VEC;
                    if (c < d)
#pragma unroll
                        for (int e = 0; e < HV; ++e) {
                            float2* cw = reinterpret_cast<float2*>(cols + c + 2 * e);
                            float2* cb = reinterpret_cast<float2*>(cols + d + c + 2 * e);
                            *cw = k ? __fadd2_rn(*cw, dw[v][e]) : dw[v][e];
                            *cb = k ? __fadd2_rn(*cb, db[v][e]) : db[v][e];
                        }
                }
            }
        }
        asm volatile("bar.sync 1, %0;" :: "r"(consumers) : "memory");
        for (int c = threadIdx.x; c < 2 * d; c += consumers) pw[c] = cols[c];
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (v * nthr + idx) * VEC;
            if (c < d)
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    *reinterpret_cast<float2*>(pw + c + 2 * e) = dw[v][e];
                    *reinterpret_cast<float2*>(pw + d + c + 2 * e) = db[v][e];
                }
        }
    }
}

// ---- rows that are not 16-byte aligned
//
// A row of d elements that is not a multiple of 16 bytes starts anywhere within a 16-byte word, but rows
// eight apart start at the same place in theirs.  So a block takes every (8 k)-th row, and sees one
// shift s: its word j holds the columns VEC j - s .. VEC j - s + VEC - 1 of each of them, and the kernels
// are those of aligned rows but for the two words at the ends, which hold elements of other rows too.
// The bulk copies bring the whole words around a row; the last row's copy ends with the last whole word
// of the array.  Arrays themselves are 16-byte aligned.
template <typename T>
struct Shifted {
    static constexpr int VEC = Vec16<T>::VEC;
    const T* p;
    int64_t Tn;
    int d, s, row_bytes, slot_bytes;     // slot_bytes: room for a row's words

    __device__ __forceinline__ Shifted(const T* p_, int64_t Tn_, int d_, int64_t row)
        : p(p_), Tn(Tn_), d(d_), s((int)(row * d_ * (int64_t)sizeof(T) & 15) / (int)sizeof(T)),
          row_bytes(d_ * (int)sizeof(T)), slot_bytes((row_bytes + 15) / 16 * 16 + 16) {}
    // first byte of the row's words, and how many bytes of them are copied
    __device__ __forceinline__ int64_t at(int64_t row) const { return row * row_bytes & ~(int64_t)15; }
    __device__ __forceinline__ int bytes(int64_t row) const {
        const int64_t up = (row * row_bytes + row_bytes + 15) & ~(int64_t)15, last = Tn * row_bytes & ~(int64_t)15;
        return (int)((up < last ? up : last) - at(row));
    }
    __device__ __forceinline__ void load(int64_t row, uint32_t dst, uint32_t bar) const {
        ptx::bulk_g2s(dst, reinterpret_cast<const unsigned char*>(p) + at(row), bytes(row), bar);
    }
    // words of a row, and how many elements of the first and the last belong to other rows
    __device__ __forceinline__ int words() const { return (d + s + VEC - 1) / VEC; }
    __device__ __forceinline__ int spare() const { return words() * VEC - d - s; }
    // ones over the elements of word j that belong to the row
    __device__ __forceinline__ uint4 mask(int j) const {
        uint32_t m[4] = {};
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = j * VEC + i - s;
            if (c >= 0 && c < d) m[i * 4 / VEC] |= sizeof(T) == 4 ? 0xFFFFFFFFu : 0xFFFFu << (16 * (i & 1));
        }
        return make_uint4(m[0], m[1], m[2], m[3]);
    }
    // The last row may end inside a word that is not copied: its elements from memory, into the slot, by
    // the thread that reads the word.
    __device__ __forceinline__ void tail(unsigned char* slot, int64_t row) const {
        const int j = words() - 1;
        T* e = reinterpret_cast<T*>(slot + 16 * j);
#pragma unroll 1
        for (int i = 0; i < VEC; ++i) {
            const int c = j * VEC + i - s;
            if (c >= 0 && c < d) e[i] = __ldg(p + row * d + c);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    // the elements of such a word that belong to the row
    __device__ __forceinline__ void store_part(T* out, int64_t row, int j, uint4 v) const {
        T* o = reinterpret_cast<T*>(reinterpret_cast<unsigned char*>(out) + at(row) + 16 * j);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = j * VEC + i - s;
            if (c < 0 || c >= d) continue;
            if constexpr (sizeof(T) == 2)
                o[i] = __ushort_as_bfloat16((unsigned short)(w[i / 2] >> (16 * (i & 1))));
            else
                o[i] = __uint_as_float(w[i]);
        }
    }
};

__device__ __forceinline__ uint4 masked(uint4 v, uint4 m) {
    return make_uint4(v.x & m.x, v.y & m.y, v.z & m.z, v.w & m.w);
}

// ln_fwd_warp_kernel for such rows; gridDim.x is a multiple of 8
template <typename T, int NV>
__global__ void __launch_bounds__(256, WARP_BLOCKS<T, NV>)
ln_fwd_shift_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ b, int64_t Tn, int d,
                    float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, int slots,
                    Limits lim) {
    constexpr int TH = 256, VEC = Vec16<T>::VEC, HV = VEC / 2, PL = VEC / 4;
    extern __shared__ float4 wb[];      // [w, b][NV][PL][32], then the warps' slots
    __shared__ __align__(8) uint64_t bars[TH / 32][WARP_SLOTS];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < TH / 32 * WARP_SLOTS) ptx::mbar_init(ptx::smem_u32(&bars[0][0] + threadIdx.x), 1);
    if (threadIdx.x == 0) abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    pdl_launch_next();
    pdl_wait();
    const Shifted<T> sx(x, Tn, d, blockIdx.x);
    const int64_t warps = (int64_t)gridDim.x * (TH / 32);
    int64_t row = (int64_t)warp * gridDim.x + blockIdx.x;
    unsigned char* ring = reinterpret_cast<unsigned char*>(wb + 2 * NV * PL * 32) + (size_t)warp * slots * sx.slot_bytes;
    int left = lim.stop;
    auto load = [&](int64_t r, int s) {
        if (left == 0) return;
        --left;
        const uint32_t bar = ptx::smem_u32(&bars[warp][s]);
        ptx::mbar_arrive_tx(bar, sx.bytes(r));
        sx.load(r, ptx::smem_u32(ring) + s * sx.slot_bytes, bar);
    };
    if (lane == 0)
        for (int s = 0; s < slots; ++s)
            if (row + s * warps < Tn) load(row + s * warps, s);
    bool ok = true;
    int slot = 0;
    uint32_t parity = 0;
    for (int i = threadIdx.x; i < NV * 32 * VEC; i += TH) {
        const int v = i / (32 * VEC), l = i / VEC % 32, e = i % VEC, c = i - sx.s;
        const int at = ((v * PL + e / 4) * 32 + l) * 4 + e % 4;
        reinterpret_cast<float*>(wb)[at] = w && c >= 0 && c < d ? __ldg(w + c) : 1.f;
        reinterpret_cast<float*>(wb)[NV * 32 * VEC + at] = b && c >= 0 && c < d ? __ldg(b + c) : 0.f;
    }
    __syncthreads();
    const float inv_d = 1.0f / (float)d;
    // this lane's words at the ends of the row: word 0, and the last one in round vl; 1 in place of their
    // elements that belong to the row, 0 of the others
    const int nw = sx.words(), vl = (nw - 1) / 32;
    const int j_lo = sx.s > 0 ? 1 : 0, j_hi = sx.spare() > 0 ? nw - 1 : nw;        // whole words
    const bool first = lane == 0 && sx.s > 0, last = lane == (nw - 1) % 32 && sx.spare() > 0;
    const uint4 mask0 = sx.mask(lane), mask1 = sx.mask(vl * 32 + lane);
    float2 keep0[HV], keep1[HV];
#pragma unroll
    for (int e = 0; e < HV; ++e) {
        auto in = [&](int j, int i) { return j * VEC + i - sx.s >= 0 && j * VEC + i - sx.s < d ? 1.f : 0.f; };
        keep0[e] = make_float2(in(lane, 2 * e), in(lane, 2 * e + 1));
        keep1[e] = make_float2(in(vl * 32 + lane, 2 * e), in(vl * 32 + lane, 2 * e + 1));
    }
    for (; row < Tn; row += warps) {
        ok = wait_until(ptx::smem_u32(&bars[warp][slot]), parity, &abort_flag, lim.wait_ns) && ok;
        unsigned char* xs = ring + (size_t)slot * sx.slot_bytes;
        if (last && row == Tn - 1) sx.tail(xs, row);
        uint4 raw[NV];
        float2 a0 = both(0.f), a1 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
        {
            raw[v] = v * 32 + lane < nw ? *reinterpret_cast<const uint4*>(xs + 16 * (v * 32 + lane))
                                        : make_uint4(0, 0, 0, 0);
            if (v == 0) raw[v] = masked(raw[v], mask0);
            if (v == vl) raw[v] = masked(raw[v], mask1);
        }
        __syncwarp();
        if (lane == 0 && row + slots * warps < Tn) load(row + slots * warps, slot);
        if (++slot == slots) {
            slot = 0;
            parity ^= 1u;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int e = 0; e < HV; e += 2) {
                a0 = __fadd2_rn(a0, f[e]);
                a1 = __fadd2_rn(a1, f[e + 1]);
            }
        }
        float sum = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float mean = sum * inv_d;
        a0 = a1 = both(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (v * 32 + lane >= nw) continue;
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int e = 0; e < HV; ++e) {
                f[e] = __fadd2_rn(f[e], both(-mean));
                if (v == 0) f[e] = __fmul2_rn(f[e], keep0[e]);
                if (v == vl) f[e] = __fmul2_rn(f[e], keep1[e]);
                if (e & 1)
                    a1 = __ffma2_rn(f[e], f[e], a1);
                else
                    a0 = __ffma2_rn(f[e], f[e], a0);
            }
        }
        sum = (a0.x + a0.y) + (a1.x + a1.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (off_centre(mean, sum, inv_d)) {
            a0 = both(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (v * 32 + lane >= nw) continue;
                float2 f[HV];
                pairs_of(raw[v], f);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    f[e] = __fadd2_rn(f[e], both(-mean));
                    if (v == 0) f[e] = __fmul2_rn(f[e], keep0[e]);
                    if (v == vl) f[e] = __fmul2_rn(f[e], keep1[e]);
                    a0 = __fadd2_rn(a0, f[e]);
                }
            }
            float t = a0.x + a0.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            centre(mean, sum, t, d);
        }
        const float rstd = 1.0f / sqrtf(fmaf(sum, inv_d, eps));
        unsigned char* yr = reinterpret_cast<unsigned char*>(y) + sx.at(row);
        uint4 end0 = make_uint4(0, 0, 0, 0), end1 = end0;      // words that are not wholly the row's
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int j = v * 32 + lane;
            float2 f[HV];
            pairs_of(raw[v], f);
#pragma unroll
            for (int h = 0; h < PL; ++h) {
                const float4 wq = wb[(v * PL + h) * 32 + lane], bq = wb[((NV + v) * PL + h) * 32 + lane];
                const float2 x0 = __fmul2_rn(__fadd2_rn(f[2 * h], both(-mean)), both(rstd));
                const float2 x1 = __fmul2_rn(__fadd2_rn(f[2 * h + 1], both(-mean)), both(rstd));
                f[2 * h] = __ffma2_rn(x0, make_float2(wq.x, wq.y), make_float2(bq.x, bq.y));
                f[2 * h + 1] = __ffma2_rn(x1, make_float2(wq.z, wq.w), make_float2(bq.z, bq.w));
            }
            const uint4 o = vector_of(f);
            if (j >= j_lo && j < j_hi) st_v4(yr + 16 * j, o);
            if (v == 0) end0 = o;
            if (v == vl) end1 = o;
        }
        if (first || last) {
#pragma unroll 1
            for (int k = 0; k < 2; ++k)
                if (k ? last : first) sx.store_part(y, row, k ? nw - 1 : 0, k ? end1 : end0);
        }
        if (lane == 0 && mean_out) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
    }
    if (!ok) land();
}

// ln_bwd_ring_kernel for such rows, R at a time per block; gridDim.x is a multiple of 8.  g is formed twice:
// the masks leave no registers to keep it in (T = 16384, d = 4081, bf16: 121 us, 136 with g kept)
template <typename T, int NV, int R, int TH>
__global__ void __launch_bounds__(TH + 32, 1)
ln_bwd_shift_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
                    const float* __restrict__ rstd, const T* __restrict__ dy, int64_t Tn, int d, T* __restrict__ dx,
                    float* __restrict__ part, bool late, int slots, Limits lim) {
    constexpr int VEC = Vec16<T>::VEC, HV = VEC / 2;
    extern __shared__ __align__(128) unsigned char smem[];      // slots of R rows of x, then of dy
    __shared__ __align__(8) uint64_t bars[2 * MAX_SLOTS];
    __shared__ int abort_flag;
    __shared__ __align__(16) float buf[128 * R];
    int phase = 0;
    const int nthr = blockDim.x - 32, idx = threadIdx.x;
    if (idx == 0) ring_init(bars, &abort_flag, slots, nthr >> 5);
    __syncthreads();
    pdl_launch_next();
    const StreamOrder order(late);
    Ring ring{bars, &abort_flag, slots, lim};
    const Shifted<T> sx(x, Tn, d, blockIdx.x), sg(dy, Tn, d, blockIdx.x);
    const int64_t step = (int64_t)gridDim.x * R;      // rows row, row + gridDim.x, .. of a batch
    if (idx >= nthr) {
        bool ok = true;
        if (idx == nthr) {
            int left = lim.stop;
            for (int64_t row = blockIdx.x; row < Tn && left != 0; row += step, ring.next(), --left) {
                if (!(ok = ring.wait(ring.empty(), ring.parity ^ 1u))) break;
                uint32_t bytes = 0;
                for (int r = 0; r < R && row + r * gridDim.x < Tn; ++r) bytes += 2 * sx.bytes(row + r * gridDim.x);
                ptx::mbar_arrive_tx(ring.full(), bytes);
                const uint32_t dst = ptx::smem_u32(smem) + ring.s * 2 * R * sx.slot_bytes;
                for (int r = 0; r < R && row + r * gridDim.x < Tn; ++r) {
                    sx.load(row + r * gridDim.x, dst + r * sx.slot_bytes, ring.full());
                    sg.load(row + r * gridDim.x, dst + (R + r) * sx.slot_bytes, ring.full());
                }
            }
            if (!ok) land();
        }
        __syncwarp();
        return;
    }
    const float inv_d = 1.0f / (float)d;
    float2 wv[NV][HV], dw[NV][HV], db[NV][HV];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < HV; ++e) {
            const int c = (v * nthr + idx) * VEC + 2 * e - sx.s;
            wv[v][e].x = w && c >= 0 && c < d ? __ldg(w + c) : 1.f;
            wv[v][e].y = w && c + 1 >= 0 && c + 1 < d ? __ldg(w + c + 1) : 1.f;
            dw[v][e] = db[v][e] = both(0.f);
        }
    const int nw = sx.words(), j_lo = sx.s > 0 ? 1 : 0, j_hi = sx.spare() > 0 ? nw - 1 : nw;      // whole words: j_lo ..
    const int vl = (nw - 1) / nthr;
    const bool last = idx == (nw - 1) % nthr && sx.spare() > 0;
    const uint4 mask0 = sx.mask(idx), mask1 = sx.mask(vl * nthr + idx);
    float mu_n[R], rs_n[R];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t q = row + r * (int64_t)gridDim.x;
            mu_n[r] = q < Tn ? __ldg(mean + q) : 0.f;
            rs_n[r] = q < Tn ? __ldg(rstd + q) : 0.f;
        }
    };
    fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < Tn; row += step, ring.next()) {
        float mu[R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mu[r] = mu_n[r];
            rs[r] = rs_n[r];
        }
        fetch(row + step);
        ring.wait(ring.full(), ring.parity);
        unsigned char* xs = smem + ring.s * 2 * R * sx.slot_bytes;
        if (last) {
#pragma unroll 1
            for (int r = 0; r < R; ++r)
                if (row + r * (int64_t)gridDim.x == Tn - 1) {
                    sx.tail(xs + r * sx.slot_bytes, Tn - 1);
                    sg.tail(xs + (R + r) * sx.slot_bytes, Tn - 1);
                }
        }
        uint4 xr[R][NV], gr[R][NV];
        float2 sa[R], sb[R];                         // sums of g, of g xh
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t q = row + r * (int64_t)gridDim.x;
            sa[r] = sb[r] = both(0.f);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int j = v * nthr + idx;
                xr[r][v] = gr[r][v] = make_uint4(0, 0, 0, 0);
                if (q >= Tn || j >= nw) continue;
                xr[r][v] = *reinterpret_cast<const uint4*>(xs + r * sx.slot_bytes + 16 * j);
                gr[r][v] = *reinterpret_cast<const uint4*>(xs + (R + r) * sx.slot_bytes + 16 * j);
                if (v == 0) {
                    xr[r][v] = masked(xr[r][v], mask0);
                    gr[r][v] = masked(gr[r][v], mask0);
                }
                if (v == vl) {
                    xr[r][v] = masked(xr[r][v], mask1);
                    gr[r][v] = masked(gr[r][v], mask1);
                }
                float2 xf[HV], gf[HV];
                pairs_of(xr[r][v], xf);
                pairs_of(gr[r][v], gf);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 xh = __fmul2_rn(__fadd2_rn(xf[e], both(-mu[r])), both(rs[r]));
                    const float2 g = __fmul2_rn(gf[e], wv[v][e]);
                    dw[v][e] = __ffma2_rn(gf[e], xh, dw[v][e]);
                    db[v][e] = __fadd2_rn(db[v][e], gf[e]);
                    sa[r] = __fadd2_rn(sa[r], g);
                    sb[r] = __ffma2_rn(g, xh, sb[r]);
                }
            }
        }
        float sums[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sums[r] = sa[r].x + sa[r].y;
            sums[R + r] = sb[r].x + sb[r].y;
        }
        __syncwarp();
        if ((idx & 31) == 0) ptx::mbar_arrive(ring.empty());
        if (!dx) continue;
        group_sum<2 * R, 0>(sums, buf, phase, nthr);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t q = row + r * (int64_t)gridDim.x;
            if (q >= Tn) break;
            // dx = rs g w - (rs k) xh - rs a
            const float2 a = both(-rs[r] * (sums[r] * inv_d)), k = both(-rs[r] * (sums[R + r] * inv_d) * rs[r]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int j = v * nthr + idx;
                if (j >= nw) continue;
                float2 xf[HV], gf[HV];
                pairs_of(xr[r][v], xf);
                pairs_of(gr[r][v], gf);
#pragma unroll
                for (int e = 0; e < HV; ++e) {
                    const float2 t = __ffma2_rn(__fadd2_rn(xf[e], both(-mu[r])), k, a);
                    gf[e] = __ffma2_rn(__fmul2_rn(gf[e], wv[v][e]), both(rs[r]), t);
                }
                const uint4 o = vector_of(gf);
                if (j >= j_lo && j < j_hi)
                    st_v4(reinterpret_cast<unsigned char*>(dx) + sx.at(q) + 16 * j, o);
                else
                    sx.store_part(dx, q, j, o);
            }
        }
    }
    if (!part) return;
    float* pw = part + (int64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (v * nthr + idx) * VEC + e - sx.s;
            if (c >= 0 && c < d) {
                pw[c] = e & 1 ? dw[v][e / 2].y : dw[v][e / 2].x;
                pw[d + c] = e & 1 ? db[v][e / 2].y : db[v][e / 2].x;
            }
        }
}

// out[c] = sum over the P blocks of part[p][c], c < 2 d: a block takes 32 columns, its 32 warps a
// strided share of the rows each, eight loads in flight, added in a fixed order
__global__ void __launch_bounds__(1024)
ln_cols_kernel(const float* __restrict__ part, int P, int d, float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float sm[32][33];
    pdl_launch_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane, ld = 2 * (int64_t)d;
    float s = 0.f;
    if (c < ld) {
        for (int p = warp; p < P; p += 256) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = p + 32 * j < P ? __ldcg(part + (int64_t)(p + 32 * j) * ld + c) : 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[j];
        }
    }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < ld) {
#pragma unroll
        for (int k = 1; k < 32; ++k) s += sm[k][lane];
        if (c < d) {
            if (dw) dw[c] = s;
        } else if (db) {
            db[c - d] = s;
        }
    }
}

// dw_c = sum_t dy_c xh_c and db_c = sum_t dy_c straight from the rows: 32 columns per block, a W-th of the
// rows per warp of its first W, four of them in flight, added in a fixed order
template <int W, typename T>
__device__ __forceinline__ void few_columns(const T* __restrict__ x, const float* __restrict__ mean,
                                            const float* __restrict__ rstd, const T* __restrict__ dy, int Tn, int d,
                                            float* __restrict__ dw, float* __restrict__ db, int block) {
    constexpr int U = 4;
    __shared__ float sm[2][W][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp >= W) return;
    const int64_t c = (int64_t)block * 32 + lane;
    float sw = 0.f, sb = 0.f;
    if (c < d) {
        for (int t = warp; t < Tn; t += W * U) {
            float xv[U], gv[U], mu[U], rs[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int64_t row = t + W * j;
                const bool in = row < Tn;
                xv[j] = in ? to_f32(__ldg(x + row * d + c)) : 0.f;
                gv[j] = in ? to_f32(__ldg(dy + row * d + c)) : 0.f;
                mu[j] = in ? __ldg(mean + row) : 0.f;
                rs[j] = in ? __ldg(rstd + row) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                sw = fmaf(gv[j], (xv[j] - mu[j]) * rs[j], sw);
                sb += gv[j];
            }
        }
    }
    sm[0][warp][lane] = sw;
    sm[1][warp][lane] = sb;
    asm volatile("bar.sync 1, %0;" :: "n"(32 * W) : "memory");
    float* const out = warp == 0 ? dw : db;
    if (warp < 2 && c < d && out) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) s += sm[warp][k][lane];
        out[c] = s;
    }
}

template <typename T>
__global__ void __launch_bounds__(1024)
ln_few_cols_kernel(const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
                   const T* __restrict__ dy, int Tn, int d, float* __restrict__ dw, float* __restrict__ db) {
    // in this order: the row kernel that starts early behind this one reads what this one waited for
    pdl_wait();
    pdl_launch_next();
    few_columns<32>(x, mean, rstd, dy, Tn, d, dw, db, blockIdx.x);
}

constexpr int FEW_WARPS = 16;            // of a column block below, and the least of a block

// Both for few rows of up to 1024 vectors, in one launch: the first col_blocks blocks sum columns, the others
// have a row each, one vector per thread of the first nthr.
template <typename T, int VEC>
__global__ void __launch_bounds__(1024)
ln_bwd_few_kernel(const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ mean,
                  const float* __restrict__ rstd, const T* __restrict__ dy, int Tn, int d, T* __restrict__ dx,
                  float* __restrict__ dw, float* __restrict__ db, int col_blocks, int nthr) {
    using P = Pack<T, VEC>;
    __shared__ float buf[64 * 2];
    pdl_launch_next();
    pdl_wait();
    if ((int)blockIdx.x < col_blocks) {
        few_columns<FEW_WARPS>(x, mean, rstd, dy, Tn, d, dw, db, blockIdx.x);
        return;
    }
    if ((int)threadIdx.x >= nthr) return;
    const int64_t row = blockIdx.x - col_blocks;
    const int c = threadIdx.x * VEC;
    const bool in = c < d;
    const typename P::raw xr = in ? P::load(x + row * d + c) : P::zero(), gr = in ? P::load(dy + row * d + c) : P::zero();
    const float mu = __ldg(mean + row), rs = __ldg(rstd + row), inv_d = 1.0f / (float)d;
    float xh[VEC], g[VEC], sums[2] = {0.f, 0.f};       // of g, of g xh; columns past d have dy = 0
    P::unpack(xr, xh);
    P::unpack(gr, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        xh[e] = (xh[e] - mu) * rs;
        g[e] *= w && in ? __ldg(w + c + e) : 1.f;
        sums[0] += g[e];
        sums[1] = fmaf(g[e], xh[e], sums[1]);
    }
    int phase = 0;
    group_sum<2, 0>(sums, buf, phase, nthr);
    const float a = sums[0] * inv_d, k = sums[1] * inv_d;
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] = rs * ((g[e] - a) - xh[e] * k);
    if (in) P::store(dx + row * d + c, g);
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
    if (cap > bwd_blocks(a.d)) cap = bwd_blocks(a.d);
    *blocks = (int)(want < cap ? want : cap);
    return launch_pdl(kern, dim3((unsigned)*blocks), dim3(threads), smem, a.stream, static_cast<const T*>(a.x), a.w,
                      a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d, static_cast<T*>(a.dx), a.part, a.late);
}

std::atomic<unsigned long long> g_wait_ns{1000000000ull};      // 1 s per wait
std::atomic<int> g_stop{-1};

Limits limits() { return Limits{g_wait_ns.load(), g_stop.load()}; }

// Shared memory of an SM that the blocks of a ring kernel split among them
constexpr int ROOM = 204800;

// The same limit at every launch, whatever the launch takes of it: another host thread may be launching the
// kernel for other rows.
template <typename K>
cudaError_t allow_room(K kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ROOM);
}

// Launch shape of a ring kernel: threads, rows per slot, and slots.  The SM's shared memory goes to
// about 640 threads' worth of blocks.
struct RingShape {
    int threads, B, slots;
    size_t bytes;
};

template <typename T>
RingShape ring_shape(int d, int nv, int r, int g, int tensors) {
    RingShape s{};
    const int chunks = d / Vec16<T>::VEC, consumers = g ? 32 * WARPS : ((chunks + nv - 1) / nv + 31) / 32 * 32;
    const int blocks = consumers >= 320 ? 3 : consumers <= 64 ? 10 : 640 / consumers;
    s.threads = consumers + 32;
    s.B = g ? WARPS * (32 / g) * r : r;
    const size_t slot = (size_t)tensors * s.B * d * sizeof(T);
    s.slots = (int)(ROOM / blocks / slot);
    s.slots = s.slots < 2 ? 2 : s.slots > MAX_SLOTS ? MAX_SLOTS : s.slots;
    s.bytes = s.slots * slot;
    return s;
}

template <typename T, int NV, int R, int G, int TH>
cudaError_t fwd_ring(const LnArgs& a) {
    const RingShape r = ring_shape<T>(a.d, NV, R, G, 1);
    auto kern = ln_fwd_ring_kernel<T, NV, R, G, TH>;
    cudaError_t e = allow_room(kern);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.T + r.B - 1) / r.B;
    int cap;
    e = resident(kern, r.threads, r.bytes, want, &cap);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(want < cap ? want : cap)), dim3(r.threads), r.bytes, a.stream,
                      static_cast<const T*>(a.x), a.w, a.b, a.T, a.d, a.eps, static_cast<T*>(a.y), a.mean, a.rstd,
                      r.slots, limits());
}

template <typename T, int NV, int R, int G, int TH>
cudaError_t bwd_ring(const LnArgs& a, int* blocks) {
    const RingShape r = ring_shape<T>(a.d, NV, R, G, 2);
    auto kern = ln_bwd_ring_kernel<T, NV, R, G, TH>;
    cudaError_t e = allow_room(kern);
    if (e != cudaSuccess) return e;
    // four rows per block at least: a block's column sums cost as much traffic as its first two rows
    const int64_t batches = (a.T + r.B - 1) / r.B, want = r.B >= 4 ? batches : (batches * r.B + 3) / 4;
    int cap;
    e = resident(kern, r.threads, r.bytes, want, &cap);
    if (e != cudaSuccess) return e;
    if (cap > bwd_blocks(a.d)) cap = bwd_blocks(a.d);
    *blocks = (int)(want < cap ? want : cap);
    return launch_pdl(kern, dim3((unsigned)*blocks), dim3(r.threads), r.bytes, a.stream, static_cast<const T*>(a.x),
                      a.w, a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d, static_cast<T*>(a.dx), a.part,
                      a.late, r.slots, limits());
}

template <typename T, int NV>
cudaError_t fwd_warp(const LnArgs& a) {
    constexpr int TH = 256;
    auto kern = ln_fwd_warp_kernel<T, NV>;
    // the SM's shared memory in equal parts
    const size_t wb = (size_t)2 * NV * 32 * Vec16<T>::VEC * 4, slot = (size_t)(TH / 32) * a.d * sizeof(T);
    int slots = (int)((ROOM / WARP_BLOCKS<T, NV> - wb) / slot);
    slots = slots < 1 ? 1 : slots > WARP_SLOTS ? WARP_SLOTS : slots;
    const size_t smem = wb + slots * slot;
    cudaError_t e = allow_room(kern);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.T + TH / 32 - 1) / (TH / 32);
    int cap;
    e = resident(kern, TH, smem, want, &cap);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((unsigned)(want < cap ? want : cap)), dim3(TH), smem, a.stream,
                      static_cast<const T*>(a.x), a.w, a.b, a.T, a.d, a.eps, static_cast<T*>(a.y), a.mean, a.rstd, slots,
                      limits());
}

template <typename T, int NV>
cudaError_t fwd_shift(const LnArgs& a) {
    constexpr int TH = 256;
    auto kern = ln_fwd_shift_kernel<T, NV>;
    const size_t wb = (size_t)2 * NV * 32 * Vec16<T>::VEC * 4;
    const size_t slot = (size_t)(TH / 32) * ((a.d * sizeof(T) + 15) / 16 * 16 + 16);
    int slots = (int)((ROOM / WARP_BLOCKS<T, NV> - wb) / slot);
    slots = slots < 1 ? 1 : slots > WARP_SLOTS ? WARP_SLOTS : slots;
    const size_t smem = wb + slots * slot;
    cudaError_t e = allow_room(kern);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.T + TH / 32 - 1) / (TH / 32);
    int cap;
    e = resident(kern, TH, smem, want, &cap);
    if (e != cudaSuccess) return e;
    const int blocks = (int)(want < cap ? want : cap) / 8 * 8;      // at least 16 rows per SM: never 0
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(TH), smem, a.stream,
                      static_cast<const T*>(a.x), a.w, a.b, a.T, a.d, a.eps, static_cast<T*>(a.y), a.mean, a.rstd, slots,
                      limits());
}

template <typename T, int NV, int R, int TH>
cudaError_t bwd_shift(const LnArgs& a, int* blocks) {
    constexpr int VEC = Vec16<T>::VEC;
    auto kern = ln_bwd_shift_kernel<T, NV, R, TH>;
    const int words = (a.d + 2 * VEC - 2) / VEC, nthr = ((words + NV - 1) / NV + 31) / 32 * 32;
    const size_t slot = (size_t)2 * R * ((a.d * sizeof(T) + 15) / 16 * 16 + 16);
    int slots = (int)(ROOM / (nthr >= 320 ? 2 : nthr <= 64 ? 10 : 640 / nthr) / slot);
    slots = slots < 2 ? 2 : slots > MAX_SLOTS ? MAX_SLOTS : slots;
    cudaError_t e = allow_room(kern);
    if (e != cudaSuccess) return e;
    const int64_t want = (a.T + 3) / 4;
    int cap;
    e = resident(kern, nthr + 32, slots * slot, want, &cap);
    if (e != cudaSuccess) return e;
    if (cap > bwd_blocks(a.d)) cap = bwd_blocks(a.d);
    *blocks = (int)(want < cap ? want : cap) / 8 * 8;       // at least 16 rows per SM: never 0
    return launch_pdl(kern, dim3((unsigned)*blocks), dim3(nthr + 32), slots * slot, a.stream, static_cast<const T*>(a.x),
                      a.w, a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d, static_cast<T*>(a.dx), a.part,
                      a.late, slots, limits());
}

// The layout of a row by its length in vectors: 8, 16 or 32 lanes with one vector each, 32 with two, a
// warp with up to 16, a block with more.  What a block's row costs is the time between its load and its
// store, which other warps have to cover: several small blocks per SM, or one of ten warps and more whose
// threads hold few registers each.  Measured, us, T = 8192, vectors per thread and rows at a time: bf16, d = 6000
// 4 and one 49 (2 and two: 58; 4 and two: 61), d = 8192 4 and two 60 (2 and two: 69, 4 and one: 73); fp32, d =
// 5000 8 and one 54 (6 and two: 66, 4 and one: 86), d = 7400 6 and two 80 (8 and one: 85, 4 and one: 98), d =
// 3328 (T = 16384) 4 and two 81 (2 and two: 98).  Up to 224 threads two blocks fit if a thread holds 128 registers
// at most (bf16, d = 6000: 76 with 136; fp32, T = 1000, d = 5376: 10.2 and 11.3).  At most one row per SM takes a
// register kernel.
// Rows that are not a multiple of 16 bytes take the shift kernels from 16 rows per SM on.  T = 16384,
// bf16: d = 4095 67 us against 137 one element at a time, d = 2559 49 against 89; fp32, d = 2559 71 against 76.
// With fewer rows filling the ring costs more than it hides: T = 1200, d = 1037, bf16 7.4 against 5.8 us, T = 2400
// 7.9 against 9.4.
template <typename T>
cudaError_t fwd_t(const LnArgs& a, int sms) {
    constexpr int V = Vec16<T>::VEC;
    if (a.d % V == 0 && rows16(a.x) && rows16(a.y)) {
        const int c = a.d / V;
        if (c <= 1024 && a.T <= sms) return fwd<T, V, 1, 1, false>(a);
        constexpr int W = 32 * WARPS;
        if (c <= 8) return fwd_ring<T, 1, 2, 8, W>(a);
        if (c <= 16) return fwd_ring<T, 1, 2, 16, W>(a);
        if (c <= 32) return fwd_ring<T, 1, 2, 32, W>(a);
        if (c <= 64) return fwd_ring<T, 2, 2, 32, W>(a);
        if (c <= 128) return fwd_warp<T, 4>(a);
        if (c <= 192) return fwd_warp<T, 6>(a);
        if (c <= 256) return fwd_warp<T, 8>(a);
        if (c <= 320) return fwd_warp<T, 10>(a);
        if (c <= 384) return fwd_warp<T, 12>(a);
        if (c <= 512) return fwd_warp<T, 16>(a);
        if (c <= 896) return fwd_ring<T, 4, V == 8 ? 1 : 2, 0, 224>(a);
        if (c <= 1024) return fwd_ring<T, 4, 2, 0, 256>(a);
        if constexpr (V == 4) {
            if (c <= 1280) return fwd_ring<T, 8, 1, 0, 256>(a);
            if (c <= 1344) return fwd_ring<T, 6, 2, 0, 224>(a);
            if (c <= 2048) return fwd_ring<T, 6, 2, 0, 352>(a);
        } else {
            if (c <= 2048) return fwd_ring<T, 4, 1, 0, 512>(a);
        }
    } else {
        // vectors that the words around a row may take
        const int c = ((int)sizeof(T) * a.d + 30) / 16;
        if (a.T >= 16 * sms && a.d > 256 && c <= 1026 && rows16(a.x) && rows16(a.y)) {
            if (c <= 128) return fwd_shift<T, 4>(a);
            if (c <= 192) return fwd_shift<T, 6>(a);
            if (c <= 256) return fwd_shift<T, 8>(a);
            if (c <= 320) return fwd_shift<T, 10>(a);
            if (c <= 384) return fwd_shift<T, 12>(a);
            if (c <= 544) return fwd_shift<T, 17>(a);
            if (c <= 768) return fwd_shift<T, 24>(a);
            return fwd_shift<T, 33>(a);          // eight rows and the columns' w and b fill the SM's shared memory
        }
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

// *done: the backward as one launch (ONE_LAUNCH_ROWS), for rows of up to 1024 vectors, or unaligned elements
template <typename T>
cudaError_t bwd_few(const LnArgs& a, bool aligned, bool* done) {
    constexpr int V = Vec16<T>::VEC;
    const bool vec = aligned && a.d % V == 0;
    if (a.d > (vec ? 1024 * V : 1024)) return cudaSuccess;
    *done = true;
    const int nthr = ((vec ? a.d / V : a.d) + 31) / 32 * 32, threads = nthr > 32 * FEW_WARPS ? nthr : 32 * FEW_WARPS;
    const int cols = a.part ? (a.d + 31) / 32 : 0, rows = a.dx ? (int)a.T : 0;
    return launch_pdl(vec ? ln_bwd_few_kernel<T, V> : ln_bwd_few_kernel<T, 1>, dim3((unsigned)(cols + rows)),
                      dim3((unsigned)threads), 0, a.stream, static_cast<const T*>(a.x), a.w, a.mean, a.rstd,
                      static_cast<const T*>(a.dy), (int)a.T, a.d, static_cast<T*>(a.dx), a.dw, a.db, cols, nthr);
}

// As forward, but a block has two vectors per thread and two rows at a time up to 512 vectors, and three
// (fp32, above 1024: six) and one above.  Measured, us, x and dy apart: T = 8192, d = 8192, bf16 78 (142 with two
// and one); fp32 140 (176 with four and one).  320 to 480 vectors: three and one, because two need six warps or
// more, whose registers leave room for one block per SM only (T = 16384, bf16, d = 2816: 60 against 72, d = 3584:
// 71 against 74; d = 4096 needs six warps either way: 77 with two and two, 109 with three and one).
// Rows that are not a multiple of 16 bytes, T = 16384, against one element at a time: bf16, d = 2559 86 and 104,
// d = 3585 101 and 157, d = 4609 two and two 138 (three and one: 175) and 283, d = 5633 three and one 173 and 302
// (at T = 7101 83, two and two 112); fp32, d = 2305 four and one 85 (three and one: 133) and 109, d = 3585 147 and
// 170.  With few rows the elements gain: T = 2400, bf16, d = 2559 24 and 20, d = 4609 30 and 38.
template <typename T>
cudaError_t bwd_t(const LnArgs& a, int sms, int* blocks) {
    constexpr int V = Vec16<T>::VEC;
    if (a.d % V == 0 && rows16(a.x) && rows16(a.dy) && rows16(a.dx)) {
        const int c = a.d / V;
        constexpr int W = 32 * WARPS;
        if (c <= 8) return bwd_ring<T, 1, 2, 8, W>(a, blocks);
        if (c <= 16) return bwd_ring<T, 1, 2, 16, W>(a, blocks);
        if (c <= 32) return bwd_ring<T, 1, 2, 32, W>(a, blocks);
        if (c <= 64) return bwd_ring<T, 2, 1, 32, W>(a, blocks);
        if (c > 320 && c <= 480) return bwd_ring<T, 3, 1, 0, 256>(a, blocks);
        if (c <= 512) return bwd_ring<T, 2, 2, 0, 256>(a, blocks);
        if (c <= 1024) return bwd_ring<T, 3, 1, 0, 352>(a, blocks);
        if constexpr (V == 4) {
            if (c <= 2048) return bwd_ring<T, 6, 1, 0, 352>(a, blocks);
        }
    } else {
        const int c = ((int)sizeof(T) * a.d + 30) / 16;
        if (a.T >= 16 * sms && a.d > 256 && c <= 1024 && rows16(a.x) && rows16(a.dy) && rows16(a.dx)) {
            if (c > 320 && c <= 480) return bwd_shift<T, 3, 1, 256>(a, blocks);
            if (c <= (V == 8 ? 480 : 512)) return bwd_shift<T, 2, 2, 256>(a, blocks);
            if constexpr (V == 8) {
                if (c <= 640) return bwd_shift<T, 2, 2, 320>(a, blocks);
            } else {
                if (c <= 640) return bwd_shift<T, 4, 1, 256>(a, blocks);
            }
            return bwd_shift<T, 3, 1, 352>(a, blocks);
        }
        if (a.d <= 256) return bwd<T, 1, 8, 1, true>(a, blocks);
        if (a.d <= 4096) return bwd<T, 1, 8, 1, false>(a, blocks);
        if (a.d <= 8192) return bwd<T, 1, 16, 1, false>(a, blocks);
    }
    int cap;
    cudaError_t e = resident(ln_bwd_long_kernel<T>, 1024, 0, a.T, &cap);
    if (e != cudaSuccess) return e;
    if (cap > bwd_blocks(a.d)) cap = bwd_blocks(a.d);
    *blocks = (int)(a.T < cap ? a.T : cap);
    return launch_pdl(ln_bwd_long_kernel<T>, dim3((unsigned)*blocks), dim3(1024), 0, a.stream,
                      static_cast<const T*>(a.x), a.w, a.mean, a.rstd, static_cast<const T*>(a.dy), a.T, a.d,
                      static_cast<T*>(a.dx), a.part, a.late);
}

}  // namespace

int64_t layer_norm_part_floats(int64_t T, int d) {
    const int64_t p = T < bwd_blocks(d) ? T : bwd_blocks(d);
    return p * 2 * d;
}

cudaError_t launch_layer_norm(const LnArgs& a) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    return a.dt == BF16 ? fwd_t<__nv_bfloat16>(a, di.sm_count) : fwd_t<float>(a, di.sm_count);
}

cudaError_t launch_layer_norm_backward(const LnArgs& args) {
    DeviceInfo di;
    cudaError_t e = device_info(&di);
    if (e != cudaSuccess) return e;
    LnArgs a = args;
    if (a.T <= ONE_LAUNCH_ROWS) {
        const bool vec = rows16(a.x) && rows16(a.dy) && rows16(a.dx);
        bool done = false;
        e = a.dt == BF16 ? bwd_few<__nv_bfloat16>(a, vec, &done) : bwd_few<float>(a, vec, &done);
        if (e != cudaSuccess || done) return e;
    }
    a.late = a.part && a.T <= FEW_ROWS;
    if (a.late) {
        const dim3 grid((unsigned)(((int64_t)a.d + 31) / 32));
        e = a.dt == BF16 ? launch_pdl(ln_few_cols_kernel<__nv_bfloat16>, grid, dim3(1024), 0, a.stream,
                                      static_cast<const __nv_bfloat16*>(a.x), a.mean, a.rstd,
                                      static_cast<const __nv_bfloat16*>(a.dy), (int)a.T, a.d, a.dw, a.db)
                         : launch_pdl(ln_few_cols_kernel<float>, grid, dim3(1024), 0, a.stream,
                                      static_cast<const float*>(a.x), a.mean, a.rstd,
                                      static_cast<const float*>(a.dy), (int)a.T, a.d, a.dw, a.db);
        a.part = nullptr;
        if (e != cudaSuccess || !a.dx) return e;
    }
    int blocks = 0;
    e = a.dt == BF16 ? bwd_t<__nv_bfloat16>(a, di.sm_count, &blocks) : bwd_t<float>(a, di.sm_count, &blocks);
    if (e != cudaSuccess || !a.part) return e;
    const unsigned grid = (unsigned)((2 * (int64_t)a.d + 31) / 32);
    return launch_pdl(ln_cols_kernel, dim3(grid), dim3(1024), 0, a.stream, a.part, blocks, a.d, a.dw, a.db);
}

void layer_norm_set_stop(int stop, unsigned long long wait_ns) {
    g_stop.store(stop);
    g_wait_ns.store(wait_ns);
}

cudaError_t layer_norm_status(unsigned* out, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(out, g_layer_norm_status, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    if (clear && *out) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_layer_norm_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace mhc
