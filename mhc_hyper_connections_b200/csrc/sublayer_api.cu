// sublayer_api.cu -- the C ABI of the sub-layer operators (layer norm, the linear product):
// host-side validation and dispatch.  As in mhc_api.cu, every argument is checked on the host
// before anything is launched, and a rejected call launches nothing.
#include "launch.cuh"
#include "mhc.h"

namespace mhc {
mhc_status report_cuda_error(cudaError_t e, const char* where);
}

using namespace mhc;

namespace {

struct Span {
    const void* p;
    size_t bytes;
};

bool overlaps(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// no output may overlap an input or another output
template <int NI, int NO>
bool aliased(const Span (&in)[NI], const Span (&out)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlaps(out[o], in[i])) return true;
        for (int p = o + 1; p < NO; ++p)
            if (overlaps(out[o], out[p])) return true;
    }
    return false;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
size_t elem_size(mhc_dtype dt) { return dt == MHC_BF16 ? 2 : 4; }
DType dtype_of(mhc_dtype dt) { return dt == MHC_BF16 ? BF16 : F32; }
bool known(mhc_dtype dt) { return dt == MHC_F32 || dt == MHC_BF16; }

constexpr int kMaxDim = 1 << 30;

// T rows of `width` elements: byte counts stay below 2^62
bool rows_ok(int64_t T, int64_t width) {
    return T >= 0 && width >= 1 && width <= kMaxDim && T <= ((int64_t)1 << 62) / (width * 8);
}

mhc_status check_linear(int64_t T, int K, int N, mhc_dtype dt) {
    if (!known(dt)) return MHC_ERR_DTYPE;
    if (!rows_ok(T, K) || !rows_ok(T, N)) return MHC_ERR_SHAPE;
    return MHC_OK;
}

bool known(mhc_act act) { return act >= MHC_ACT_NONE && act <= MHC_ACT_SILU; }

}  // namespace

extern "C" {

mhc_status mhc_layer_norm(const void* x, const float* weight, const float* bias, int64_t T, int d, float eps,
                          mhc_dtype dt, void* y, float* mean, float* rstd, mhc_stream_t stream) {
    if (!known(dt)) return MHC_ERR_DTYPE;
    if (!rows_ok(T, d)) return MHC_ERR_SHAPE;
    if (T == 0) return MHC_OK;
    if (!x || !y || !mean != !rstd) return MHC_ERR_NULL;
    const size_t es = elem_size(dt), nx = (size_t)T * d * es;
    if (!aligned(x, es) || !aligned(y, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return MHC_ERR_ALIGN;
    const Span in[3] = {{x, nx}, {weight, (size_t)d * 4}, {bias, (size_t)d * 4}};
    const Span out[3] = {{y, nx}, {mean, (size_t)T * 4}, {rstd, (size_t)T * 4}};
    if (aliased(in, out)) return MHC_ERR_ALIAS;
    LnArgs a{};
    a.x = x; a.w = weight; a.b = bias; a.T = T; a.d = d; a.eps = eps; a.dt = dtype_of(dt);
    a.y = y; a.mean = mean; a.rstd = rstd;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_layer_norm(a);
    return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_layer_norm");
}

size_t mhc_layer_norm_backward_workspace_bytes(int64_t T, int d) {
    return rows_ok(T, d) ? (size_t)layer_norm_part_floats(T, d) * 4 : 0;
}

mhc_status mhc_layer_norm_backward(const void* x, const float* weight, const float* mean, const float* rstd,
                                   int64_t T, int d, mhc_dtype dt, const void* dy, void* dx, float* dweight,
                                   float* dbias, void* workspace, size_t workspace_bytes, mhc_stream_t stream) {
    if (!known(dt)) return MHC_ERR_DTYPE;
    if (!rows_ok(T, d)) return MHC_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: the parameter gradients are zero
        cudaError_t e = cudaSuccess;
        if (!aligned(dweight, 4) || !aligned(dbias, 4)) return MHC_ERR_ALIGN;
        if (overlaps({dweight, (size_t)d * 4}, {dbias, (size_t)d * 4})) return MHC_ERR_ALIAS;
        if (dweight) e = cudaMemsetAsync(dweight, 0, (size_t)d * 4, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, (size_t)d * 4, s);
        return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_layer_norm_backward");
    }
    const bool params = dweight || dbias;
    if (!x || !mean || !rstd || !dy || (params && !workspace)) return MHC_ERR_NULL;
    const size_t es = elem_size(dt), nx = (size_t)T * d * es, nd = (size_t)d * 4, nt = (size_t)T * 4;
    if (!aligned(x, es) || !aligned(dy, es) || !aligned(dx, es) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || (params && !aligned(workspace, 256)))
        return MHC_ERR_ALIGN;
    const size_t need = params ? mhc_layer_norm_backward_workspace_bytes(T, d) : 0;
    if (params && workspace_bytes < need) return MHC_ERR_WORKSPACE;
    const Span in[5] = {{x, nx}, {weight, nd}, {mean, nt}, {rstd, nt}, {dy, nx}};
    const Span out[4] = {{dx, nx}, {dweight, nd}, {dbias, nd}, {workspace, need}};
    if (aliased(in, out)) return MHC_ERR_ALIAS;
    if (!dx && !params) return MHC_OK;
    LnArgs a{};
    a.x = x; a.w = weight; a.T = T; a.d = d; a.dt = dtype_of(dt);
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dy = dy; a.dx = dx; a.dw = dweight; a.db = dbias;
    a.part = params ? static_cast<float*>(workspace) : nullptr;
    a.stream = s;
    const cudaError_t e = launch_layer_norm_backward(a);
    return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_layer_norm_backward");
}

size_t mhc_linear_workspace_bytes(int64_t T, int K, int N, mhc_dtype dt) {
    return check_linear(T, K, N, dt) == MHC_OK && T > 0 ? linear_workspace(T, K, N, dtype_of(dt)) : 0;
}

mhc_status mhc_linear(const void* x, const void* W, const float* bias, const void* residual, int64_t T, int K,
                      int N, mhc_act act, mhc_dtype dt, void* y, void* z, void* workspace,
                      size_t workspace_bytes, mhc_stream_t stream) {
    const mhc_status st = check_linear(T, K, N, dt);
    if (st != MHC_OK) return st;
    if (!known(act)) return MHC_ERR_UNSUPPORTED;
    if (T == 0) return MHC_OK;
    const size_t need = mhc_linear_workspace_bytes(T, K, N, dt);
    if (!x || !W || !y || (need && !workspace)) return MHC_ERR_NULL;
    const size_t es = elem_size(dt), nx = (size_t)T * K * es, nw = (size_t)N * K * es, ny = (size_t)T * N * es;
    if (!aligned(x, es) || !aligned(W, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(z, es) ||
        !aligned(bias, 4) || (need && !aligned(workspace, 256)))
        return MHC_ERR_ALIGN;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    const Span in[4] = {{x, nx}, {W, nw}, {bias, (size_t)N * 4}, {residual, ny}};
    const Span out[3] = {{y, ny}, {z, ny}, {workspace, need}};
    if (aliased(in, out)) return MHC_ERR_ALIAS;
    LinearArgs a{};
    a.x = x; a.W = W; a.bias = bias; a.residual = residual; a.T = T; a.K = K; a.N = N;
    a.act = (Act)act; a.dt = dtype_of(dt); a.y = y; a.z = z; a.workspace = workspace;
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_linear(a);
    return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_linear");
}

size_t mhc_linear_backward_workspace_bytes(int64_t T, int K, int N, mhc_dtype dt) {
    return check_linear(T, K, N, dt) == MHC_OK && T > 0 ? linear_backward_workspace(T, K, N, dtype_of(dt)) : 0;
}

mhc_status mhc_linear_backward(const void* x, const void* W, const void* z, int64_t T, int K, int N, mhc_act act,
                               mhc_dtype dt, const void* dy, void* dx, void* dW, float* dbias, void* workspace,
                               size_t workspace_bytes, mhc_stream_t stream) {
    const mhc_status st = check_linear(T, K, N, dt);
    if (st != MHC_OK) return st;
    if (!known(act)) return MHC_ERR_UNSUPPORTED;
    const size_t es = elem_size(dt), nx = (size_t)T * K * es, nw = (size_t)N * K * es, ny = (size_t)T * N * es;
    const size_t nb = (size_t)N * 4;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: the parameter gradients are zero
        cudaError_t e = cudaSuccess;
        if (!aligned(dW, es) || !aligned(dbias, 4)) return MHC_ERR_ALIGN;
        if (overlaps({dW, nw}, {dbias, nb})) return MHC_ERR_ALIAS;
        if (dW) e = cudaMemsetAsync(dW, 0, nw, s);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, nb, s);
        return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_linear_backward");
    }
    if (act == MHC_ACT_NONE) z = nullptr;
    if (!dy || (dx && !W) || (dW && !x) || (act != MHC_ACT_NONE && !z) || !workspace) return MHC_ERR_NULL;
    if (!aligned(x, es) || !aligned(W, es) || !aligned(z, es) || !aligned(dy, es) || !aligned(dx, es) ||
        !aligned(dW, es) || !aligned(dbias, 4) || !aligned(workspace, 256))
        return MHC_ERR_ALIGN;
    const size_t need = mhc_linear_backward_workspace_bytes(T, K, N, dt);
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    const Span in[4] = {{x, nx}, {W, nw}, {z, ny}, {dy, ny}};
    const Span out[4] = {{dx, nx}, {dW, nw}, {dbias, nb}, {workspace, need}};
    if (aliased(in, out)) return MHC_ERR_ALIAS;
    LinearArgs a{};
    a.x = x; a.W = W; a.z = const_cast<void*>(z); a.T = T; a.K = K; a.N = N; a.act = (Act)act;
    a.dt = dtype_of(dt); a.dy = dy; a.dx = dx; a.dW = dW; a.dbias = dbias; a.workspace = workspace;
    a.stream = s;
    const cudaError_t e = launch_linear_backward(a);
    return e == cudaSuccess ? MHC_OK : report_cuda_error(e, "mhc_linear_backward");
}

mhc_status mhc_debug_sublayer_stop_after(int32_t stages, uint32_t wait_limit_us) {
    if (wait_limit_us < 1000u || wait_limit_us > 10000000u) return MHC_ERR_SHAPE;
    const int stop = stages < 0 ? -1 : (int)stages;
    layer_norm_set_stop(stop, (unsigned long long)wait_limit_us * 1000ull);
    linear_tc_set_stop(stop, (unsigned long long)wait_limit_us * 1000ull);
    return MHC_OK;
}

}  // extern "C"
