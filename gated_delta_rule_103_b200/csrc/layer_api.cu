// C ABI of the layer operators around the recurrences: the short causal
// convolution, the state-space scan and the group norm.  Argument validation
// and dispatch; include/kda.h has the contract.
#include "arg_check.h"
#include "layer.h"

namespace {

using kda::device_ptr_ok;
using kda::elem_size;
using kda::overlaps;
using kda::Region;
using kda::workspace_ok;

// The call's tensors as they are checked: every one that holds anything must
// be valid device memory, and an output may share memory with no other tensor.
class Tensors {
public:
    // A tensor of n bytes; an optional one may be null.
    void in(const void* p, size_t n, bool optional = false) { add(p, n, optional, false); }
    void out(const void* p, size_t n, bool optional = false) { add(p, n, optional, true); }
    // The state read and then written in place: one tensor.
    void in_out_state(const void* init, void* fin, size_t n)
    {
        if (fin && fin == init) {
            add(fin, n, false, true);
        } else {
            add(init, n, true, false);
            add(fin, n, true, true);
        }
    }
    bool ok() const
    {
        if (!ok_) return false;
        for (int i = 0; i < n_; ++i)
            for (int j = i + 1; j < n_; ++j)
                if ((written_[i] || written_[j]) && overlaps(r_[i].p, r_[i].n, r_[j].p, r_[j].n)) return false;
        return true;
    }
    bool workspace(const void* ws, size_t bytes, size_t need) const { return workspace_ok(ws, bytes, need, r_, n_); }

private:
    void add(const void* p, size_t n, bool optional, bool written)
    {
        if (!p && (optional || n == 0)) return;
        if (n == 0) return;  // nothing is read or written there
        if (dev_ < 0 && cudaGetDevice(&dev_) != cudaSuccess) ok_ = false;
        if (!device_ptr_ok(p, dev_)) ok_ = false;
        r_[n_] = {p, n};
        written_[n_++] = written;
    }
    Region r_[24];
    bool written_[24];
    int n_ = 0, dev_ = -1;
    bool ok_ = true;
};

constexpr size_t kMostTokens = (size_t)1 << 30;  // and sequences
constexpr int kMostChannels = 1 << 24;

// Sizes that every call over sequences shares; KDA_OK: go on.
kda_status check_sizes(int B, int T, int C, int N, const void* cu, kda_dtype dtype)
{
    if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || C <= 0 || N < 0) return KDA_ERR_INVALID_ARG;
    if (cu) {
        if (B != 1 || (N == 0 && T > 0)) return KDA_ERR_INVALID_ARG;
    } else if (N != B) {
        return KDA_ERR_INVALID_ARG;
    }
    if ((size_t)B * (size_t)T > kMostTokens || (size_t)N > kMostTokens || C > kMostChannels)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// A launcher answers cudaErrorInvalidConfiguration, before it has enqueued
// anything, where a call would take more blocks than a grid has.
kda_status status_of(cudaError_t e)
{
    if (e == cudaSuccess) return KDA_OK;
    return e == cudaErrorInvalidConfiguration ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

kda_status check_conv(int W, unsigned flags)
{
    if (flags & ~(unsigned)KDA_FLAG_SILU) return KDA_ERR_UNSUPPORTED;
    if (W <= 0) return KDA_ERR_INVALID_ARG;
    return W >= 2 && W <= 4 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status check_scan(int D, int S, int G, unsigned flags)
{
    if (flags & ~(unsigned)KDA_FLAG_SOFTPLUS) return KDA_ERR_UNSUPPORTED;
    if (S <= 0 || G <= 0 || D % G != 0) return KDA_ERR_INVALID_ARG;
    return S <= 128 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

bool sizes_ok(int B, int T, int C, int N, int packed)
{
    return B >= 0 && T >= 0 && C > 0 && N >= 0 && (packed ? B == 1 && !(N == 0 && T > 0) : N == B) &&
           (size_t)B * (size_t)T <= kMostTokens && (size_t)N <= kMostTokens && C <= kMostChannels;
}

bool dtype_ok(kda_dtype d) { return d == KDA_DTYPE_F32 || d == KDA_DTYPE_BF16; }

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                              const int32_t* cu_seqlens, void* out, void* final_state, int B, int T, int C, int W,
                              int N, kda_dtype dtype, unsigned flags, cudaStream_t stream)
{
    if (kda_status s = check_sizes(B, T, C, N, cu_seqlens, dtype)) return s;
    if (kda_status s = check_conv(W, flags)) return s;
    const size_t es = elem_size(dtype), n_x = (size_t)B * T * C * es, n_s = (size_t)N * (W - 1) * C * es;
    Tensors t;
    t.in(x, n_x);
    t.in(weight, (size_t)C * W * 4);
    t.in(bias, (size_t)C * 4, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.in_out_state(initial_state, final_state, n_s);
    t.out(out, n_x);
    if (!t.ok()) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.initial_state = initial_state; a.cu_seqlens = cu_seqlens;
    a.out = out; a.final_state = final_state;
    a.B = B; a.T = T; a.C = C; a.W = W; a.N = N; a.silu = (flags & KDA_FLAG_SILU) != 0;
    return status_of(kda::launch_conv_fwd(a, dtype, stream));
}

kda_status kda_short_conv_step(const void* x, const float* weight, const float* bias, void* state, void* out, int N,
                               int C, int W, kda_dtype dtype, unsigned flags, cudaStream_t stream)
{
    if (kda_status s = check_sizes(N, 1, C, N, nullptr, dtype)) return s;
    if (kda_status s = check_conv(W, flags)) return s;
    if (N == 0) return KDA_OK;
    const size_t es = elem_size(dtype), n_x = (size_t)N * C * es;
    Tensors t;
    t.in(x, n_x);
    t.in(weight, (size_t)C * W * 4);
    t.in(bias, (size_t)C * 4, true);
    t.out(state, n_x * (W - 1));
    t.out(out, n_x);
    if (!t.ok()) return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.final_state = state; a.out = out;
    a.C = C; a.W = W; a.N = N; a.silu = (flags & KDA_FLAG_SILU) != 0;
    return status_of(kda::launch_conv_step(a, dtype, stream));
}

size_t kda_short_conv_bwd_workspace_bytes(int B, int T, int C, int W, int N, int packed, kda_dtype dtype)
{
    if (!sizes_ok(B, T, C, N, packed) || !dtype_ok(dtype) || W < 2 || W > 4) return 0;
    return kda::conv_bwd_workspace(B, T, C, W, N, dtype);
}

kda_status kda_short_conv_bwd(const void* x, const float* weight, const float* bias, const void* initial_state,
                              const int32_t* cu_seqlens, const void* d_out, const float* d_final_state,
                              float* grad_x, float* grad_weight, float* grad_bias, float* grad_initial_state, int B,
                              int T, int C, int W, int N, kda_dtype dtype, unsigned flags, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream)
{
    if (kda_status s = check_sizes(B, T, C, N, cu_seqlens, dtype)) return s;
    if (kda_status s = check_conv(W, flags)) return s;
    const size_t es = elem_size(dtype), n_x = (size_t)B * T * C, n_s = (size_t)N * (W - 1) * C;
    Tensors t;
    t.in(x, n_x * es);
    t.in(weight, (size_t)C * W * 4);
    t.in(bias, (size_t)C * 4, true);
    t.in(initial_state, n_s * es, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.in(d_out, n_x * es);
    t.in(d_final_state, n_s * 4, true);
    t.out(grad_x, n_x * 4);
    t.out(grad_weight, (size_t)C * W * 4);
    t.out(grad_bias, (size_t)C * 4, true);
    t.out(grad_initial_state, n_s * 4, true);
    if (!t.ok() || !t.workspace(workspace, workspace_bytes, kda::conv_bwd_workspace(B, T, C, W, N, dtype)))
        return KDA_ERR_INVALID_ARG;
    kda::ConvArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.initial_state = initial_state; a.cu_seqlens = cu_seqlens;
    a.d_out = d_out; a.d_final_state = d_final_state;
    a.grad_x = grad_x; a.grad_weight = grad_weight; a.grad_bias = grad_bias;
    a.grad_initial_state = grad_initial_state; a.workspace = workspace;
    a.B = B; a.T = T; a.C = C; a.W = W; a.N = N; a.silu = (flags & KDA_FLAG_SILU) != 0;
    return status_of(kda::launch_conv_bwd(a, dtype, stream));
}

size_t kda_ssm_scan_fwd_workspace_bytes(int B, int T, int D, int S, int G, int N, int packed, kda_dtype dtype)
{
    if (!sizes_ok(B, T, D, N, packed) || !dtype_ok(dtype) || check_scan(D, S, G, 0)) return 0;
    return kda::scan_fwd_workspace(B, T, D, S, G, N, packed, dtype);
}

kda_status kda_ssm_scan_fwd(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                            const float* skip, const void* z, const float* delta_bias, const float* initial_state,
                            const int32_t* cu_seqlens, void* out, float* final_state, int B, int T, int D, int S,
                            int G, int N, kda_dtype dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream)
{
    if (kda_status s = check_sizes(B, T, D, N, cu_seqlens, dtype)) return s;
    if (kda_status s = check_scan(D, S, G, flags)) return s;
    const size_t es = elem_size(dtype), tokens = (size_t)B * T, n_u = tokens * D * es, n_b = tokens * G * S * es;
    const size_t n_s = (size_t)N * D * S * 4;
    Tensors t;
    t.in(u, n_u);
    t.in(delta, n_u);
    t.in(A, (size_t)D * S * 4);
    t.in(Bm, n_b);
    t.in(Cm, n_b);
    t.in(skip, (size_t)D * 4, true);
    t.in(z, n_u, true);
    t.in(delta_bias, (size_t)D * 4, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.in_out_state(initial_state, final_state, n_s);
    t.out(out, n_u);
    if (!t.ok() || !t.workspace(workspace, workspace_bytes,
                                kda::scan_fwd_workspace(B, T, D, S, G, N, cu_seqlens != nullptr, dtype)))
        return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a = {};
    a.u = u; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.delta_bias = delta_bias;
    a.initial_state = initial_state; a.cu_seqlens = cu_seqlens; a.out = out; a.final_state = final_state;
    a.workspace = workspace;
    a.B = B; a.T = T; a.D = D; a.S = S; a.G = G; a.N = N; a.softplus = (flags & KDA_FLAG_SOFTPLUS) != 0;
    return status_of(kda::launch_scan_fwd(a, dtype, stream));
}

kda_status kda_ssm_step(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                        const float* skip, const void* z, const float* delta_bias, float* state, void* out, int N,
                        int D, int S, int G, kda_dtype dtype, unsigned flags, cudaStream_t stream)
{
    if (kda_status s = check_sizes(N, 1, D, N, nullptr, dtype)) return s;
    if (kda_status s = check_scan(D, S, G, flags)) return s;
    if (N == 0) return KDA_OK;
    const size_t es = elem_size(dtype), n_u = (size_t)N * D * es, n_b = (size_t)N * G * S * es;
    Tensors t;
    t.in(u, n_u);
    t.in(delta, n_u);
    t.in(A, (size_t)D * S * 4);
    t.in(Bm, n_b);
    t.in(Cm, n_b);
    t.in(skip, (size_t)D * 4, true);
    t.in(z, n_u, true);
    t.in(delta_bias, (size_t)D * 4, true);
    t.out(state, (size_t)N * D * S * 4);
    t.out(out, n_u);
    if (!t.ok()) return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a = {};
    a.u = u; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.delta_bias = delta_bias;
    a.out = out; a.final_state = state;
    a.D = D; a.S = S; a.G = G; a.N = N; a.softplus = (flags & KDA_FLAG_SOFTPLUS) != 0;
    return status_of(kda::launch_scan_step(a, dtype, stream));
}

size_t kda_ssm_scan_bwd_workspace_bytes(int B, int T, int D, int S, int G, int N, int packed, kda_dtype dtype)
{
    if (!sizes_ok(B, T, D, N, packed) || !dtype_ok(dtype) || check_scan(D, S, G, 0)) return 0;
    return kda::scan_bwd_workspace(B, T, D, S, G, N, packed, dtype);
}

kda_status kda_ssm_scan_bwd(const void* u, const void* delta, const float* A, const void* Bm, const void* Cm,
                            const float* skip, const void* z, const float* delta_bias, const float* initial_state,
                            const int32_t* cu_seqlens, const void* d_out, const float* d_final_state, float* grad_u,
                            float* grad_delta, float* grad_A, float* grad_B, float* grad_C, float* grad_skip,
                            float* grad_z, float* grad_delta_bias, float* grad_initial_state, int B, int T, int D,
                            int S, int G, int N, kda_dtype dtype, unsigned flags, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream)
{
    if (kda_status s = check_sizes(B, T, D, N, cu_seqlens, dtype)) return s;
    if (kda_status s = check_scan(D, S, G, flags)) return s;
    const size_t es = elem_size(dtype), tokens = (size_t)B * T, n_u = tokens * D, n_b = tokens * G * S;
    const size_t n_s = (size_t)N * D * S * 4;
    Tensors t;
    t.in(u, n_u * es);
    t.in(delta, n_u * es);
    t.in(A, (size_t)D * S * 4);
    t.in(Bm, n_b * es);
    t.in(Cm, n_b * es);
    t.in(skip, (size_t)D * 4, true);
    t.in(z, n_u * es, true);
    t.in(delta_bias, (size_t)D * 4, true);
    t.in(initial_state, n_s, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.in(d_out, n_u * es);
    t.in(d_final_state, n_s, true);
    t.out(grad_u, n_u * 4);
    t.out(grad_delta, n_u * 4);
    t.out(grad_A, (size_t)D * S * 4);
    t.out(grad_B, n_b * 4);
    t.out(grad_C, n_b * 4);
    t.out(grad_skip, (size_t)D * 4, true);
    t.out(grad_z, z ? n_u * 4 : 0);
    t.out(grad_delta_bias, (size_t)D * 4, true);
    t.out(grad_initial_state, n_s, true);
    if (!t.ok() || !t.workspace(workspace, workspace_bytes,
                                kda::scan_bwd_workspace(B, T, D, S, G, N, cu_seqlens != nullptr, dtype)))
        return KDA_ERR_INVALID_ARG;
    kda::ScanArgs a = {};
    a.u = u; a.delta = delta; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.delta_bias = delta_bias;
    a.initial_state = initial_state; a.cu_seqlens = cu_seqlens; a.d_out = d_out; a.d_final_state = d_final_state;
    a.grad_u = grad_u; a.grad_delta = grad_delta; a.grad_A = grad_A; a.grad_B = grad_B; a.grad_C = grad_C;
    a.grad_skip = grad_skip; a.grad_z = grad_z; a.grad_delta_bias = grad_delta_bias;
    a.grad_initial_state = grad_initial_state; a.workspace = workspace;
    a.B = B; a.T = T; a.D = D; a.S = S; a.G = G; a.N = N; a.softplus = (flags & KDA_FLAG_SOFTPLUS) != 0;
    return status_of(kda::launch_scan_bwd(a, dtype, stream));
}

size_t kda_group_norm_fwd_workspace_bytes(int B, int T, int C, int G, int N, int packed, kda_dtype dtype,
                                          unsigned flags)
{
    if (!sizes_ok(B, T, C, N, packed) || !dtype_ok(dtype) || G <= 0 || C % G != 0) return 0;
    return kda::norm_fwd_workspace(B, T, C, G, N, (flags & KDA_FLAG_PER_TOKEN) != 0, packed, dtype);
}

size_t kda_group_norm_bwd_workspace_bytes(int B, int T, int C, int G, int N, int packed, kda_dtype dtype,
                                          unsigned flags)
{
    if (!sizes_ok(B, T, C, N, packed) || !dtype_ok(dtype) || G <= 0 || C % G != 0) return 0;
    return kda::norm_bwd_workspace(B, T, C, G, N, (flags & KDA_FLAG_PER_TOKEN) != 0, packed, dtype);
}

kda_status kda_group_norm_fwd(const void* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                              float eps, void* out, float* mean, float* rstd, int B, int T, int C, int G, int N,
                              kda_dtype dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream)
{
    if (flags & ~(unsigned)(KDA_FLAG_SILU | KDA_FLAG_PER_TOKEN)) return KDA_ERR_UNSUPPORTED;
    if (kda_status s = check_sizes(B, T, C, N, cu_seqlens, dtype)) return s;
    if (G <= 0 || C % G != 0) return KDA_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps < 1e30f)) return KDA_ERR_INVALID_ARG;
    const bool per_token = (flags & KDA_FLAG_PER_TOKEN) != 0;
    const size_t tokens = (size_t)B * T, n_x = tokens * C * elem_size(dtype);
    const size_t n_m = (per_token ? tokens : (size_t)N) * G * 4;
    Tensors t;
    t.in(x, n_x);
    t.in(weight, (size_t)C * 4, true);
    t.in(bias, (size_t)C * 4, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.out(out, n_x);
    t.out(mean, n_m);
    t.out(rstd, n_m);
    if (!t.ok() || !t.workspace(workspace, workspace_bytes,
                                kda::norm_fwd_workspace(B, T, C, G, N, per_token, cu_seqlens != nullptr, dtype)))
        return KDA_ERR_INVALID_ARG;
    if (n_m == 0) return KDA_OK;
    kda::NormArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.cu_seqlens = cu_seqlens; a.out = out; a.mean = mean; a.rstd = rstd;
    a.workspace = workspace; a.eps = eps;
    a.B = B; a.T = T; a.C = C; a.G = G; a.N = N; a.per_token = per_token; a.silu = (flags & KDA_FLAG_SILU) != 0;
    return status_of(kda::launch_norm_fwd(a, dtype, stream));
}

kda_status kda_group_norm_bwd(const void* x, const float* weight, const float* bias, const int32_t* cu_seqlens,
                              const float* mean, const float* rstd, const void* d_out, float* grad_x,
                              float* grad_weight, float* grad_bias, int B, int T, int C, int G, int N,
                              kda_dtype dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                              cudaStream_t stream)
{
    if (flags & ~(unsigned)(KDA_FLAG_SILU | KDA_FLAG_PER_TOKEN)) return KDA_ERR_UNSUPPORTED;
    if (kda_status s = check_sizes(B, T, C, N, cu_seqlens, dtype)) return s;
    if (G <= 0 || C % G != 0) return KDA_ERR_INVALID_ARG;
    const bool per_token = (flags & KDA_FLAG_PER_TOKEN) != 0;
    const size_t tokens = (size_t)B * T, n_x = tokens * C, es = elem_size(dtype);
    const size_t n_m = (per_token ? tokens : (size_t)N) * G * 4;
    Tensors t;
    t.in(x, n_x * es);
    t.in(weight, (size_t)C * 4, true);
    t.in(bias, (size_t)C * 4, true);
    t.in(cu_seqlens, ((size_t)N + 1) * 4, true);
    t.in(mean, n_m);
    t.in(rstd, n_m);
    t.in(d_out, n_x * es);
    t.out(grad_x, n_x * 4);
    t.out(grad_weight, (size_t)C * 4, true);
    t.out(grad_bias, (size_t)C * 4, true);
    if (!t.ok() || !t.workspace(workspace, workspace_bytes,
                                kda::norm_bwd_workspace(B, T, C, G, N, per_token, cu_seqlens != nullptr, dtype)))
        return KDA_ERR_INVALID_ARG;
    kda::NormArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.cu_seqlens = cu_seqlens;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.d_out = d_out; a.grad_x = grad_x; a.grad_weight = grad_weight; a.grad_bias = grad_bias; a.workspace = workspace;
    a.B = B; a.T = T; a.C = C; a.G = G; a.N = N; a.per_token = per_token; a.silu = (flags & KDA_FLAG_SILU) != 0;
    return status_of(kda::launch_norm_bwd(a, dtype, stream));
}

}  // extern "C"
