// Selective state-space scan, forward: prompts (packed or not) and single
// tokens.  See ssm_common.cuh for the recurrence and the thread layout.
//
// Bound by the exponentials: one a = exp(dt A) per token, channel and state,
// 16 a clock on an SM's special function unit, against 8 bytes of traffic per
// token and channel.  Chains (a sequence's channel) run one after another
// along the tokens, so few chains leave SMs idle; then sequences are cut into
// units.  The recurrence is affine with a diagonal factor, h_out =
// exp(A sum dt) h_in + e, so a first pass computes every unit's e and sum of
// dt, a small kernel chains the entry states, and the second pass runs all
// units at once.
#include "ssm_common.cuh"

namespace kda {
namespace {

using namespace ssm;

// kCarry: the first pass, end state from zero and sum of dt of every unit that
// another one follows.
template <typename T, int L, bool kCarry>
__global__ void __launch_bounds__(kThreads, 2)
kda_ssm_scan_kernel(Params<T> p)
{
    using Tl = Tile<L>;
    constexpr int CH = Tl::CH, TT = Tl::TT, SP = Tl::SP, Q = Tl::Q, YP = Tl::YP, IPT = Tl::IPT;
    __shared__ __align__(16) float2 s_dt[2][TT][CH];  // dt, dt u
    __shared__ __align__(16) float s_B[2][TT * SP];
    __shared__ __align__(16) float s_C[kCarry ? 1 : 2][kCarry ? 4 : TT * SP];
    __shared__ __align__(16) float s_y[kCarry ? 1 : 2][kCarry ? 4 : TT * YP];

    const int tid = threadIdx.x, lane = tid & 31;
    const int across = p.G * p.cpb;
    const long long slot = blockIdx.x / across;
    const int gb = (int)(blockIdx.x % across), g = gb / p.cpb;
    int n, seg;
    long long t0, end;
    if (!p.units.locate(slot, n, seg, t0, end)) return;
    const bool last = seg + 1 == p.units.count(n);
    if (kCarry && last) return;
    const int cg = (gb % p.cpb) * CH;                      // first channel within the group
    const int nch = p.Dg - cg < CH ? p.Dg - cg : CH;       // channels of this block
    const int c0 = g * p.Dg + cg;

    // this thread's channel and states
    const int ch = tid / L, s0 = (tid % L) * 4;
    const bool chan = ch < nch;
    const size_t row = (size_t)(c0 + (chan ? ch : 0)) * p.S;
    float A[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool ok = chan && s0 + i < p.S;
        A[i] = ok ? p.A[row + s0 + i] * kLog2e : 0.f;
        h[i] = 0.f;
        if (ok && !kCarry) {
            if (p.ends) h[i] = p.ends[(size_t)slot * p.D * p.S + row + s0 + i];
            else if (p.init) h[i] = p.init[(size_t)n * p.D * p.S + row + s0 + i];
        }
    }

    const float2 A01 = make_float2(A[0], A[1]), A23 = make_float2(A[2], A[3]);
    float2 h01 = make_float2(h[0], h[1]), h23 = make_float2(h[2], h[3]);

    // this thread's channel quad when tiles are staged and written out
    const int q4 = (tid % Q) * 4;
    float bias[4], skip[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bias[i] = p.delta_bias && q4 + i < nch ? p.delta_bias[c0 + q4 + i] : 0.f;
        skip[i] = p.skip && q4 + i < nch ? p.skip[c0 + q4 + i] : 0.f;
    }

    ChannelRows<T, Tl> u, d, z, u_now, z_now;
    StateRows<T, Tl, !kCarry> bc;
    float dt_sum[4] = {0.f, 0.f, 0.f, 0.f};

    auto fetch = [&](long long t) {
        u.load(p.u, p, t, end, c0, nch, tid);
        d.load(p.delta, p, t, end, c0, nch, tid);
        if (!kCarry && p.z) z.load(p.z, p, t, end, c0, nch, tid);
        bc.load(p, t, end, g, tid);
    };
    auto stage = [&](long long t, int buf) {
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const int tt = (tid + k * kThreads) / Q;
            if (tt >= TT) break;
            float x[4], dv[4];
            u.r[k].get(x);
            d.r[k].get(dv);
            const bool in = t + tt < end;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = dv[i] + bias[i];
                if (p.softplus) v = softplus(v);
                if (!in) v = 0.f;
                if (kCarry) dt_sum[i] += v;
                dv[i] = v;
            }
            float4* o = reinterpret_cast<float4*>(&s_dt[buf][tt][q4]);
            o[0] = make_float4(dv[0], dv[0] * x[0], dv[1], dv[1] * x[1]);
            o[1] = make_float4(dv[2], dv[2] * x[2], dv[3], dv[3] * x[3]);
        }
        bc.put(s_B[buf], s_C[kCarry ? 0 : buf], tid);
    };

    fetch(t0);
    stage(t0, 0);
    u_now = u;
    if (!kCarry && p.z) z_now = z;
    if (t0 + TT < end) fetch(t0 + TT);
    __syncthreads();
    int buf = 0;
    for (long long t = t0; t < end; t += TT, buf ^= 1) {
        ChannelRows<T, Tl> u_next, z_next;
        if (t + TT < end) {
            stage(t + TT, buf ^ 1);
            u_next = u;
            if (!kCarry && p.z) z_next = z;
            if (t + 2 * TT < end) fetch(t + 2 * TT);
        }
#pragma unroll 2
        for (int tb = 0; tb < TT; tb += 4) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 dd = s_dt[buf][tb + j][ch];
                const float4 B = *reinterpret_cast<const float4*>(&s_B[buf][(tb + j) * SP + s0]);
                const float2 dt = both(dd.x), du = both(dd.y);
                h01 = fma2(ex2(mul2(dt, A01)), h01, mul2(du, make_float2(B.x, B.y)));
                h23 = fma2(ex2(mul2(dt, A23)), h23, mul2(du, make_float2(B.z, B.w)));
                if constexpr (!kCarry) {
                    const float4 C = *reinterpret_cast<const float4*>(&s_C[buf][(tb + j) * SP + s0]);
                    const float2 yy = fma2(h01, make_float2(C.x, C.y), mul2(h23, make_float2(C.z, C.w)));
                    y[j] = yy.x + yy.y;
                }
            }
            if constexpr (!kCarry) {
                fold<4, L, 1>(y, lane);
                constexpr int KEEP = L >= 4 ? 1 : 4 / L;      // tokens a lane is left with
                constexpr int BITS = L >= 4 ? 2 : (L == 2 ? 1 : 0);
                if (tid % L < 4) {
                    const int at = fold_index<BITS>(lane, 1) * KEEP;
#pragma unroll
                    for (int i = 0; i < KEEP; ++i) s_y[buf][(tb + at + i) * YP + ch] = y[i];
                }
            }
        }
        __syncthreads();
        if constexpr (!kCarry) {
#pragma unroll
            for (int k = 0; k < IPT; ++k) {
                const int tt = (tid + k * kThreads) / Q;
                if (tt >= TT || t + tt >= end || q4 >= nch) continue;
                const float4 y4 = *reinterpret_cast<const float4*>(&s_y[buf][tt * YP + q4]);
                float x[4], zz[4], y[4] = {y4.x, y4.y, y4.z, y4.w};
                u_now.r[k].get(x);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = fmaf(skip[i], x[i], y[i]);
                if (p.z) {
                    z_now.r[k].get(zz);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] *= silu(zz[i]);
                }
                store4(p.out + (size_t)(t + tt) * p.D + c0 + q4, y, p.vec_d, nch - q4);
            }
            u_now = u_next;
            if (p.z) z_now = z_next;
        }
    }

    h[0] = h01.x;
    h[1] = h01.y;
    h[2] = h23.x;
    h[3] = h23.y;
    if constexpr (kCarry) {
        float* e = p.ends + (size_t)slot * p.D * p.S + row + s0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (chan && s0 + i < p.S) e[i] = h[i];
        // sum of dt over the threads that staged a channel's tokens
        float* red = reinterpret_cast<float*>(&s_dt[0][0][0]);
        __syncthreads();
        if (tid / Q < TT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) red[(tid / Q) * CH + q4 + i] = dt_sum[i];
        }
        __syncthreads();
        if (tid < nch) {
            float s = 0.f;
            for (int r = 0; r < Tl::ROWS; ++r) s += red[r * CH + tid];
            p.steps[(size_t)slot * p.D + c0 + tid] = s;
        }
    } else if (last && p.fin && chan) {
        float* f = p.fin + (size_t)n * p.D * p.S + row + s0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s0 + i < p.S) f[i] = h[i];
    }
}

// Entry states of the units of every (sequence, channel, state), in place of
// their end states: h <- exp(A sum dt) h + e, unit after unit.
__global__ void __launch_bounds__(256)
kda_ssm_chain_kernel(const float* __restrict__ A, const float* __restrict__ init, float* ends,
                     const float* __restrict__ steps, Units units, int D, int S)
{
    const size_t DS = (size_t)D * S;
    const int per = (int)((DS + 255) / 256);
    const int n = (int)(blockIdx.x / per);
    const size_t i = (size_t)(blockIdx.x % per) * 256 + threadIdx.x;
    if (i >= DS) return;
    const float a = A[i] * kLog2e;
    const size_t d = i / S;
    const long long first = units.first(n);
    const int cnt = units.count(n);
    float h = init ? init[(size_t)n * DS + i] : 0.f;
    float* e = ends + (size_t)first * DS + i;
    const float* st = steps + (size_t)first * D + d;
    constexpr int U = 4;
    for (int k = 0; k < cnt; k += U) {
        float end[U], dt[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const bool ok = k + j + 1 < cnt;  // the last unit's end is no one's entry
            end[j] = ok ? e[(size_t)(k + j) * DS] : 0.f;
            dt[j] = ok ? st[(size_t)(k + j) * D] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (k + j < cnt) {
                e[(size_t)(k + j) * DS] = h;
                h = fmaf(ex2(a * dt[j]), h, end[j]);
            }
    }
}

// One token for each of N sequences, the state read and written once in place
// (memory-bound).  L lanes share a channel, each holding 4 neighbouring
// states: whole rows of states go by in 16-byte accesses.  A thread takes its
// channel of R sequences, whose states are in flight together and share A.
template <typename T, int L, bool kVec, int R>
__global__ void __launch_bounds__(256)
kda_ssm_step_kernel(const T* __restrict__ u, const T* __restrict__ delta, const float* __restrict__ A,
                    const T* __restrict__ Bm, const T* __restrict__ Cm, const float* __restrict__ skip,
                    const T* __restrict__ z, const float* __restrict__ delta_bias, float* state,
                    T* __restrict__ out, int N, int D, int S, int Dg, int G, int across, int use_softplus)
{
    const int at = (int)(blockIdx.x % across) * (256 / L) + threadIdx.x / L;
    const int n0 = (int)(blockIdx.x / across) * R;
    const int l = threadIdx.x % L, s0 = l * 4;
    const bool live = at < D;
    const int d = live ? at : 0;
    const int g = d / Dg;
    float h[R][4], a[4], B[R][4], C[R][4], x[R][1], dv[R][1], zz[R][1];
    auto row4 = [&](const auto* p, float(&v)[4]) {
        if constexpr (kVec) {
            if (s0 < S) {
                load_vec<4>(p, v);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float w[1] = {0.f};
            if (!kVec && s0 + i < S) load_vec<1>(p + i, w);
            v[i] = w[0];
        }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r < N ? n0 + r : N - 1;
        row4(state + ((size_t)n * D + d) * S + s0, h[r]);
    }
    row4(A + (size_t)d * S + s0, a);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r < N ? n0 + r : N - 1;
        const size_t bc = ((size_t)n * G + g) * S + s0, nd = (size_t)n * D + d;
        row4(Bm + bc, B[r]);
        row4(Cm + bc, C[r]);
        load_vec<1>(u + nd, x[r]);
        load_vec<1>(delta + nd, dv[r]);
        zz[r][0] = 0.f;
        if (z) load_vec<1>(z + nd, zz[r]);
    }
    const float bias = delta_bias ? delta_bias[d] : 0.f, sk = skip ? skip[d] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] *= kLog2e;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r;
        float dt = dv[r][0] + bias;
        if (use_softplus) dt = softplus(dt);
        const float du = dt * x[r][0];
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[r][i] = fmaf(ex2(dt * a[i]), h[r][i], du * B[r][i]);
            y = fmaf(h[r][i], C[r][i], y);
        }
        const bool here = live && n < N;
        if (here) store4(state + ((size_t)n * D + d) * S + s0, h[r], kVec && s0 < S, S - s0);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (here && l == 0) {
            y = fmaf(sk, x[r][0], y);
            if (z) y *= silu(zz[r][0]);
            const float o[1] = {y};
            store_vec<1>(out + (size_t)n * D + d, o);
        }
    }
}

// A unit's tokens are passed over twice where sequences are cut.
constexpr int kWarps = 12, kShortest = 64;

template <typename T, int L>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st)
{
    const Cut c = cut_of(a.B, a.T, a.D, a.S, a.N, a.cu_seqlens != nullptr, kWarps, kShortest);
    Params<T> p = params_of<T>(a, c.len, Tile<L>::CH);
    const long long slots = p.units.slots();
    const long long blocks = slots * p.G * p.cpb;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    if (c.cut) {
        p.ends = (float*)a.workspace;
        p.steps = (float*)((char*)a.workspace + round256((size_t)slots * a.D * a.S * 4));
        kda_ssm_scan_kernel<T, L, true><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
        if (cudaError_t e = launch_ssm_chain(a.A, a.initial_state, p.ends, p.steps, p.units, a.D, a.S, st)) return e;
    }
    kda_ssm_scan_kernel<T, L, false><<<(unsigned)blocks, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int L>
cudaError_t step(const ScanArgs& a, cudaStream_t st)
{
    const int across = (int)(((long long)a.D * L + 255) / 256);
    // four sequences a thread once that still fills every SM's threads
    const int R = (long long)across * a.N >= 4LL * 8 * sm_count() ? 4 : 1;
    const long long blocks = (long long)across * ((a.N + R - 1) / R);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    const bool vec = a.S % 4 == 0;
    auto* k = R == 4 ? (vec ? &kda_ssm_step_kernel<T, L, true, 4> : &kda_ssm_step_kernel<T, L, false, 4>)
                     : (vec ? &kda_ssm_step_kernel<T, L, true, 1> : &kda_ssm_step_kernel<T, L, false, 1>);
    k<<<(unsigned)blocks, 256, 0, st>>>((const T*)a.u, (const T*)a.delta, a.A, (const T*)a.Bm, (const T*)a.Cm, a.skip,
                                        (const T*)a.z, a.delta_bias, a.final_state, (T*)a.out, a.N, a.D, a.S,
                                        a.D / a.G, a.G, across, a.softplus);
    return cudaGetLastError();
}

template <typename T, bool kStep>
cudaError_t by_states(const ScanArgs& a, cudaStream_t st)
{
    switch (lanes_of(a.S)) {
#define KDA_SSM_L(L) \
    case L:          \
        return kStep ? step<T, L>(a, st) : fwd<T, L>(a, st);
        KDA_SSM_L(1)
        KDA_SSM_L(2)
        KDA_SSM_L(4)
        KDA_SSM_L(8)
        KDA_SSM_L(16)
        KDA_SSM_L(32)
#undef KDA_SSM_L
    }
    return cudaErrorInvalidValue;
}

}  // namespace

namespace ssm {
cudaError_t launch_ssm_chain(const float* A, const float* init, float* ends, const float* steps, const Units& units,
                             int D, int S, cudaStream_t st)
{
    const long long blocks = ((long long)D * S + 255) / 256 * units.s.N;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    kda_ssm_chain_kernel<<<(unsigned)blocks, 256, 0, st>>>(A, init, ends, steps, units, D, S);
    return cudaGetLastError();
}
}  // namespace ssm

size_t scan_fwd_workspace(int B, int T, int D, int S, int, int N, int packed, kda_dtype)
{
    const Cut c = cut_of(B, T, D, S, N, packed, kWarps, kShortest);
    if (!c.cut) return 0;
    const size_t slots = (size_t)slots_of(B, T, N, packed, c.len);
    return round256(slots * D * S * 4) + slots * D * 4;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? by_states<__nv_bfloat16, false>(a, st) : by_states<float, false>(a, st);
}

cudaError_t launch_scan_step(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? by_states<__nv_bfloat16, true>(a, st) : by_states<float, true>(a, st);
}

}  // namespace kda
