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

// A block is one warp and needs no barrier: with some 7 warps an SM, as many as
// four prompts of 4096 channels give it, larger blocks leave SMs with one block
// more or less than others.  Few warps also mean that latency has to be hidden
// inside each: operands come from shared memory two tokens ahead, decays are
// computed one token ahead, and the register bound is wide (11 warps an SM; with
// the compiler's own 128 registers the same code took 712 us against 538).
//
// 4 x 4096 tokens of 4096 channels, 16 states, bf16: 539 us.  Its 67 M x 20
// special function results take 295 us, its bytes 83 us.  The unit is busy 54 %
// of the time, issue slots 54 %: two warps a scheduler do not fill more.  Four
// states of one channel a lane (600 us) and sixteen (977 us) were slower: there
// the reads of B and C, 128 bytes a clock back to the registers, are as long as
// the exponentials, which come back the same way.
template <int LANES>
using Fwd = Shape<LANES, 16, 32>;

enum Mode {
    kOut,     // outputs and final states
    kCarry,   // end state from zero and sum of dt of every unit that another one follows
    kEntries  // the state at every tile's entry
};

template <typename T, int LANES, Mode mode>
__global__ void __launch_bounds__(32, 11)
kda_ssm_scan_kernel(Params<T> p)
{
    using Tl = Fwd<LANES>;
    constexpr int L = Tl::L, CH = Tl::CH, TT = Tl::TT, SP = Tl::SP, TB = Tl::TB, NB = Tl::NB, OWN = Tl::OWN;
    constexpr int PAIRS = Tl::PAIRS;
    __shared__ __align__(16) float2 s_dt[TT][PAIRS][2];  // dt, dt u
    __shared__ __align__(16) float s_B[TT * SP];
    __shared__ __align__(16) float s_C[mode != kOut ? 4 : TT * SP];

    const int lane = threadIdx.x & 31;
    const int across = p.G * p.cpb;
    const int slot = blockIdx.x / across;
    const int gb = (int)(blockIdx.x % across), g = gb / p.cpb;
    int n, seg, t0, end;
    bool last;
    if (!p.units.locate(slot, n, seg, last, t0, end)) return;
    if (mode == kCarry && last) return;
    const int cg = (gb % p.cpb) * CH;                      // first channel within the group
    const int nch = p.Dg - cg < CH ? p.Dg - cg : CH;       // channels of this block
    const int c0 = g * p.Dg + cg;

    // this lane's states of its pair's channels (a channel behind the last stands
    // for the last and is not stored)
    const int pair = lane / L, s0 = (lane % L) * 4;
    // A sequence of several units takes every entry state from `ends`, its
    // initial state too: the block of its last unit may write `fin` over it.
    const bool chained = p.ends && !(seg == 0 && last);
    float A[2][4], h[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int c = pair * 2 + r;
        const size_t row = (size_t)(c0 + (c < nch ? c : nch - 1)) * p.S + s0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool ok = s0 + i < p.S;
            A[r][i] = ok ? rate(p.A[row + i]) : 0.f;
            h[r][i] = 0.f;
            if (ok && mode != kCarry) {
                if (chained) h[r][i] = p.ends[(size_t)slot * p.D * p.S + row + i];
                else if (p.init) h[r][i] = p.init[(size_t)n * p.D * p.S + row + i];
            }
        }
    }

    // this lane's own elements: tokens TB e + tok of the channels own[], e = 0 .. NB - 1
    const int tok = fold_index<Tl::BITS>(lane, 2);
    int own[OWN];
    float bias[OWN], skip[OWN], dt_sum[OWN];
    bool mine[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int c = pair * 2 + (OWN == 2 ? o : lane & 1);
        mine[o] = c < nch;
        own[o] = c0 + (c < nch ? c : nch - 1);
        bias[o] = p.delta_bias ? p.delta_bias[own[o]] : 0.f;
        skip[o] = p.skip ? p.skip[own[o]] : 0.f;
        dt_sum[o] = 0.f;
    }
    const bool gate = mode == kOut && p.z;

    T u[NB][OWN], d[NB][OWN], z[NB][OWN];
    StateRows<T, Tl, mode == kOut> bc;
    // the tile from token t on (tokens behind the end repeat the last)
    const size_t step = (size_t)TB * p.D;
    auto fetch = [&](int t) {
        if (t + TT <= end) {
            size_t at = (size_t)(t + tok) * p.D;
#pragma unroll
            for (int e = 0; e < NB; ++e, at += step)
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    u[e][o] = p.u[at + own[o]];
                    d[e][o] = p.delta[at + own[o]];
                    if (gate) z[e][o] = p.z[at + own[o]];
                }
        } else {
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                const int tt = t + e * TB + tok;
                const size_t at = (size_t)(tt < end ? tt : end - 1) * p.D;
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    u[e][o] = p.u[at + own[o]];
                    d[e][o] = p.delta[at + own[o]];
                    if (gate) z[e][o] = p.z[at + own[o]];
                }
            }
        }
        bc.load(p, t, end, g, lane);
    };

    if (t0 < end) fetch(t0);
    for (int t = t0; t < end; t += TT) {
        const int left = end - t < TT ? end - t : TT;
        if constexpr (mode == kEntries) {
            float* to = p.entries + (size_t)(t0 / TT + slot + (t - t0) / TT) * p.D * p.S;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int c = pair * 2 + r;
                if (c < nch) store4(to + (size_t)(c0 + c) * p.S + s0, h[r], p.vec_s && s0 < p.S, p.S - s0);
            }
            if (t + TT >= end) break;
        }
        float x[NB][OWN], zz[NB][OWN], dt[NB * OWN];
#pragma unroll
        for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                float w[1];
                load_vec<1>(&u[e][o], w);
                x[e][o] = w[0];
                load_vec<1>(&d[e][o], w);
                dt[e * OWN + o] = w[0] + bias[o];
                if (gate) {
                    load_vec<1>(&z[e][o], w);
                    zz[e][o] = w[0];
                }
            }
        if (p.softplus) {
            if constexpr (NB * OWN % 2 == 0) {
#pragma unroll
                for (int i = 0; i < NB * OWN; i += 2) {
                    const float2 v = softplus2(make_float2(dt[i], dt[i + 1]));
                    dt[i] = v.x;
                    dt[i + 1] = v.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NB * OWN; ++i) dt[i] = softplus(dt[i]);
            }
        }
#pragma unroll
        for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const bool in = e * TB + tok < left;  // behind the end: a step of nothing
                const float v = in ? dt[e * OWN + o] : 0.f, w = in ? v * x[e][o] : 0.f;
                if (mode == kCarry) dt_sum[o] += v;
                s_dt[e * TB + tok][pair][OWN == 2 ? o : lane & 1] = make_float2(v, w);
            }
        bc.put(s_B, s_C, lane);
        if (t + TT < end) fetch(t + TT);
        __syncwarp();
        // Two tokens ahead: what is read from shared memory; one ahead: the
        // decays, so that neither's latency stands in the recurrence's way.
        float4 dd[3], B[3], C[3];
        float a[2][2][4], mean[2];
        auto read = [&](int tt) {
            dd[tt % 3] = *reinterpret_cast<const float4*>(&s_dt[tt][pair][0]);
            B[tt % 3] = *reinterpret_cast<const float4*>(&s_B[tt * SP + s0]);
            if constexpr (mode == kOut) C[tt % 3] = *reinterpret_cast<const float4*>(&s_C[tt * SP + s0]);
        };
        auto decays = [&](int tt) {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) a[tt % 2][r][i] = decay(r ? dd[tt % 3].z : dd[tt % 3].x, A[r][i], mean[r]);
        };
        read(0);
        read(1);
        mean[0] = mean_error(dd[0].x, slowest(A[0]));
        mean[1] = mean_error(dd[0].z, slowest(A[1]));
        decays(0);
        size_t at = (size_t)(t + tok) * p.D;
#pragma unroll
        for (int e = 0; e < NB; ++e, at += step) {
            float y[2 * TB];
#pragma unroll
            for (int j = 0; j < TB; ++j) {
                const int tt = e * TB + j;
                if (tt + 2 < TT) read(tt + 2);
                if (tt + 1 < TT) decays(tt + 1);
                const float4 b = B[tt % 3];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float du = r ? dd[tt % 3].w : dd[tt % 3].y;
                    h[r][0] = fmaf(a[tt % 2][r][0], h[r][0], du * b.x);
                    h[r][1] = fmaf(a[tt % 2][r][1], h[r][1], du * b.y);
                    h[r][2] = fmaf(a[tt % 2][r][2], h[r][2], du * b.z);
                    h[r][3] = fmaf(a[tt % 2][r][3], h[r][3], du * b.w);
                    if constexpr (mode == kOut) {
                        const float4 c = C[tt % 3];
                        y[r * TB + j] = fmaf(h[r][3], c.w, fmaf(h[r][2], c.z, fmaf(h[r][1], c.y, h[r][0] * c.x)));
                    }
                }
            }
            if constexpr (mode == kOut) {
                fold<2 * TB, L, 1>(y, lane);
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    float v[1] = {fmaf(skip[o], x[e][o], y[o])};
                    if (gate) v[0] *= silu(zz[e][o]);
                    if (mine[o] && e * TB + tok < left) store_vec<1>(p.out + at + own[o], v);
                }
            }
        }
        __syncwarp();
    }

    if (mode == kCarry || (mode == kOut && last && p.fin)) {
        __syncwarp();  // every lane has its initial state, which `fin` may be
        float* to = mode == kCarry ? p.ends + (size_t)slot * p.D * p.S : p.fin + (size_t)n * p.D * p.S;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int c = pair * 2 + r;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c < nch && s0 + i < p.S) to[(size_t)(c0 + c) * p.S + s0 + i] = h[r][i];
        }
    }
    if constexpr (mode == kCarry) {
        // a channel's tokens lie with the lanes of its parity
#pragma unroll
        for (int o = 0; o < OWN; ++o) {
#pragma unroll
            for (int i = 2; i < L; i <<= 1) dt_sum[o] += __shfl_xor_sync(0xffffffffu, dt_sum[o], i);
            if (mine[o] && lane % L < 2) p.steps[(size_t)slot * p.D + own[o]] = dt_sum[o];
        }
    }
}

__global__ void __launch_bounds__(256)
kda_ssm_chain_kernel(const float* __restrict__ A, const float* __restrict__ init, float* ends,
                     const float* __restrict__ steps, Units units, int D, int S, int span)
{
    chain_states(blockIdx.x, A, init, ends, steps, units, D, S, span);
}

// One token for each of N sequences, the state read and written once in place
// (memory-bound).  L lanes share a channel, each holding 4 neighbouring
// states: whole rows of states go by in 16-byte accesses.  A thread takes its
// channel of R sequences, whose states are in flight together and share A.  256
// sequences of 4096 channels, 16 states: 30 us, 4.8 TB/s (75 % of the measured
// copy rate); R = 1, 2 and 8 took 48, 32 and 37 us.  The lanes' common work (step,
// gate, addresses) fills 71 % of the issue slots.
template <typename T, int L, bool kVec, int R>
__global__ void __launch_bounds__(256, 4)
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
    // every state first: each is read once and written once (streaming accesses)
    float4 h[R];
    T x[R], dv[R], zz[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r < N ? n0 + r : N - 1;
        const float* st = state + ((size_t)n * D + d) * S + s0;
        if (!live) {
            h[r] = make_float4(0.f, 0.f, 0.f, 0.f);  // channel 0's is written meanwhile
        } else if (kVec && s0 < S) {
            h[r] = __ldcs(reinterpret_cast<const float4*>(st));
        } else {
            float v[4];
            row4(st, v);
            h[r] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const size_t nd = (size_t)(n0 + r < N ? n0 + r : N - 1) * D + d;
        x[r] = u[nd];
        dv[r] = delta[nd];
        if (z) zz[r] = z[nd];
    }
    float a[4];
    row4(A + (size_t)d * S + s0, a);
    const float bias = delta_bias ? delta_bias[d] : 0.f, sk = skip ? skip[d] : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = rate(a[i]);
    const float slow = slowest(a);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r;
        const size_t bc = ((size_t)(n < N ? n : N - 1) * G + g) * S + s0;
        float B[4], C[4], xx[1], dd[1];
        row4(Bm + bc, B);
        row4(Cm + bc, C);
        load_vec<1>(&x[r], xx);
        load_vec<1>(&dv[r], dd);
        float dt = dd[0] + bias;
        if (use_softplus) dt = softplus(dt);
        const float du = dt * xx[0], mean = mean_error(dt, slow);
        float hh[4] = {h[r].x, h[r].y, h[r].z, h[r].w}, y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hh[i] = fmaf(decay(dt, a[i], mean), hh[i], du * B[i]);
            y = fmaf(hh[i], C[i], y);
        }
        const bool here = live && n < N;
        if (here) {
            float* st = state + ((size_t)n * D + d) * S + s0;
            if (kVec && s0 < S) __stcs(reinterpret_cast<float4*>(st), make_float4(hh[0], hh[1], hh[2], hh[3]));
            else store4(st, hh, false, S - s0);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (here && l == 0) {
            y = fmaf(sk, xx[0], y);
            if (z) {
                load_vec<1>(&zz[r], xx);
                y *= silu(xx[0]);
            }
            const float o[1] = {y};
            store_vec<1>(out + (size_t)n * D + d, o);
        }
    }
}

// A unit's tokens are passed over twice where sequences are cut, and whole ones
// take as long as their chain is, so what decides is how many warps the chains give
// an SM.  bf16, 16 states, whole against cut: 1 x 16384 tokens of 4096 channels (1.7
// warps) 1466 and 812 us, 7 x 2340 of 1024 (3.0) 217 and 258, 2 x 8192 of 4096
// (3.5) 751 and 870, 4 x 4096 (6.9) 539 and 912; 2 x 1024 (3.5) 99 and 127.  Of a
// packed batch the longest sequence is not known, and cut at the mean it may be
// little shorter: 5 ragged sequences of 2048 channels, 16384 tokens in all (4.3
// warps), 592 to 759 us at the mean, 455 to 501 in units for sixteen warps an SM; 3
// of 4096 (5.2) 964 to 1011 and 849 to 959.  Units for sixteen warps: 20011 packed
// tokens of 1100 channels 287 us, 348 for twelve.  The two launches more are worth
// some hundred tokens.
constexpr int kFewWarps = 3, kFewWarpsPacked = 6, kWantWarps = 16, kShortest = 32, kLeast = 128;

Cut fwd_cut(int B, int T, int D, int S, int N, int packed)
{
    return cut_of(B, T, N, packed, (double)D * lanes_of(S) / 64.0, packed ? kFewWarpsPacked : kFewWarps, kWantWarps,
                  kShortest, kLeast);
}

template <typename T, int L>
cudaError_t fwd(const ScanArgs& a, cudaStream_t st)
{
    const Cut c = fwd_cut(a.B, a.T, a.D, a.S, a.N, a.cu_seqlens != nullptr);
    Params<T> p = params_of<T>(a, c.len, Fwd<L>::CH);
    const int slots = p.units.slots();
    const long long blocks = (long long)slots * p.G * p.cpb;
    const ChainGrid chain = chain_grid(a.D, a.S, a.N);
    if (blocks > INT32_MAX || chain.blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    if (c.cut) {
        p.ends = (float*)a.workspace;
        p.steps = (float*)((char*)a.workspace + round256((size_t)slots * a.D * a.S * 4));
        kda_ssm_scan_kernel<T, L, kCarry><<<(unsigned)blocks, 32, 0, st>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
        kda_ssm_chain_kernel<<<(unsigned)chain.blocks, 256, 0, st>>>(a.A, a.initial_state, p.ends, p.steps, p.units,
                                                                    a.D, a.S, chain.span);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_ssm_scan_kernel<T, L, kOut><<<(unsigned)blocks, 32, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T, int L>
cudaError_t step(const ScanArgs& a, cudaStream_t st)
{
    const int across = (int)(((long long)a.D * L + 255) / 256);
    // four sequences a thread once that still fills every SM's four blocks
    const int R = (long long)across * a.N >= 4LL * 4 * sm_count() ? 4 : 1;
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

template <typename T, int L>
cudaError_t entries(const ScanArgs& a, int len, float* ends, float* to, cudaStream_t st)
{
    Params<T> p = params_of<T>(a, len, Fwd<L>::CH);
    p.ends = ends;
    p.entries = to;
    const long long blocks = (long long)p.units.slots() * p.G * p.cpb;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks > 0) kda_ssm_scan_kernel<T, L, kEntries><<<(unsigned)blocks, 32, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t entries_by_states(const ScanArgs& a, int len, float* ends, float* to, cudaStream_t st)
{
    switch (lanes_of(a.S)) {
        case 1: return entries<T, 1>(a, len, ends, to, st);
        case 2: return entries<T, 2>(a, len, ends, to, st);
        case 4: return entries<T, 4>(a, len, ends, to, st);
        case 8: return entries<T, 8>(a, len, ends, to, st);
        case 16: return entries<T, 16>(a, len, ends, to, st);
        case 32: return entries<T, 32>(a, len, ends, to, st);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t fwd_by_states(const ScanArgs& a, cudaStream_t st)
{
    switch (lanes_of(a.S)) {
        case 1: return fwd<T, 1>(a, st);
        case 2: return fwd<T, 2>(a, st);
        case 4: return fwd<T, 4>(a, st);
        case 8: return fwd<T, 8>(a, st);
        case 16: return fwd<T, 16>(a, st);
        case 32: return fwd<T, 32>(a, st);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t step_by_states(const ScanArgs& a, cudaStream_t st)
{
    if (a.S <= 4) return step<T, 1>(a, st);
    if (a.S <= 8) return step<T, 2>(a, st);
    if (a.S <= 16) return step<T, 4>(a, st);
    if (a.S <= 32) return step<T, 8>(a, st);
    if (a.S <= 64) return step<T, 16>(a, st);
    return step<T, 32>(a, st);
}

}  // namespace

namespace ssm {
cudaError_t launch_ssm_entries(const ScanArgs& a, int len, float* ends, float* to, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? entries_by_states<__nv_bfloat16>(a, len, ends, to, st)
                                   : entries_by_states<float>(a, len, ends, to, st);
}

}  // namespace ssm

size_t scan_fwd_workspace(int B, int T, int D, int S, int, int N, int packed, kda_dtype)
{
    const Cut c = fwd_cut(B, T, D, S, N, packed);
    if (!c.cut) return 0;
    const size_t slots = (size_t)slots_of(B, T, N, packed, c.len);
    return round256(slots * D * S * 4) + slots * D * 4;
}

cudaError_t launch_scan_fwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? fwd_by_states<__nv_bfloat16>(a, st) : fwd_by_states<float>(a, st);
}

cudaError_t launch_scan_step(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? step_by_states<__nv_bfloat16>(a, st) : step_by_states<float>(a, st);
}

}  // namespace kda
