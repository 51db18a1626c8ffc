// Backward pass of the selective state-space scan (ssm_scan.cu has the
// forward).  With dy = d_out silu(z) and g_t the adjoint of h_t:
//
//     g_t = C_t dy_t + a_{t+1} g_{t+1}                  (a g of the unit behind, or d_final_state)
//     dC_t = sum_d dy_t h_t           dB_t = sum_d g_t dt u
//     du   = dt (g . B) + skip dy     d dt = u (g . B) + sum_s g_t a_t h_{t-1} A
//     dA   = sum_t g_t a_t h_{t-1} dt
//     dz   = d_out y silu'(z)         d delta = d dt softplus'(delta + bias)
//
// The state at every tile's entry is written to the workspace first (a forward
// walk, ssm_scan.cu); then a block goes through its unit's tiles from the last
// to the first: a tile's states are computed again, four tokens at a time held in
// registers, and used up from the last token to the first.  Sums over a
// channel's lanes and over a warp's channels are folded (ssm_common.cuh), the
// warps' in shared memory, the blocks' and units' by kernels in a fixed order,
// so that results do not change from run to run.
//
// Where sequences are cut into units, a pass before it gives every unit its
// end state from zero, its sum of dt, and the adjoint it hands to the unit in
// front, sum_t (prod_{s <= t} a_s) C_t dy_t, all in one walk.
//
// 4 x 1024 tokens of 4096 channels, 16 states, bf16: 471 us for the walk back,
// 106 us for the entry states, 14 us for the sums; their exponentials alone are
// some 250 us of the special function unit.  The walk back takes 240 instructions
// a warp, token and 16 channels (states again 56, adjoints and their sums 90,
// folds 46) at two warps a scheduler, which fill half of the issue slots.  A lane
// per channel and 4 states, in packed arithmetic, took 650 us: twice the folds,
// and the reads of B and C.
#include "ssm_common.cuh"

namespace kda {
namespace {

using namespace ssm;

template <int LANES>
using Carry = Shape<LANES, 4, 32>;
template <int LANES>
using Bwd = Shape<LANES, 4, 128>;

template <typename T>
struct BwdParams {
    Params<T> f;
    const T* d_out;
    const float* d_fin;
    float *gu, *gdelta, *gz, *ginit;
    float* exits;    // per slot [D][S]: adjoint handed to the unit in front, then the one from behind
    float* part_bc;  // [cpb][tokens][G][2][S]
    float* part_A;   // per slot [D][S]
    float* part_d;   // per slot [2][D]: skip, delta_bias
};

// This lane's elements of a tile, raw: tokens TB e + tok of its channels.
template <typename T, typename Sh>
struct Elements {
    T u[Sh::NB][Sh::OWN], d[Sh::NB][Sh::OWN], z[Sh::NB][Sh::OWN], o[Sh::NB][Sh::OWN];
    // tokens behind the end repeat the last
    __device__ __forceinline__ void fetch(const BwdParams<T>& p, int t, int end, const int (&own)[Sh::OWN])
    {
#pragma unroll
        for (int e = 0; e < Sh::NB; ++e) {
            const int tt = t + e * Sh::TB;
            const size_t at = (size_t)(tt < end ? tt : end - 1) * p.f.D;
#pragma unroll
            for (int i = 0; i < Sh::OWN; ++i) {
                u[e][i] = p.f.u[at + own[i]];
                d[e][i] = p.f.delta[at + own[i]];
                o[e][i] = p.d_out[at + own[i]];
                if (p.f.z) z[e][i] = p.f.z[at + own[i]];
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ float one(const T& v)
{
    float x[1];
    load_vec<1>(&v, x);
    return x[0];
}

// A block's place: its unit and channels.
struct Place {
    int slot, g, gb, c0, nch, n, seg, t0, end;
    bool last, found;
    template <typename T>
    __device__ __forceinline__ Place(const Params<T>& p, int CH)
    {
        const int across = p.G * p.cpb;
        slot = blockIdx.x / across;
        gb = (int)(blockIdx.x % across);
        g = gb / p.cpb;
        gb -= g * p.cpb;
        nch = p.Dg - gb * CH < CH ? p.Dg - gb * CH : CH;
        c0 = g * p.Dg + gb * CH;
        found = p.units.locate(slot, n, seg, last, t0, end);
    }
};

// End state from zero, sum of dt and handed-on adjoint of every unit.
template <typename T, int LANES>
__global__ void __launch_bounds__(32)
kda_ssm_bwd_carry_kernel(BwdParams<T> p)
{
    using Sh = Carry<LANES>;
    constexpr int L = Sh::L, TT = Sh::TT, SP = Sh::SP, TB = Sh::TB, NB = Sh::NB, OWN = Sh::OWN, PAIRS = Sh::PAIRS;
    __shared__ __align__(16) float2 s_dt[TT][PAIRS][2];  // dt, dt u
    __shared__ __align__(16) float s_dy[TT][PAIRS][2];
    __shared__ __align__(16) float s_B[TT * SP], s_C[TT * SP];
    const Place at(p.f, Sh::CH);
    if (!at.found || (at.seg == 0 && at.last)) return;
    const int lane = threadIdx.x & 31, pair = lane / L, s0 = lane % L * 4;
    float A[2][4], h[2][4], P[2][4], R[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int c = pair * 2 + r < at.nch ? pair * 2 + r : at.nch - 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            A[r][i] = s0 + i < p.f.S ? rate(p.f.A[(size_t)(at.c0 + c) * p.f.S + s0 + i]) : 0.f;
            h[r][i] = R[r][i] = 0.f;
            P[r][i] = 1.f;
        }
    }
    const int tok = fold_index<Sh::BITS>(lane, 2);
    const bool owner = L == 1 || lane % L < 2 * TB;
    int own[OWN];
    float bias[OWN], dt_sum[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int c = pair * 2 + (OWN == 2 ? o : lane & 1);
        own[o] = at.c0 + (c < at.nch ? c : at.nch - 1);
        bias[o] = p.f.delta_bias ? p.f.delta_bias[own[o]] : 0.f;
        dt_sum[o] = 0.f;
    }
    Elements<T, Sh> el;
    StateRows<T, Sh, true> bc;
    el.fetch(p, at.t0 + tok, at.end, own);
    bc.load(p.f, at.t0, at.end, at.g, lane);
    for (int t = at.t0; t < at.end; t += TT) {
#pragma unroll
        for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int tt = e * TB + tok, c = OWN == 2 ? o : lane & 1;
                float dt = one(el.d[e][o]) + bias[o];
                if (p.f.softplus) dt = softplus(dt);
                if (t + tt >= at.end) dt = 0.f;  // a step of nothing
                float dy = t + tt < at.end ? one(el.o[e][o]) : 0.f;
                if (p.f.z) dy *= silu(one(el.z[e][o]));
                if (owner) {
                    dt_sum[o] += dt;
                    s_dt[tt][pair][c] = make_float2(dt, t + tt < at.end ? dt * one(el.u[e][o]) : 0.f);
                    s_dy[tt][pair][c] = t + tt < at.end ? dy : 0.f;
                }
            }
        bc.put(s_B, s_C, lane);
        if (t + TT < at.end) {
            el.fetch(p, t + TT + tok, at.end, own);
            bc.load(p.f, t + TT, at.end, at.g, lane);
        }
        __syncwarp();
        const float4 d0 = *reinterpret_cast<const float4*>(&s_dt[0][pair][0]);
        const float mean[2] = {mean_error(d0.x, slowest(A[0])), mean_error(d0.z, slowest(A[1]))};
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            const float4 dd = *reinterpret_cast<const float4*>(&s_dt[tt][pair][0]);
            const float2 dy = *reinterpret_cast<const float2*>(&s_dy[tt][pair][0]);
            const float4 B4 = *reinterpret_cast<const float4*>(&s_B[tt * SP + s0]);
            const float4 C4 = *reinterpret_cast<const float4*>(&s_C[tt * SP + s0]);
            const float B[4] = {B4.x, B4.y, B4.z, B4.w}, C[4] = {C4.x, C4.y, C4.z, C4.w};
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = decay(r ? dd.z : dd.x, A[r][i], mean[r]);
                    h[r][i] = fmaf(a, h[r][i], (r ? dd.w : dd.y) * B[i]);
                    P[r][i] *= a;
                    R[r][i] = fmaf(P[r][i], (r ? dy.y : dy.x) * C[i], R[r][i]);
                }
        }
        __syncwarp();
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (pair * 2 + r < at.nch) {
            const size_t row = ((size_t)at.slot * p.f.D + at.c0 + pair * 2 + r) * p.f.S + s0;
            const bool whole = p.f.vec_s && s0 < p.f.S;
            store4(p.f.ends + row, h[r], whole, p.f.S - s0);
            store4(p.exits + row, R[r], whole, p.f.S - s0);
        }
    // a channel's tokens lie with the lanes of its parity
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
#pragma unroll
        for (int i = 2; i < L; i <<= 1) dt_sum[o] += __shfl_xor_sync(0xffffffffu, dt_sum[o], i);
        const int c = pair * 2 + (OWN == 2 ? o : lane & 1);
        if (c < at.nch && lane % L < 2) p.f.steps[(size_t)at.slot * p.f.D + at.c0 + c] = dt_sum[o];
    }
}

// The entry states (the first half of the blocks), and the adjoint that enters
// every unit from behind, in place of the one it hands on: c <- exp(A sum dt) c
// + R, from a sequence's last unit to its first.
__global__ void __launch_bounds__(256)
kda_ssm_bwd_chain_kernel(const float* __restrict__ A, const float* __restrict__ init, float* ends,
                         const float* __restrict__ d_fin, float* exits, const float* __restrict__ steps,
                         Units units, int D, int S, int span)
{
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half) {
        chain_states(blockIdx.x, A, init, ends, steps, units, D, S, span);
        return;
    }
    const size_t DS = (size_t)D * S;
    const int per = (int)((DS + span - 1) / span), n = (blockIdx.x - half) / per;
    const int cnt = units.count(n);
    if (cnt == 1) return;  // a sequence's last unit has the final state's adjoint
    const int first = units.first(n);
    const size_t i0 = (size_t)((blockIdx.x - half) % per) * span, i1 = i0 + span < DS ? i0 + span : DS;
    for (size_t i = i0 + threadIdx.x; i < i1; i += 256) {
        const float a = rate(A[i]);
        float c = d_fin ? d_fin[(size_t)n * DS + i] : 0.f;
        float* e = exits + (size_t)first * DS + i;
        const float* st = steps + (size_t)first * D + (unsigned)i / (unsigned)S;
        constexpr int U = 8;
        for (int k = cnt - 1; k >= 0; k -= U) {
            float r[U], dt[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const bool ok = k - j > 0;  // the first unit hands on to no one
                r[j] = ok ? e[(size_t)(k - j) * DS] : 0.f;
                dt[j] = ok ? st[(size_t)(k - j) * D] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (k - j >= 0) {
                    e[(size_t)(k - j) * DS] = c;
                    c = fmaf(layer::ex2(a * dt[j]), c, r[j]);
                }
        }
    }
}

// Shared memory of the main kernel, in floats.
template <typename Sh>
struct BwdSpace {
    static constexpr int kB = 0;                                            // [TT][SP]
    static constexpr int kC = kB + Sh::TT * Sh::SP;                          // [TT][SP]
    static constexpr int kDt = kC + Sh::TT * Sh::SP;                         // per warp [TT][PAIRS][2]: dt, dt u
    static constexpr int kDy = kDt + Sh::WARPS * Sh::TT * Sh::PAIRS * 4;     // per warp [TT][PAIRS][2]
    static constexpr int kEl = kDy + Sh::WARPS * Sh::TT * Sh::PAIRS * 2;     // per thread [NB OWN][4]: its elements
    static constexpr int kM = kEl + Sh::THREADS * Sh::NB * Sh::OWN * 4;      // per thread [TT / 4][8]: states
    static constexpr int kW = kM + Sh::THREADS * Sh::TT / 4 * 8;             // per warp [TT][2][SP]: dB, dC
    static constexpr int kAll = kW + Sh::WARPS * Sh::TT * 2 * Sh::SP;
};

template <typename T, int LANES>
__global__ void __launch_bounds__(128, 2)
kda_ssm_bwd_kernel(BwdParams<T> p)
{
    using Sh = Bwd<LANES>;
    using Sp = BwdSpace<Sh>;
    constexpr int L = Sh::L, TT = Sh::TT, SP = Sh::SP, TB = Sh::TB, NB = Sh::NB, OWN = Sh::OWN, PAIRS = Sh::PAIRS;
    constexpr int THREADS = Sh::THREADS, WARPS = Sh::WARPS, BPG = 4 / TB;  // batches per four tokens
    extern __shared__ __align__(16) float smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float* s_B = smem + Sp::kB;
    float* s_C = smem + Sp::kC;
    float4* s_dt = reinterpret_cast<float4*>(smem + Sp::kDt) + warp * TT * PAIRS;  // of a pair's two channels
    float2* s_dy = reinterpret_cast<float2*>(smem + Sp::kDy) + warp * TT * PAIRS;
    float4* s_el = reinterpret_cast<float4*>(smem + Sp::kEl) + tid;                // stride THREADS
    float4* s_m = reinterpret_cast<float4*>(smem + Sp::kM) + tid;
    float* s_w = smem + Sp::kW;
    const int D = p.f.D, S = p.f.S;
    const size_t DS = (size_t)D * S;
    const Place at(p.f, Sh::CH);
    const int pair = lane / L, s0 = lane % L * 4, ch0 = warp * Sh::WCH + pair * 2;  // the pair's first channel
    const bool whole = p.f.vec_s && s0 < S;
    if (!at.found) {
        // an empty slot adds nothing to the parameters' gradients
        for (int c = tid; c < at.nch; c += THREADS) {
            for (int s = 0; s < S; ++s) p.part_A[(size_t)at.slot * DS + (size_t)(at.c0 + c) * S + s] = 0.f;
            p.part_d[(size_t)at.slot * 2 * D + at.c0 + c] = p.part_d[((size_t)at.slot * 2 + 1) * D + at.c0 + c] = 0.f;
        }
        return;
    }
    // tiles of all units, numbered so that no count of earlier ones is needed
    const int tile0 = at.t0 / TT + at.slot, tiles = (at.end - at.t0 + TT - 1) / TT;

    float A[2][4], c[2][4], dA[2][4];
    size_t row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int ch = ch0 + r < at.nch ? ch0 + r : at.nch - 1;
        row[r] = (size_t)(at.c0 + ch) * S + s0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool ok = s0 + i < S;
            A[r][i] = ok ? rate(p.f.A[row[r] + i]) : 0.f;
            c[r][i] = dA[r][i] = 0.f;
            if (ok) {
                if (p.f.ends && !at.last) c[r][i] = p.exits[(size_t)at.slot * DS + row[r] + i];
                else if (p.d_fin) c[r][i] = p.d_fin[(size_t)at.n * DS + row[r] + i];
            }
        }
    }
    // this lane's elements
    const int tok = fold_index<Sh::BITS>(lane, 2);
    const bool owner = L == 1 || lane % L < 2 * TB;
    int own[OWN];
    float bias[OWN], skip[OWN], sum_skip[OWN], sum_bias[OWN];
    bool mine[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int ch = ch0 + (OWN == 2 ? o : lane & 1);
        mine[o] = owner && ch < at.nch;
        own[o] = at.c0 + (ch < at.nch ? ch : at.nch - 1);
        bias[o] = p.f.delta_bias ? p.f.delta_bias[own[o]] : 0.f;
        skip[o] = p.f.skip ? p.f.skip[own[o]] : 0.f;
        sum_skip[o] = sum_bias[o] = 0.f;
    }

    Elements<T, Sh> el;
    StateRows<T, Sh, true> bc;
    float h[2][4], mean[2];
    auto fetch = [&](int k) {
        const int t = at.t0 + k * TT;
        el.fetch(p, t + tok, at.end, own);
        bc.load(p.f, t, at.end, at.g, tid);
        const float* e = p.f.entries + (size_t)(tile0 + k) * DS;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (whole) {
                load_vec<4>(e + row[r], h[r]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[r][i] = s0 + i < S ? e[row[r] + i] : 0.f;
            }
        }
    };
    auto advance = [&](int tt) {
        const float4 dd = s_dt[tt * PAIRS + pair];
        const float4 B4 = *reinterpret_cast<const float4*>(&s_B[tt * SP + s0]);
        const float B[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[r][i] = fmaf(decay(r ? dd.z : dd.x, A[r][i], mean[r]), h[r][i], (r ? dd.w : dd.y) * B[i]);
    };

    if (tiles > 0) fetch(tiles - 1);
    for (int k = tiles - 1; k >= 0; --k) {
        const int t = at.t0 + k * TT;
        const int fours = at.end - t < TT ? (at.end - t + 3) / 4 : TT / 4;  // with a token in them
        // what depends on (token, channel) alone
#pragma unroll
        for (int e = 0; e < NB; ++e)
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int tt = e * TB + tok, ch = OWN == 2 ? o : lane & 1;
                const bool in = t + tt < at.end && ch0 + ch < at.nch;  // others have no step and no adjoint
                const float x = one(el.u[e][o]), raw = one(el.d[e][o]) + bias[o], dout = one(el.o[e][o]);
                float slope = 1.f, dt = raw, dy = dout, dz = 0.f;
                if (p.f.softplus) dt = softplus(raw, slope);
                if (p.f.z) {
                    const float zz = one(el.z[e][o]), sg = sigmoid(zz);
                    dz = dout * (sg * fmaf(zz, 1.f - sg, 1.f));
                    dy = dout * (zz * sg);
                }
                if (!in) dt = 0.f;
                if (owner) {
                    reinterpret_cast<float2*>(s_dt)[(tt * PAIRS + pair) * 2 + ch] = make_float2(dt, in ? dt * x : 0.f);
                    reinterpret_cast<float*>(s_dy)[(tt * PAIRS + pair) * 2 + ch] = in ? dy : 0.f;
                    s_el[(e * OWN + o) * THREADS] = make_float4(x, dy, dz, slope);
                }
            }
        bc.put(s_B, s_C, tid);
        __syncthreads();
        mean[0] = mean_error(s_dt[pair].x, slowest(A[0]));
        mean[1] = mean_error(s_dt[pair].z, slowest(A[1]));
        // the states in front of every four tokens
#pragma unroll
        for (int q = 0; q < TT / 4; ++q) {
            s_m[(2 * q) * THREADS] = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
            s_m[(2 * q + 1) * THREADS] = make_float4(h[1][0], h[1][1], h[1][2], h[1][3]);
            if (q + 1 >= fours) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) advance(q * 4 + j);
        }
        if (k > 0) fetch(k - 1);
        // a tile's sum of dA first: long sums of small terms keep their digits
        float dA_t[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) dA_t[r][i] = 0.f;
#pragma unroll 1
        for (int q = fours - 1; q >= 0; --q) {
            const float4 m0 = s_m[(2 * q) * THREADS], m1 = s_m[(2 * q + 1) * THREADS];
            const float b[2][4] = {{m0.x, m0.y, m0.z, m0.w}, {m1.x, m1.y, m1.z, m1.w}};
            float hs[4][2][4], as[4][2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 dd = s_dt[(q * 4 + j) * PAIRS + pair];
                const float4 B4 = *reinterpret_cast<const float4*>(&s_B[(q * 4 + j) * SP + s0]);
                const float B[4] = {B4.x, B4.y, B4.z, B4.w};
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        as[j][r][i] = decay(r ? dd.z : dd.x, A[r][i], mean[r]);
                        hs[j][r][i] = fmaf(as[j][r][i], j ? hs[j > 0 ? j - 1 : 0][r][i] : b[r][i], (r ? dd.w : dd.y) * B[i]);
                    }
            }
#pragma unroll
            for (int eb = BPG - 1; eb >= 0; --eb) {
                float o[3][2 * TB];  // g . B, sum g a h A, C . h of [channel][token]
#pragma unroll
                for (int jj = TB - 1; jj >= 0; --jj) {
                    const int j = eb * TB + jj, tt = q * 4 + j;
                    const float4 dd = s_dt[tt * PAIRS + pair];
                    const float2 dy2 = s_dy[tt * PAIRS + pair];
                    const float4 B4 = *reinterpret_cast<const float4*>(&s_B[tt * SP + s0]);
                    const float4 C4 = *reinterpret_cast<const float4*>(&s_C[tt * SP + s0]);
                    const float B[4] = {B4.x, B4.y, B4.z, B4.w}, C[4] = {C4.x, C4.y, C4.z, C4.w};
                    float bc8[8];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float dt = r ? dd.z : dd.x, du = r ? dd.w : dd.y, dy = r ? dy2.y : dy2.x;
                        float2 sB = both(0.f), sA = sB, sC = sB;
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            // the recurrence in scalars (shorter latency), the sums in pairs
                            const float g0 = fmaf(C[i], dy, c[r][i]), g1 = fmaf(C[i + 1], dy, c[r][i + 1]);
                            c[r][i] = as[j][r][i] * g0;
                            c[r][i + 1] = as[j][r][i + 1] * g1;
                            const float2 gg = make_float2(g0, g1), h2 = make_float2(hs[j][r][i], hs[j][r][i + 1]);
                            const float2 hp = j ? make_float2(hs[j > 0 ? j - 1 : 0][r][i], hs[j > 0 ? j - 1 : 0][r][i + 1])
                                                : make_float2(b[r][i], b[r][i + 1]);
                            const float2 w = mul2(make_float2(c[r][i], c[r][i + 1]), hp);
                            const float2 da = fma2(w, both(dt), make_float2(dA_t[r][i], dA_t[r][i + 1]));
                            dA_t[r][i] = da.x;
                            dA_t[r][i + 1] = da.y;
                            sB = fma2(gg, make_float2(B[i], B[i + 1]), sB);
                            sA = fma2(w, make_float2(A[r][i], A[r][i + 1]), sA);
                            sC = fma2(h2, make_float2(C[i], C[i + 1]), sC);
                            const float2 pb = r ? fma2(gg, both(du), make_float2(bc8[i], bc8[i + 1])) : mul2(gg, both(du));
                            const float2 pc = r ? fma2(h2, both(dy), make_float2(bc8[4 + i], bc8[5 + i])) : mul2(h2, both(dy));
                            bc8[i] = pb.x;
                            bc8[i + 1] = pb.y;
                            bc8[4 + i] = pc.x;
                            bc8[5 + i] = pc.y;
                        }
                        const float gB = sB.x + sB.y, wA = sA.x + sA.y, hC = sC.x + sC.y;
                        o[0][r * TB + jj] = gB;
                        o[1][r * TB + jj] = wA;
                        o[2][r * TB + jj] = hC;
                    }
                    // over the warp's pairs
                    fold<8, PAIRS, L>(bc8, lane);
                    constexpr int KEEP = PAIRS >= 8 ? 1 : 8 / PAIRS;
                    constexpr int BITS = PAIRS >= 8 ? 3 : (PAIRS == 4 ? 2 : (PAIRS == 2 ? 1 : 0));
                    if (PAIRS <= 8 || lane / L < 8) {
                        const int first = fold_index<BITS>(lane, L) * KEEP;  // of {B: 0..3, C: 4..7}
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) {
                            const int v = first + i;
                            s_w[((warp * TT + tt) * 2 + (v >> 2)) * SP + s0 + (v & 3)] = bc8[i];
                        }
                    }
                }
                // over a pair's lanes, each left with its own element
                fold<2 * TB, L, 1>(o[0], lane);
                fold<2 * TB, L, 1>(o[1], lane);
                if (p.f.z) fold<2 * TB, L, 1>(o[2], lane);
                const int e = q * BPG + eb, tt = e * TB + tok;
#pragma unroll
                for (int i = 0; i < OWN; ++i) {
                    if (!mine[i] || t + tt >= at.end) continue;
                    const float4 v = s_el[(e * OWN + i) * THREADS];  // u, dy, d_out silu'(z), softplus'
                    const float dt = reinterpret_cast<float2*>(s_dt)[(tt * PAIRS + pair) * 2 + (OWN == 2 ? i : lane & 1)].x;
                    const size_t to = (size_t)(t + tt) * D + own[i];
                    if (p.f.z) p.gz[to] = v.z * fmaf(skip[i], v.x, o[2][i]);
                    p.gu[to] = fmaf(dt, o[0][i], skip[i] * v.y);
                    sum_skip[i] = fmaf(v.y, v.x, sum_skip[i]);
                    const float gd = fmaf(v.x, o[0][i], o[1][i] * kLn2) * v.w;
                    sum_bias[i] += gd;
                    p.gdelta[to] = gd;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) dA[r][i] += dA_t[r][i];
        __syncthreads();
        // dB and dC of this block's channels
        for (int q = tid; q < TT * 2 * SP; q += THREADS) {
            const int j = q / (2 * SP), ws = q - j * 2 * SP, s = ws % SP;
            if (t + j >= at.end || s >= S) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) sum += s_w[w * TT * 2 * SP + q];
            p.part_bc[((((size_t)at.gb * p.f.units.s.total + t + j) * p.f.G + at.g) * 2 + ws / SP) * S + s] = sum;
        }
    }

#pragma unroll
    for (int r = 0; r < 2; ++r)
        if (ch0 + r < at.nch) {
            store4(p.part_A + (size_t)at.slot * DS + row[r], dA[r], whole, S - s0);
            if (at.seg == 0 && p.ginit) store4(p.ginit + (size_t)at.n * DS + row[r], c[r], whole, S - s0);
        }
    // a channel's tokens lie with the lanes of its parity
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
#pragma unroll
        for (int i = 2; i < L; i <<= 1) {
            sum_skip[o] += __shfl_xor_sync(0xffffffffu, sum_skip[o], i);
            sum_bias[o] += __shfl_xor_sync(0xffffffffu, sum_bias[o], i);
        }
        const int ch = ch0 + (OWN == 2 ? o : lane & 1);
        if (ch < at.nch && lane % L < 2) {
            p.part_d[(size_t)at.slot * 2 * D + at.c0 + ch] = sum_skip[o];
            p.part_d[((size_t)at.slot * 2 + 1) * D + at.c0 + ch] = sum_bias[o];
        }
    }
}

// The first `bc_blocks` blocks: grad_B and grad_C [tokens][G][S] from the
// channel blocks' sums [cpb][tokens][G][2][S]; rows in front of the first
// sequence or behind the last belong to none and are left alone.  The others:
// grad_A [D][S] (i < DS), then grad_skip and grad_delta_bias [D], from the
// units' sums, 32 values per block, eight lanes over the units.
__global__ void __launch_bounds__(256)
kda_ssm_bwd_sums_kernel(const float* __restrict__ part_bc, float* __restrict__ grad_B, float* __restrict__ grad_C,
                        Seqs seqs, int G, int cpb, int bc_blocks, const float* __restrict__ part_A,
                        const float* __restrict__ part_d, float* __restrict__ grad_A,
                        float* __restrict__ grad_skip, float* __restrict__ grad_bias, int D, int S, int slots)
{
    __shared__ float red[8][33];
    if ((int)blockIdx.x < bc_blocks) {
        const long long all = (long long)seqs.total * G * 2 * S;
        const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
        if (i >= all) return;
        const long long row = i / (2 * S), t = row / G;
        const int ws = (int)(i - row * 2 * S);
        if (seqs.cu && (t < seqs.start(0) || t >= seqs.start(seqs.N))) return;
        float s = 0.f;
#pragma unroll 8
        for (int k = 0; k < cpb; ++k) s += part_bc[(size_t)k * all + i];
        if (ws < S) grad_B[row * S + ws] = s;
        else grad_C[row * S + ws - S] = s;
        return;
    }
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long long DS = (long long)D * S, i = (long long)(blockIdx.x - bc_blocks) * 32 + lane;
    const bool isA = i < DS, live = i < DS + 2 * D;
    const float* src = isA ? part_A + i : part_d + (i - DS);
    const size_t stride = isA ? (size_t)DS : (size_t)2 * D;
    float s = 0.f;
    if (live)
#pragma unroll 4
        for (int k = y; k < slots; k += 8) s += src[(size_t)k * stride];
    red[y][lane] = s;
    __syncthreads();
    if (y == 0 && live) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += red[k][lane];
        if (isA) grad_A[i] = t;
        else if (i < DS + D) {
            if (grad_skip) grad_skip[i - DS] = t;
        } else if (grad_bias) {
            grad_bias[i - DS - D] = t;
        }
    }
}

// Sequences are cut where the chains give the SMs fewer warps than this: another
// walk then goes over most tokens, a fifth of the whole.  Forward and backward of
// 4096 channels, 16 states, bf16, whole against cut: 1 x 4096 tokens (1.7 warps an
// SM) 2133 and 881 us, 2 x 2048 (3.5) 1088 and 944, 3 x 1365 (5.2) 970 and 993, 4 x
// 1024 (6.9) 734 and 1003.  Units for 16 warps of at least 32 tokens against 8 and
// 64: 17245 x 640 628 against 676 us, small calls 5 to 20 % less.
constexpr int kBwdFewWarps = 5, kBwdWantWarps = 16, kBwdShortest = 32;

struct Layout {
    Cut c;
    size_t slots, tiles, ends, exits, steps, entries, bc, A, d, total;
};

Layout layout_of(int B, int T, int D, int S, int G, int N, int packed)
{
    Layout l = {};
    const size_t tokens = (size_t)B * T, DS = (size_t)D * S, L = lanes_of(S);
    l.c = cut_of(B, T, N, packed, (double)D * L / 64.0, kBwdFewWarps, kBwdWantWarps, kBwdShortest, 2 * kBwdShortest);
    l.slots = (size_t)slots_of(B, T, N, packed, l.c.len);
    const size_t CH = 256 / L, cpb = ((size_t)(D / G) + CH - 1) / CH, TT = L >= 4 ? 16 : 4 * L;  // as in Bwd<L>
    l.tiles = tokens / TT + l.slots + 1;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += round256(floats * 4);
        return here;
    };
    l.ends = take(l.c.cut ? l.slots * DS : 0);
    l.exits = take(l.c.cut ? l.slots * DS : 0);
    l.steps = take(l.c.cut ? l.slots * D : 0);
    l.entries = take(l.tiles * DS);
    l.bc = take(cpb * tokens * G * 2 * S);
    l.A = take(l.slots * DS);
    l.d = take(l.slots * 2 * D);
    l.total = at;
    return l;
}

template <typename T, int L>
cudaError_t bwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    static_assert(Bwd<L>::CH == 256 / L && Bwd<L>::TT == Shape<L, 16, 32>::TT, "workspace layout");
    const Layout l = layout_of(a.B, a.T, a.D, a.S, a.G, a.N, a.cu_seqlens != nullptr);
    char* ws = (char*)a.workspace;
    BwdParams<T> p = {};
    p.f = params_of<T>(a, l.c.len, Bwd<L>::CH);
    p.d_out = (const T*)a.d_out;
    p.d_fin = a.d_final_state;
    p.gu = a.grad_u;
    p.gdelta = a.grad_delta;
    p.gz = a.grad_z;
    p.ginit = a.grad_initial_state;
    if (l.c.cut) {
        p.f.ends = (float*)(ws + l.ends);
        p.exits = (float*)(ws + l.exits);
        p.f.steps = (float*)(ws + l.steps);
    }
    p.f.entries = (float*)(ws + l.entries);
    p.part_bc = (float*)(ws + l.bc);
    p.part_A = (float*)(ws + l.A);
    p.part_d = (float*)(ws + l.d);
    const long long blocks = (long long)l.slots * p.f.G * p.f.cpb;
    const ChainGrid chain = chain_grid(a.D, a.S, a.N);
    const long long bc = ((long long)a.B * a.T * a.G * 2 * a.S + 255) / 256;
    const long long params = ((long long)a.D * (a.S + 2) + 31) / 32;
    if (blocks > INT32_MAX || 2 * chain.blocks > INT32_MAX || bc + params > INT32_MAX) return cudaErrorInvalidConfiguration;
    constexpr size_t smem = sizeof(float) * BwdSpace<Bwd<L>>::kAll;
    if (cudaError_t e = cudaFuncSetAttribute(kda_ssm_bwd_kernel<T, L>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem))
        return e;
    if (blocks > 0) {
        if (l.c.cut) {
            BwdParams<T> q = p;
            q.f.cpb = (q.f.Dg + Carry<L>::CH - 1) / Carry<L>::CH;
            const long long carry = (long long)l.slots * q.f.G * q.f.cpb;
            if (carry > INT32_MAX) return cudaErrorInvalidConfiguration;
            kda_ssm_bwd_carry_kernel<T, L><<<(unsigned)carry, 32, 0, st>>>(q);
            if (cudaError_t e = cudaGetLastError()) return e;
            kda_ssm_bwd_chain_kernel<<<(unsigned)(2 * chain.blocks), 256, 0, st>>>(
                a.A, a.initial_state, p.f.ends, a.d_final_state, p.exits, p.f.steps, p.f.units, a.D, a.S,
                chain.span);
            if (cudaError_t e = cudaGetLastError()) return e;
        }
        if (cudaError_t e = launch_ssm_entries(a, l.c.len, p.f.ends, p.f.entries, dtype, st)) return e;
        kda_ssm_bwd_kernel<T, L><<<(unsigned)blocks, Bwd<L>::THREADS, smem, st>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_ssm_bwd_sums_kernel<<<(unsigned)(bc + params), 256, 0, st>>>(
        p.part_bc, a.grad_B, a.grad_C, p.f.units.s, a.G, p.f.cpb, (int)bc, p.part_A, p.part_d, a.grad_A, a.grad_skip,
        a.grad_delta_bias, a.D, a.S, (int)l.slots);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    switch (lanes_of(a.S)) {
        case 1: return bwd<T, 1>(a, dtype, st);
        case 2: return bwd<T, 2>(a, dtype, st);
        case 4: return bwd<T, 4>(a, dtype, st);
        case 8: return bwd<T, 8>(a, dtype, st);
        case 16: return bwd<T, 16>(a, dtype, st);
        case 32: return bwd<T, 32>(a, dtype, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

size_t scan_bwd_workspace(int B, int T, int D, int S, int G, int N, int packed, kda_dtype)
{
    return layout_of(B, T, D, S, G, N, packed).total;
}

cudaError_t launch_scan_bwd(const ScanArgs& a, kda_dtype dtype, cudaStream_t st)
{
    return dtype == KDA_DTYPE_BF16 ? by_states<__nv_bfloat16>(a, dtype, st) : by_states<float>(a, dtype, st);
}

}  // namespace kda
