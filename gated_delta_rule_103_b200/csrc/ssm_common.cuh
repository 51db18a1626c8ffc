// Shared device code of the state-space scan's kernels.
//
//     dt = delta + bias, or softplus of it;   a = exp(dt A[d, s])
//     h[d, s] = a h[d, s] + dt u B[g, s];     y = sum_s h C[g, s] + skip u
//     out = y, or y silu(z)
//
// States are padded to 4 L with A = B = C = 0 behind S.
#pragma once

#include <cfloat>

#include "layer.h"
#include "layer_common.cuh"

namespace kda {
namespace ssm {

using namespace layer;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// How a warp's lanes share the work of every pass over tokens: L lanes share
// two channels and hold four states of each, so that what a lane reads of B and
// C from shared memory serves eight states (a 16-byte read returns 512 bytes to
// a warp's registers, four clocks of an SM's 128 bytes; one channel a lane would
// spend as long on them as on the exponentials).  What depends on (token,
// channel) alone is worked out once, by the lane that also ends up with that
// element's sums: in a batch of TB tokens, lane l has channel l % 2 of its pair
// and one token, and the fold over the lanes of the batch's 2 TB sums leaves
// each lane with its own (lanes from 2 TB on have none).
template <int LANES, int BATCH, int BLOCK>
struct Shape {
    static constexpr int L = LANES, THREADS = BLOCK, WARPS = BLOCK / 32;
    static constexpr int PAIRS = 32 / L, WCH = 2 * PAIRS, CH = WCH * WARPS;  // channels of a warp, of a block
    static constexpr int SP = 4 * L;                                        // padded states
    static constexpr int TB = L >= 2 ? (L / 2 < BATCH ? L / 2 : BATCH) : 1;  // tokens per batch
    static constexpr int TT = L >= 4 ? 16 : 4 * L;                          // tokens per tile
    static constexpr int NB = TT / TB;                                      // batches per tile
    static constexpr int OWN = L == 1 ? 2 : 1;                              // elements of a lane per batch
    static constexpr int BITS = TB == 16 ? 4 : TB == 8 ? 3 : TB == 4 ? 2 : TB == 2 ? 1 : 0;
};

// Two fp32 values in one instruction: half the issue slots, the same time of the
// pipe and a longer latency.  For sums that nothing waits for; in the recurrence
// itself, with two warps per scheduler, pairs were slower (708 us against 538 on
// 4 x 4096 tokens of 4096 channels).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A log2 e, held finite: a state with A = -inf (an -exp(A_log) that overflowed)
// forgets at every step, but not at the steps of nothing behind a sequence's end
// (dt = 0), where 0 * -inf would be NaN.
__device__ __forceinline__ float rate(float A)
{
    const float a = A * kLog2e;
    return a < -FLT_MAX ? -FLT_MAX : a;
}

// The decay e^(dt A) of one token from A log2 e.  A state carries the mean error
// of its decays times the tokens it remembers, 1 / |x| with x = dt A.  The fast
// 2^x is low in the mean by 5e-9 to 7e-9 of its value for x from -2^-14 to -2^-9
// (1e-8 at -2^-18), by 1.1e-8 to 3.0e-8 from there to -1 (a million values an octave
// of x, read off the states after one token without input); a constant in the
// exponent takes the middle of that back, at no instruction: the product becomes a
// fused one.  Final states that remember 64, 256, 1024 and 4096 tokens are off by
// 3e-7, 1.0e-6, 0.9e-6 and 2.3e-6 (without a constant by 1.2e-6, 4.4e-6, 4.2e-6 and
// 1.5e-5; with 1.8e-8 for every x by 4e-7, 1.5e-6, 8.6e-6 and 3.5e-5).  Which of the
// two applies is settled for a tile and four states at a time, by the tile's first
// token and the slowest state (0 where states are padding): 1 to 2 % of the scan's
// time; one choice a decay cost the step 7 %.
constexpr float kMeanLong = 6e-9f * kLog2e, kMean = 2.2e-8f * kLog2e;
constexpr float kLongRate = -0.0027f * kLog2e;  // 2^-8.5
__device__ __forceinline__ float slowest(const float (&A)[4])
{
    return fmaxf(fmaxf(A[0], A[1]), fmaxf(A[2], A[3]));
}
__device__ __forceinline__ float mean_error(float dt, float slow) { return dt * slow > kLongRate ? kMeanLong : kMean; }
__device__ __forceinline__ float decay(float dt, float A, float mean) { return ex2(fmaf(dt, A, mean)); }

// log(1 + e^x) = max(x, 0) + log1p(w), w = e^-|x|.  log1p(w) = 2 artanh(r)
// with r = w / (2 + w) <= 1/3, by its power series to r^15 (the rest is below
// 3e-9 of it): small steps keep their relative precision, which log(1 + w)
// would lose.
__device__ __forceinline__ float softplus(float x)
{
    const float w = fast_exp(-fabsf(x));
    const float r = w * fast_rcp(2.f + w), q = r * r;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * r, p, fmaxf(x, 0.f));
}

// ... and its slope 1 / (1 + e^-x), which shares the exponential.
__device__ __forceinline__ float softplus(float x, float& slope)
{
    const float w = fast_exp(-fabsf(x)), r1 = fast_rcp(1.f + w);
    slope = x >= 0.f ? r1 : w * r1;
    return softplus(x);
}

// ... of two values, the series in packed arithmetic.
__device__ __forceinline__ float2 softplus2(float2 x)
{
    const float2 w = make_float2(fast_exp(-fabsf(x.x)), fast_exp(-fabsf(x.y)));
    const float2 r = mul2(w, make_float2(fast_rcp(2.f + w.x), fast_rcp(2.f + w.y))), q = mul2(r, r);
    float2 p = both(1.f / 15.f);
    p = fma2(p, q, both(1.f / 13.f));
    p = fma2(p, q, both(1.f / 11.f));
    p = fma2(p, q, both(1.f / 9.f));
    p = fma2(p, q, both(1.f / 7.f));
    p = fma2(p, q, both(1.f / 5.f));
    p = fma2(p, q, both(1.f / 3.f));
    p = fma2(p, q, both(1.f));
    return fma2(mul2(r, both(2.f)), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// Four values as they lie in memory, loaded before they are needed.
template <typename T> struct Raw4;
template <> struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void load_some(const float* p, int n)
    {
        v.x = n > 0 ? p[0] : 0.f;
        v.y = n > 1 ? p[1] : 0.f;
        v.z = n > 2 ? p[2] : 0.f;
        v.w = n > 3 ? p[3] : 0.f;
    }
    __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
};
template <> struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n)
    {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
        const uint32_t a = n > 0 ? h[0] : 0u, b = n > 1 ? h[1] : 0u, c = n > 2 ? h[2] : 0u, d = n > 3 ? h[3] : 0u;
        v = make_uint2(a | b << 16, c | d << 16);
    }
    __device__ __forceinline__ void get(float (&x)[4]) const
    {
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    }
};

// Four values to memory, or the first n of them.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4], bool whole, int n)
{
    if (whole) {
        store_vec<4>(p, x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) {
            const float y[1] = {x[i]};
            store_vec<1>(p + i, y);
        }
}

template <typename T>
struct Params {
    const T* u;
    const T* delta;
    const float* A;
    const T* Bm;
    const T* Cm;
    const float* skip;
    const T* z;
    const float* delta_bias;
    const float* init;
    T* out;
    float* fin;
    float* ends;     // per slot [D][S]: end states, then entry states; nullptr: no unit follows another
    float* steps;    // per slot [D]: sum of dt
    float* entries;  // per tile [D][S]: state at the tile's entry (wanted by the backward pass)
    Units units;
    int D, S, G, Dg, cpb;  // channels, states, groups, channels and blocks per group
    int vec_s;             // rows of states load in fours
    int softplus;
};

// Sums of NV values over LANES lanes that are `stride` apart.  While several
// values are left, a lane hands half of them over and keeps the other half
// (half as many shuffles as summing each on its own), so that at the end lane
// bits, first stage first, number the value a lane holds; then plain sums.
template <int NV, int LANES, int STRIDE>
__device__ __forceinline__ void fold(float (&v)[NV], int lane)
{
    if constexpr (LANES > 1) {
        if constexpr (NV > 1) {
            const bool up = (lane & STRIDE) != 0;
            float k[NV / 2];
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) {
                const float send = up ? v[i] : v[i + NV / 2];
                const float keep = up ? v[i + NV / 2] : v[i];
                k[i] = keep + __shfl_xor_sync(0xffffffffu, send, STRIDE);
            }
            fold<NV / 2, LANES / 2, STRIDE * 2>(k, lane);
#pragma unroll
            for (int i = 0; i < NV / 2; ++i) v[i] = k[i];
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], STRIDE);
            fold<1, LANES / 2, STRIDE * 2>(v, lane);
        }
    }
}
// the value numbered by the first `bits` lane bits from `stride` on
template <int BITS>
__device__ __forceinline__ int fold_index(int lane, int stride)
{
    int r = 0;
#pragma unroll
    for (int i = 0; i < BITS; ++i) r = r << 1 | ((lane & (stride << i)) ? 1 : 0);
    return r;
}

// B (and C) of one tile: raw loads (they stay in flight), then fp32 rows
// [token][SP] in shared memory.
template <typename T, typename Tl, bool kC>
struct StateRows {
    static constexpr int TT = Tl::TT, SQ = Tl::SP / 4, ONE = TT * SQ, ALL = (kC ? 2 : 1) * ONE;
    static constexpr int NB = (ALL + Tl::THREADS - 1) / Tl::THREADS;
    // whole rounds of the threads over B, then C: which is which is known at compile time
    static constexpr bool kRounds = ONE % Tl::THREADS == 0 && Tl::THREADS % SQ == 0;
    Raw4<T> r[NB];
    __device__ __forceinline__ void load(const Params<T>& p, int t0, int end, int g, int tid)
    {
        const int left = end - t0 < TT ? end - t0 : TT;
        const int s = (tid % SQ) * 4;
        if constexpr (kRounds) {
            constexpr int PER = ONE / Tl::THREADS, STEP = Tl::THREADS / SQ;
            const size_t at = ((size_t)(t0 + tid / SQ) * p.G + g) * p.S + s;
            const size_t step = (size_t)STEP * p.G * p.S;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int j = k % PER;
                r[k].zero();
                if (tid / SQ + j * STEP < left && s < p.S) {
                    const T* q = (k < PER ? p.Bm : p.Cm) + at + j * step;
                    if (p.vec_s) r[k].load(q);
                    else r[k].load_some(q, p.S - s);
                }
            }
        } else {
            static_assert(Tl::THREADS % SQ == 0, "state quads");
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int i = tid + k * Tl::THREADS, t = i % ONE / SQ;
                r[k].zero();
                if (i < ALL && t < left && s < p.S) {
                    const T* q = (kC && i >= ONE ? p.Cm : p.Bm) + ((size_t)(t0 + t) * p.G + g) * p.S + s;
                    if (p.vec_s) r[k].load(q);
                    else r[k].load_some(q, p.S - s);
                }
            }
        }
    }
    __device__ __forceinline__ void put(float* sB, float* sC, int tid) const
    {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = tid + k * Tl::THREADS;
            float* to;
            if constexpr (kRounds) {
                constexpr int PER = ONE / Tl::THREADS;
                to = (k < PER ? sB : sC) + (tid + k % PER * Tl::THREADS) * 4;
            } else {
                if (i >= ALL) break;
                to = (kC && i >= ONE ? sC : sB) + i % ONE * 4;
            }
            float x[4];
            r[k].get(x);
            *reinterpret_cast<float4*>(to) = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
};

// Entry states of the units of every (sequence, channel, state), in place of
// their end states: h <- exp(A sum dt) h + e, unit after unit.  256 threads,
// `span` values a block: one a thread, or four where there are blocks enough
// (most blocks of many short sequences find one unit and nothing to do).
struct ChainGrid {
    int span;
    long long blocks;
};
inline ChainGrid chain_grid(int D, int S, int N)
{
    const long long DS = (long long)D * S, blocks = (DS + 255) / 256 * N;
    ChainGrid c = {blocks > 32LL * sm_count() ? 1024 : 256, 0};
    c.blocks = (DS + c.span - 1) / c.span * N;
    return c;
}

__device__ __forceinline__ void chain_states(int block, const float* __restrict__ A,
                                             const float* __restrict__ init, float* ends,
                                             const float* __restrict__ steps, const Units& units, int D, int S,
                                             int span)
{
    const size_t DS = (size_t)D * S;
    const int per = (int)((DS + span - 1) / span), n = block / per;
    const int cnt = units.count(n);
    if (cnt == 1) return;  // a sequence's first unit begins from its initial state
    const int first = units.first(n);
    const size_t i0 = (size_t)(block % per) * span, i1 = i0 + span < DS ? i0 + span : DS;
    for (size_t i = i0 + threadIdx.x; i < i1; i += 256) {
        const float a = rate(A[i]);
        float h = init ? init[(size_t)n * DS + i] : 0.f;
        float* e = ends + (size_t)first * DS + i;
        const float* st = steps + (size_t)first * D + (unsigned)i / (unsigned)S;
        constexpr int U = 8;
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
}

// Lanes that share two channels of S states.
inline int lanes_of(int S)
{
    int l = 1;
    while (4 * l < S) l <<= 1;
    return l;
}

inline Units units_of(const int32_t* cu, int B, int T, int N, int len)
{
    Units u;
    u.s.cu = cu;
    u.s.N = N;
    u.s.T = T;
    u.s.total = B * T;
    u.len = len;
    u.per_seq = T > 0 ? (T + len - 1) / len : 1;
    return u;
}
inline long long slots_of(int B, int T, int N, int packed, int len)
{
    return packed ? (long long)B * T / len + N : (long long)N * (T > 0 ? (T + len - 1) / len : 1);
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// How the token axis is cut into units: `len` tokens each, a multiple of 16;
// cut: some sequence may have more than one.
struct Cut {
    int len;
    bool cut;
};
// Cut only where the chains (chain_warps warps a sequence) give the SMs under
// `few` warps each, then into units that give them `want`; no unit is shorter
// than `shortest` tokens, and no call of fewer than `least` is cut.
inline Cut cut_of(int B, int T, int N, int packed, double chain_warps, int few, int want, int shortest, int least)
{
    Cut c = {T > 0 ? (T + 15) / 16 * 16 : 16, false};
    const long long tokens = (long long)B * T;
    if (tokens == 0 || N == 0 || T < least) return c;
    const bool many = (double)sm_count() * few <= chain_warps * N;
    if (many && !packed) return c;
    const double units = (double)sm_count() * want / chain_warps;
    double len = (double)tokens / (units < 1.0 ? 1.0 : units);
    if (packed) {
        // The longest sequence is not known here, and the whole call would wait
        // for it: no unit is longer than the mean, and where there are many
        // chains none shorter (sequences of one length then stay whole).
        const double mean = (double)tokens / N;
        if (many || len > mean) len = mean;
    }
    long long l = ((long long)len + 15) / 16 * 16;
    if (l < shortest) l = shortest;
    if (l >= T) return c;
    c.len = (int)l;
    c.cut = true;
    return c;
}

template <typename T>
Params<T> params_of(const ScanArgs& a, int len, int CH)
{
    Params<T> p = {};
    p.u = (const T*)a.u;
    p.delta = (const T*)a.delta;
    p.A = a.A;
    p.Bm = (const T*)a.Bm;
    p.Cm = (const T*)a.Cm;
    p.skip = a.skip;
    p.z = (const T*)a.z;
    p.delta_bias = a.delta_bias;
    p.init = a.initial_state;
    p.out = (T*)a.out;
    p.fin = a.final_state;
    p.units = units_of(a.cu_seqlens, a.B, a.T, a.N, len);
    p.D = a.D;
    p.S = a.S;
    p.G = a.G;
    p.Dg = a.D / a.G;
    p.cpb = (p.Dg + CH - 1) / CH;
    p.vec_s = a.S % 4 == 0;
    p.softplus = a.softplus;
    return p;
}

// The forward walk with the state at every tile's entry as its only result.
cudaError_t launch_ssm_entries(const ScanArgs& a, int len, float* ends, float* entries, kda_dtype dtype,
                               cudaStream_t st);

}  // namespace ssm
}  // namespace kda
