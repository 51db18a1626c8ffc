// Shared device code of the state-space scan's kernels.
//
//     dt = delta + bias, or softplus of it;   a = exp(dt A[d, s])
//     h[d, s] = a h[d, s] + dt u B[g, s];     y = sum_s h C[g, s] + skip u
//     out = y, or y silu(z)
//
// Thread layout of every pass over tokens: a block of 256 threads takes 256 /
// L channels of one group; L neighbouring lanes share a channel and hold 4
// states each (S <= 4 L; states behind S have A = B = C = 0).  Tokens go by in
// tiles: what depends on (token, channel) alone is computed once per element
// and handed to the L lanes through shared memory.
#pragma once

#include "layer.h"
#include "layer_common.cuh"

namespace kda {
namespace ssm {

using namespace layer;

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int L, int TOKENS = (L == 1 ? 4 : L == 2 ? 8 : 16)>
struct Tile {
    static constexpr int CH = kThreads / L;            // channels per block
    static constexpr int TT = TOKENS;                  // tokens per tile
    static constexpr int SP = 4 * L;                   // padded states
    static constexpr int Q = CH / 4;                   // channel quads
    static constexpr int IPT = (TT * Q + kThreads - 1) / kThreads;     // quads per thread
    static constexpr int ROWS = kThreads / Q < TT ? kThreads / Q : TT;  // threads that share a quad
    static constexpr int YP = CH + 8;                  // padded row of per-(token, channel) results
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values in one instruction: half the issue slots of the products and
// sums that surround the exponentials.
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
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

// log(1 + e^x) = max(x, 0) + log1p(w), w = e^-|x|.  log1p(w) = 2 artanh(r)
// with r = w / (2 + w) <= 1/3, by its power series to r^15 (the rest is below
// 3e-9 of it): small steps keep their relative precision, which log(1 + w)
// would lose.
__device__ __forceinline__ float softplus(float x)
{
    const float w = __expf(-fabsf(x));
    const float r = __fdividef(w, 2.f + w), q = r * r;
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
    float* ends;   // per slot [D][S]: end states, then entry states; nullptr: no unit follows another
    float* steps;  // per slot [D]: sum of dt
    Units units;
    int D, S, G, Dg, cpb;  // channels, states, groups, channels and blocks per group
    int vec_d, vec_s;      // rows of channels, of states load in fours
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
    static constexpr int TT = Tl::TT, L = Tl::SP / 4, ALL = (kC ? 2 : 1) * TT * L;
    static constexpr int NB = (ALL + kThreads - 1) / kThreads;
    Raw4<T> r[NB];
    __device__ __forceinline__ void load(const Params<T>& p, long long t0, long long end, int g, int tid)
    {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = tid + k * kThreads;
            const int which = i / (TT * L), j = i - which * (TT * L);
            const long long t = t0 + j / L;
            const int s = (j % L) * 4;
            r[k].zero();
            if (i < ALL && t < end && s < p.S) {
                const T* q = (kC && which ? p.Cm : p.Bm) + ((size_t)t * p.G + g) * p.S + s;
                if (p.vec_s) r[k].load(q);
                else r[k].load_some(q, p.S - s);
            }
        }
    }
    __device__ __forceinline__ void put(float* sB, float* sC, int tid) const
    {
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const int i = tid + k * kThreads;
            const int which = i / (TT * L), j = i - which * (TT * L);
            if (i < ALL) {
                float x[4];
                r[k].get(x);
                *reinterpret_cast<float4*>((kC && which ? sC : sB) + j * 4) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
};

// Rows of one (token, channel) operand of one tile, raw.
template <typename T, typename Tl>
struct ChannelRows {
    Raw4<T> r[Tl::IPT];
    __device__ __forceinline__ void load(const T* base, const Params<T>& p, long long t0, long long end, int c0,
                                         int nch, int tid)
    {
#pragma unroll
        for (int k = 0; k < Tl::IPT; ++k) {
            const int i = tid + k * kThreads;
            const int t = i / Tl::Q, c = (i % Tl::Q) * 4;
            r[k].zero();
            if (t < Tl::TT && t0 + t < end && c < nch) {
                const T* q = base + (size_t)(t0 + t) * p.D + c0 + c;
                if (p.vec_d) r[k].load(q);
                else r[k].load_some(q, nch - c);
            }
        }
    }
};

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
    u.s.total = (long long)B * T;
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
// Cut only where the chains' warps (L lanes a channel) leave the SMs under
// `warps` warps each; no unit is shorter than `shortest` tokens.
inline Cut cut_of(int B, int T, int D, int S, int N, int packed, int warps, int shortest)
{
    Cut c = {T > 0 ? (T + 15) / 16 * 16 : 16, false};
    const long long tokens = (long long)B * T;
    if (tokens == 0 || N == 0) return c;
    const double chain_warps = (double)D * lanes_of(S) / 32.0;  // of one sequence
    const double units = (double)sm_count() * warps / chain_warps;
    double len = (double)tokens / (units < 1.0 ? 1.0 : units);
    if (packed) {
        // the longest sequence is not known here: no unit is longer than twice the mean
        const double mean = 2.0 * (double)tokens / N;
        if (len > mean) len = mean;
    } else if (len >= T) {
        return c;
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
    p.vec_d = p.Dg % 4 == 0;
    p.vec_s = a.S % 4 == 0;
    p.softplus = a.softplus;
    return p;
}

// Entry states of the units of every (sequence, channel, state), in place of
// their end states.
cudaError_t launch_ssm_chain(const float* A, const float* init, float* ends, const float* steps, const Units& units,
                             int D, int S, cudaStream_t st);

}  // namespace ssm
}  // namespace kda
