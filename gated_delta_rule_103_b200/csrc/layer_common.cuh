// Shared device code of the layer operators around the recurrences (short
// convolution, state-space scan, group norm): vector loads and stores in
// fp32, the activations, and where the tokens of a packed batch belong.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace kda {
namespace layer {

// V consecutive values as fp32.  V * sizeof(T) is 2, 4, 8 or 16 bytes and the
// address is aligned to it.
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[V])
{
    if constexpr (V == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else if constexpr (V == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[V])
{
    if constexpr (V == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    } else if constexpr (V == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    } else if constexpr (V == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
        x[0] = bf16_lo(v); x[1] = bf16_hi(v);
    } else {
        static_assert(V == 1, "vector width");
        x[0] = __bfloat162float(*p);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    } else {
        p[0] = x[0];
    }
}
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[V])
{
    if constexpr (V == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
    } else {
        static_assert(V == 1, "vector width");
        *p = __float2bfloat16_rn(x[0]);
    }
}

// V values as they lie in memory: loads that stay in flight in as few registers
// as the type allows.
template <typename T, int V>
struct Raw {
    alignas(sizeof(T) * V) T v[V];
    __device__ __forceinline__ void load(const T* p)
    {
        constexpr int N = (int)sizeof(T) * V;
        if constexpr (N == 16) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (N == 8) *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        else if constexpr (N == 4) *reinterpret_cast<uint32_t*>(v) = *reinterpret_cast<const uint32_t*>(p);
        else v[0] = p[0];
    }
    __device__ __forceinline__ void get(float (&x)[V]) const { load_vec<V>(v, x); }
};

// 2^x, e^x and 1 / x in one or two instructions each, subnormals taken as zero.
// 2^x is good to some 2^-22 of its value and 1 / x to 2^-23; e^x to 2^-22 + 1.2
// |x| 2^-24, since the product x log2 e and the constant are rounded.  fp32 calls
// use them too: the sum delta + bias in front of the softplus is itself rounded
// by up to |x| 2^-24, which is that much of e^x, and silu(v) is off by at most v^2
// e^v 2^-24 where v is far below zero, under 2^-24 everywhere (outputs of the fp32
// convolution and norm are 6.7e-8 and 8.9e-8 from 64 bits, plain fp32 arithmetic's
// 7.4e-8 and 8.9e-8).  CUDA's expf and a division made fp32 norms and scans 20 to
// 45 % slower, the product's low part in an fma up to 28 %.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_exp(float x) { return ex2(x * 1.4426950408889634f); }
__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-x).  e^-x = inf gives 0.
__device__ __forceinline__ float sigmoid(float x) { return fast_rcp(1.f + fast_exp(-x)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d silu(v) / dv = s (1 + v (1 - s)), s = sigmoid(v)
__device__ __forceinline__ float silu_slope(float v)
{
    const float s = sigmoid(v);
    return s * fmaf(v, 1.f - s, 1.f);
}

// The sequences of a call: N sequences of T tokens each, or, packed, sequence
// n at tokens [cu[n], cu[n + 1]) of `total`.  Bounds are held to [0, total],
// so that an array that breaks the contract gives wrong values and no access
// out of range.  (Up to 2^30 tokens and sequences: a token's number, and that of
// a unit below, fits an int.)
struct Seqs {
    const int32_t* cu;
    int N;
    int T;
    int total;
    __device__ __forceinline__ int start(int n) const
    {
        if (!cu) return n * T;
        const int s = cu[n];
        return s < 0 ? 0 : (s > total ? total : s);
    }
    __device__ __forceinline__ void bounds(int n, int& a, int& b) const
    {
        a = start(n);
        b = cu ? start(n + 1) : a + T;
        if (b < a) b = a;
    }
    // the last sequence that begins at or before token t
    __device__ __forceinline__ int find(int t) const
    {
        if (!cu) return T > 0 ? (int)((unsigned)t / (unsigned)T) : 0;
        int lo = 0, len = N;
        while (len > 1) {
            const int half = len >> 1;
            if (start(lo + half) <= t) {
                lo += half;
                len -= half;
            } else {
                len = half;
            }
        }
        return lo;
    }
};

// Every sequence cut into units of `len` tokens (the last one ragged; an empty
// sequence has one empty unit).  Packed sequences: unit numbers are slots of
// which some stay empty, sequence n owning those from start(n) / len + n on,
// so that no count of earlier units is needed.
struct Units {
    Seqs s;
    int len;
    int per_seq;  // units of a sequence that is not packed
    __host__ __device__ int slots() const { return s.cu ? s.total / len + s.N : s.N * per_seq; }
    __device__ __forceinline__ int first(int n) const
    {
        return s.cu ? (int)((unsigned)s.start(n) / (unsigned)len) + n : n * per_seq;
    }
    __device__ __forceinline__ int count_of(int a, int b) const
    {
        return b > a ? (int)((unsigned)(b - a + len - 1) / (unsigned)len) : 1;
    }
    __device__ __forceinline__ int count(int n) const
    {
        if (!s.cu) return per_seq;
        int a, b;
        s.bounds(n, a, b);
        return count_of(a, b);
    }
    // Sequence, index, whether it is the sequence's last, and tokens [a, b) of
    // slot j; false: an empty slot.  Called by whole warps.
    __device__ __forceinline__ bool locate(int j, int& n, int& seg, bool& last, int& a, int& b) const
    {
        if (!s.cu) {
            n = (int)((unsigned)j / (unsigned)per_seq);
            seg = j - n * per_seq;
            last = seg + 1 == per_seq;
            const int s0 = n * s.T;
            a = s0 + seg * len;
            b = a + len < s0 + s.T ? a + len : s0 + s.T;
            return true;
        }
        // 32 probes a round: two or three rounds of loads instead of ten
        const int lane = threadIdx.x & 31;
        int lo = 0, cnt = s.N;
        while (cnt > 1) {
            const int step = (cnt + 31) >> 5;
            const bool ok = lane * step < cnt && first(lo + lane * step) <= j;
            const int hits = __popc(__ballot_sync(0xffffffffu, ok));
            const int at = (hits > 0 ? hits - 1 : 0) * step;
            lo += at;
            cnt = cnt - at < step ? cnt - at : step;
        }
        n = lo;
        int s0, s1;
        s.bounds(n, s0, s1);
        const int k = j - ((int)((unsigned)s0 / (unsigned)len) + n), all = count_of(s0, s1);
        if (k < 0 || k >= all) return false;
        seg = k;
        last = k + 1 == all;
        a = s0 + k * len;
        b = a + len < s1 ? a + len : s1;
        return true;
    }
};

// SMs of the current device.
inline int sm_count()
{
    static std::atomic<int> known[64];  // by device; a count does not change: any thread stores the same
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return sms;
    const bool slot = dev >= 0 && dev < 64;
    if (slot)
        if (const int n = known[dev].load(std::memory_order_relaxed)) return n;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
    if (slot) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

}  // namespace layer
}  // namespace kda
