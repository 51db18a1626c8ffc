// Group norm with an optional SiLU, channels last:
//
//     xhat = (x - mean) rstd,   v = xhat w + b,   y = v or silu(v)
//
// with mean and 1 / sqrt(var + eps) over a sample's tokens and the C / G
// channels of a group.  A sample is a token (the per-head norm of a mixer's
// output) or a whole sequence.
//
// Per token, a row of one group is contiguous and fits the registers of a few
// lanes, at most a block's: one read, one write (memory-bound).  16384 x 4096 in bf16, 32 groups,
// SiLU: 70 us, 3.9 TB/s (60 % of the measured copy rate); instructions (64 % of
// the slots) and the SiLU's two special functions (51 %) are as near their limits.
// Two rows at a time in 64 registers and four blocks an SM; four rows in 103
// registers and two blocks took 98 us.
//
// Over sequences, three launches: partial statistics of units of tokens, their
// combination in a fixed order, and the normalisation (x is read twice; what
// fits the 126 MB L2 comes from HBM once).  24007 x 640 in 11 sequences, forward
// and backward: 100 us in six launches, against 28 us for its bytes: each launch
// is a few microseconds of finding its unit, latency and its own ramp.
//
// Sums of squares run over deviations: within a thread from the thread's first
// value, across threads and units from the common mean,
//     q = sum_i (q_i + n_i (m_i - m)^2),
// so that a mean far from zero costs no digits.  Sums over many tokens run in
// short chains, and their parts are added up in 64 bits: fp32 results are 0.8 to
// 1.3e-7 from 64 bits, dweight and dbias of 27000 tokens too (2.1e-7 in one chain).
#include "layer.h"
#include "layer_common.cuh"

namespace kda {
namespace {

using namespace layer;

template <int LANES>
__device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over groups of `lanes` neighbouring lanes (a power of two).
__device__ __forceinline__ float part_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums over a row's LANES lanes of each of v: lanes of a warp, or all 256 threads
// of the block (red: theirs to use; every thread of the block takes part).
template <int LANES, int U>
__device__ __forceinline__ void row_sums(float (&v)[U], float (*red)[8])
{
#pragma unroll
    for (int q = 0; q < U; ++q) v[q] = lane_sum<(LANES < 32 ? LANES : 32)>(v[q]);
    if constexpr (LANES > 32) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int q = 0; q < U; ++q) red[q][threadIdx.x >> 5] = v[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < U; ++q) {
            v[q] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[q] += red[q][i];
        }
    }
}

// ---- per token --------------------------------------------------------------
// LANES lanes (up to a warp, or the block's 256 threads) hold one row of Cg = C / G values, NV vectors of V each (lane l:
// values (l + i LANES) V; kFull: they are Cg to the last one).  A lane keeps to
// one group, so that its weights stay in registers while it walks the tokens, U
// at a time: their loads are in flight and their sums are folded together.
// By the values a lane holds of a row: blocks per SM, and rows at a time.
constexpr int rows_blocks(int values, bool full, bool bwd)
{
    return bwd ? (values <= 4 ? 3 : values <= 8 ? 2 : 1) : (values <= 8 ? (full ? 4 : 3) : 2);
}
constexpr int rows_at_once(int values, bool bwd)
{
    return values <= 2 || (values <= 4 && !bwd) ? 4 : values <= 8 ? 2 : 1;
}
// fp32: rows that a lane's sums for dweight and dbias run over before they go to
// sums of those sums, in shared memory (chains of 8 and rows / 8 roundings; up to
// 2 % of the time).  Not for bf16, whose inputs carry 2^-9: there the registers of
// a lane with 32 values spill (16384 x 1024 in one group: 92 us against 68).
constexpr int kRowsASum = 8;
template <typename T>
constexpr bool kSumsOfSums = sizeof(T) == 4;
// Vectors of a row that a lane holds at most: 16 values in a warp's lane (32 in
// vectors of 8), then the row takes the block; 32 in a block's, 16 in vectors of
// one.  Forward and backward, SiLU, bf16: 3191 x 4640 in 32 groups (of 145: 5
// values a lane) 107 us in a warp, 435 in a block; 4096 x 8190 in one group 179 in
// a block, 360 reading the row again; but 8192 x 4097 923 in a block of 32 values a
// lane, 298 reading it again.
constexpr int most_vectors(int V, int lanes) { return V > 1 && (lanes > 32 || V > 4) ? 32 / V : 16 / V; }

template <typename T, int V, int LANES, int NV, bool kFull, bool kBwd>
__global__ void __launch_bounds__(256, rows_blocks(V * NV, kFull, kBwd))
kda_norm_rows_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                     T* __restrict__ out, float* __restrict__ mean, float* __restrict__ rstd,
                     const T* __restrict__ d_out, float* __restrict__ grad_x, float* __restrict__ part,
                     int rows, int G, int Cg, int walkers, float eps, int act)
{
    // walker k of group g takes rows k, k + walkers, ...
    const long long id = ((long long)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int lane = threadIdx.x & (LANES - 1);
    const int g = (int)(id % G), k = (int)(id / G);
    const bool live = k < walkers;  // a row's lanes agree; the warp stays together for the sums
    auto in = [&](int i) { return kFull || (lane + i * LANES) * V < Cg; };
    const size_t col = (size_t)g * Cg + lane * V, C = (size_t)G * Cg;
    float w[NV][V], b[NV][V];
    float dw[kBwd ? NV : 1][V], db[kBwd ? NV : 1][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = in(i) && weight ? weight[col + i * LANES * V + j] : 1.f;
            b[i][j] = in(i) && bias ? bias[col + i * LANES * V + j] : 0.f;
            if (kBwd) dw[kBwd ? i : 0][j] = db[kBwd ? i : 0][j] = 0.f;
        }
    const float inv = 1.f / (float)Cg;
    constexpr int U = rows_at_once(V * NV, kBwd);
    __shared__ float red[LANES > 32 ? U : 1][8];
    constexpr bool kSums = kBwd && kSumsOfSums<T>;
    extern __shared__ float sums[];  // kSums: this thread's, [2][NV V][256]
    float* own = sums + threadIdx.x;
    if (kSums)
#pragma unroll
        for (int i = 0; i < 2 * NV * V; ++i) own[i * 256] = 0.f;
    auto flush = [&] {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float& a = dw[kBwd ? i : 0][j];
                float& c = db[kBwd ? i : 0][j];
                own[(i * V + j) * 256] += a;
                own[((NV + i) * V + j) * 256] += c;
                a = c = 0.f;
            }
    };
    const int steps = (rows + walkers - 1) / walkers;
    for (int s = 0; s < steps; s += U) {
        size_t at[U];
        bool here[U];
        Raw<T, V> rx[U][NV], rd[kBwd ? U : 1][kBwd ? NV : 1];
        float m[U], rs[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int r = live && s + q < steps ? k + (s + q) * walkers : rows;
            here[q] = r < rows;
            at[q] = (size_t)(here[q] ? r : rows - 1) * C + col;  // a row behind the last repeats it
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in(i)) {
                    rx[q][i].load(x + at[q] + i * LANES * V);
                    if constexpr (kBwd) rd[q][i].load(d_out + at[q] + i * LANES * V);
                }
            if (kBwd) {
                m[q] = mean[(size_t)(here[q] ? r : rows - 1) * G + g];
                rs[q] = rstd[(size_t)(here[q] ? r : rows - 1) * G + g];
            }
        }
        float v[U][NV][V], s1[U], s2[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            s1[q] = s2[q] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (in(i)) rx[q][i].get(v[q][i]);
                else
#pragma unroll
                    for (int j = 0; j < V; ++j) v[q][i][j] = 0.f;
            }
        }
        if constexpr (!kBwd) {
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) s1[q] += v[q][i][j];
            }
            row_sums<LANES>(s1, red);
#pragma unroll
            for (int q = 0; q < U; ++q) m[q] = s1[q] * inv;
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (in(i))
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float d = v[q][i][j] - m[q];
                            s2[q] = fmaf(d, d, s2[q]);
                        }
            }
            row_sums<LANES>(s2, red);
#pragma unroll
            for (int q = 0; q < U; ++q) rs[q] = 1.f / sqrtf(fmaf(s2[q], inv, eps));
#pragma unroll
            for (int q = 0; q < U; ++q) {
                if (!here[q]) continue;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!in(i)) continue;
                    float y[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        y[j] = fmaf((v[q][i][j] - m[q]) * rs[q], w[i][j], b[i][j]);
                        if (act) y[j] = silu(y[j]);
                    }
                    store_vec<V>(out + at[q] + i * LANES * V, y);
                }
                if (lane == 0) {
                    const size_t r = (size_t)(k + (s + q) * walkers) * G + g;
                    mean[r] = m[q];
                    rstd[r] = rs[q];
                }
            }
        } else {
            float dy[U][NV][V];
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (in(i)) rd[q][i].get(dy[q][i]);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float& d = dy[q][i][j];
                        if (!in(i)) d = 0.f;
                        const float xh = v[q][i][j] = (v[q][i][j] - m[q]) * rs[q];
                        if (act) d *= silu_slope(fmaf(xh, w[i][j], b[i][j]));
                        if (!here[q]) d = 0.f;
                        dw[i][j] = fmaf(d, xh, dw[i][j]);
                        db[i][j] += d;
                        d *= w[i][j];
                        s1[q] += d;
                        s2[q] = fmaf(d, xh, s2[q]);
                    }
                }
            }
            row_sums<LANES>(s1, red);
            row_sums<LANES>(s2, red);
#pragma unroll
            for (int q = 0; q < U; ++q) {
                s1[q] *= inv;
                s2[q] *= inv;
                if (!here[q]) continue;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (!in(i)) continue;
                    float dx[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) dx[j] = rs[q] * (dy[q][i][j] - s1[q] - v[q][i][j] * s2[q]);
                    store_vec<V>(grad_x + at[q] + i * LANES * V, dx);
                }
            }
            if (kSums && (s + U) % kRowsASum == 0) flush();
        }
    }
    if (kBwd && live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in(i)) continue;
            float (&a)[V] = dw[kBwd ? i : 0];
            float (&c)[V] = db[kBwd ? i : 0];
            if (kSums)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    a[j] += own[(i * V + j) * 256];
                    c[j] += own[((NV + i) * V + j) * 256];
                }
            store_vec<V>(part + ((size_t)k * 2) * C + col + i * LANES * V, a);
            store_vec<V>(part + ((size_t)k * 2 + 1) * C + col + i * LANES * V, c);
        }
    }
}

__device__ __forceinline__ float block_sum(float v, float* red)
{
    v = lane_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red[i];
    return s;
}

// Rows too long for a block's registers: a block per (walker, group), the row
// read again from L1/L2 for each pass.  The parameters' sums stay in the
// block's own rows of `part`, where only this thread adds to them.
template <typename T, int V, bool kBwd>
__global__ void __launch_bounds__(256)
kda_norm_long_rows_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                          const float* __restrict__ bias, T* __restrict__ out, float* __restrict__ mean,
                          float* __restrict__ rstd, const T* __restrict__ d_out, float* __restrict__ grad_x,
                          float* __restrict__ part, long long rows, int G, int Cg, int walkers, float eps, int act)
{
    __shared__ float red[8];
    const int g = blockIdx.x % G, k = blockIdx.x / G;
    const float inv = 1.f / (float)Cg;
    const size_t C = (size_t)G * Cg;
    const float* w = weight ? weight + (size_t)g * Cg : nullptr;
    const float* b = bias ? bias + (size_t)g * Cg : nullptr;
    float* pw = part + ((size_t)k * 2) * C + (size_t)g * Cg;
    float* pb = pw + C;
    if (kBwd)
        for (int c = threadIdx.x * V; c < Cg; c += 256 * V)
#pragma unroll
            for (int j = 0; j < V; ++j) pw[c + j] = pb[c + j] = 0.f;
    for (long long r = k; r < rows; r += walkers) {
        const size_t at = ((size_t)r * G + g) * Cg;
        if constexpr (!kBwd) {
            float sum = 0.f, sq = 0.f, v[V];
            for (int c = threadIdx.x * V; c < Cg; c += 256 * V) {
                load_vec<V>(x + at + c, v);
#pragma unroll
                for (int j = 0; j < V; ++j) sum += v[j];
            }
            const float m = block_sum(sum, red) * inv;
            for (int c = threadIdx.x * V; c < Cg; c += 256 * V) {
                load_vec<V>(x + at + c, v);
#pragma unroll
                for (int j = 0; j < V; ++j) sq = fmaf(v[j] - m, v[j] - m, sq);
            }
            const float rs = 1.f / sqrtf(fmaf(block_sum(sq, red), inv, eps));
            for (int c = threadIdx.x * V; c < Cg; c += 256 * V) {
                load_vec<V>(x + at + c, v);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] = fmaf((v[j] - m) * rs, w ? w[c + j] : 1.f, b ? b[c + j] : 0.f);
                    if (act) v[j] = silu(v[j]);
                }
                store_vec<V>(out + at + c, v);
            }
            if (threadIdx.x == 0) {
                mean[(size_t)r * G + g] = m;
                rstd[(size_t)r * G + g] = rs;
            }
        } else {
            const float m = mean[(size_t)r * G + g], rs = rstd[(size_t)r * G + g];
            float s1 = 0.f, s2 = 0.f, v[V], dy[V];
            for (int c = threadIdx.x * V; c < Cg; c += 256 * V) {
                load_vec<V>(x + at + c, v);
                load_vec<V>(d_out + at + c, dy);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (v[j] - m) * rs, wj = w ? w[c + j] : 1.f;
                    if (act) dy[j] *= silu_slope(fmaf(xh, wj, b ? b[c + j] : 0.f));
                    pw[c + j] = fmaf(dy[j], xh, pw[c + j]);
                    pb[c + j] += dy[j];
                    s1 = fmaf(dy[j], wj, s1);
                    s2 = fmaf(dy[j] * wj, xh, s2);
                }
            }
            s1 = block_sum(s1, red) * inv;
            s2 = block_sum(s2, red) * inv;
            for (int c = threadIdx.x * V; c < Cg; c += 256 * V) {
                load_vec<V>(x + at + c, v);
                load_vec<V>(d_out + at + c, dy);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (v[j] - m) * rs, wj = w ? w[c + j] : 1.f;
                    if (act) dy[j] *= silu_slope(fmaf(xh, wj, b ? b[c + j] : 0.f));
                    dy[j] = rs * (dy[j] * wj - s1 - xh * s2);
                }
                store_vec<V>(grad_x + at + c, dy);
            }
        }
    }
}

// ---- over sequences ---------------------------------------------------------
// A block takes one unit of tokens and `gb` whole groups.  Where gb groups fit
// 256 threads (cols = gb Cg / V columns), a thread keeps to one column and
// strides over the tokens; a group wider than 256 columns has a block of its
// own whose threads walk the columns too.
struct Layout {
    int cols, cpg, gb, ngb, ty, threads;  // columns per block and per group, groups per block, blocks across, token lanes
    int len;                              // tokens per unit
};

// One unit's tokens of the column at p, ty apart, kBatch rows in flight.  `f` is
// told which is a batch's first, `done` follows its last: sums run over a batch
// first, so that the chains of roundings are short.  (The backward pass's sums over
// two tensors' rows run on: batches cost them 18 % and left dweight at 1.1e-7 of
// 64 bits instead of 1.3e-7.)
constexpr int kBatch = 8;
template <typename T, int V, typename F, typename E>
__device__ __forceinline__ void each_token(const T* p, int a, int b, int C, int ty, F&& f, E&& done)
{
    for (int t = a; t < b; t += kBatch * ty) {
        Raw<T, V> r[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (t + i * ty < b) r[i].load(p + (size_t)(t + i * ty) * C);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (t + i * ty < b) {
                float v[V];
                r[i].get(v);
                f(t + i * ty, i == 0, v);
            }
        done();
    }
}
// ... of the columns at p and q
template <typename T, int V, typename F>
__device__ __forceinline__ void each_token2(const T* p, const T* q, int a, int b, int C, int ty, F&& f)
{
    constexpr int U = kBatch / 2;
    for (int t = a; t < b; t += U * ty) {
        Raw<T, V> r[U], s[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (t + i * ty < b) {
                r[i].load(p + (size_t)(t + i * ty) * C);
                s[i].load(q + (size_t)(t + i * ty) * C);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (t + i * ty < b) {
                float v[V], w[V];
                r[i].get(v);
                s[i].get(w);
                f(t + i * ty, v, w);
            }
    }
}

// Partial statistics: part[(unit G + g) 2 ..] = mean and squared deviations of
// the unit's tokens of group g (its count is known from the unit).
template <typename T, int V>
__global__ void __launch_bounds__(256)
kda_norm_stats_kernel(const T* __restrict__ x, float* __restrict__ part, Units units, Layout l, int C, int G)
{
    __shared__ float sn[256], sm[256], sq[256];  // per thread: count, mean, squared deviations
    int n, seg, a, b;
    bool last;
    const int unit = blockIdx.x / l.ngb;
    if (!units.locate(unit, n, seg, last, a, b)) return;
    const int g0 = (int)(blockIdx.x % l.ngb) * l.gb;
    const int groups = G - g0 < l.gb ? G - g0 : l.gb;
    const int wide = l.cols > 256;
    const int ty = wide ? 0 : threadIdx.x / l.cols;
    const int cx = wide ? threadIdx.x : threadIdx.x % l.cols;
    float cnt = 0.f, mean = 0.f, dev = 0.f;
    if (ty < l.ty && a + ty < b) {
        const float rows = (float)((b - a - ty + l.ty - 1) / l.ty * V);
        for (int c = cx; c < groups * l.cpg; c += wide ? l.threads : l.cols) {
            const T* p = x + ((size_t)g0 * l.cpg + c) * V;
            float first[V], s1 = 0.f, s2 = 0.f, b1, b2;
            load_vec<V>(p + (size_t)(a + ty) * C, first);
            const float k = first[0];
            each_token<T, V>(p, a + ty, b, C, l.ty, [&](int, bool start, const float (&v)[V]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float d = v[j] - k;
                    b1 = start && j == 0 ? d : b1 + d;
                    b2 = start && j == 0 ? d * d : fmaf(d, d, b2);
                }
            }, [&] {
                s1 += b1;
                s2 += b2;
            });
            const float d = s1 / rows, m = k + d, q = fmaxf(s2 - s1 * d, 0.f);
            // another column of the same group (wide): shares by the counts
            const float all = cnt + rows, r = rows / all, e = m - mean;
            dev += q + e * e * cnt * r;
            mean = fmaf(e, r, mean);
            cnt = all;
        }
    }
    sn[threadIdx.x] = cnt;
    sm[threadIdx.x] = mean;
    sq[threadIdx.x] = dev;
    __syncthreads();
    // over a group's threads, `lg` lanes a group: all groups at once where they fit
    const int per = wide ? l.threads : l.cpg * l.ty;
    int lg = 32;
    while (lg > 1 && (lg / 2 >= per || lg * groups > l.threads)) lg >>= 1;
    const int sub = threadIdx.x % lg, across = l.threads / lg;
    const float inv = 1.f / ((float)(b - a) * (float)(l.cpg * V));
    for (int g1 = 0; g1 < groups; g1 += across) {
        const int g = g1 + threadIdx.x / lg;
        auto at = [&](int i) { return wide ? i : (i / l.cpg) * l.cols + g * l.cpg + i % l.cpg; };
        const float k = g < groups ? sm[at(0)] : 0.f;
        float s1 = 0.f, s2 = 0.f, rest = 0.f;
        if (g < groups)
            for (int i = sub; i < per; i += lg) s1 = fmaf(sn[at(i)], sm[at(i)] - k, s1);
        float m = fmaf(part_sum(s1, lg), inv, k);
        if (g < groups)
            for (int i = sub; i < per; i += lg) {
                const float e = sm[at(i)] - m;
                rest = fmaf(sn[at(i)], e, rest);  // what k's rounding left of the mean
                s2 += fmaf(sn[at(i)] * e, e, sq[at(i)]);
            }
        s2 = part_sum(s2, lg);
        m = fmaf(part_sum(rest, lg), inv, m);
        if (g < groups && sub == 0)
            *reinterpret_cast<float2*>(part + ((size_t)unit * G + g0 + g) * 2) = make_float2(m, s2);
    }
}

// Sum over a block's rows of 32 lanes, for every lane; red is [32][33].
__device__ __forceinline__ double rows_sum(double v, double (*red)[33])
{
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    __syncthreads();
    red[y][lane] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += red[i][lane];
    return s;
}

// mean and rstd of every (sequence, group): a block takes 32 groups of a
// sequence, its 32 warps the sequence's units in turn.  In 64 bits: one number's
// sum of 32 and more parts would lose what its threads' sums have kept.
__global__ void __launch_bounds__(1024)
kda_norm_merge_kernel(const float* __restrict__ part, float* __restrict__ mean, float* __restrict__ rstd,
                      Units units, int G, int Cg, int across, float eps)
{
    __shared__ double red[32][33];
    const int n = blockIdx.x / across, lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int g = (int)(blockIdx.x % across) * 32 + lane, gg = g < G ? g : G - 1;
    int a, b;
    units.s.bounds(n, a, b);
    const int cnt = b > a ? units.count_of(a, b) : 0;
    const float2* p = reinterpret_cast<const float2*>(part) + (size_t)units.first(n) * G + gg;
    const double inv = b > a ? 1.0 / ((double)(b - a) * Cg) : 0.0;
    auto weight = [&](int i) {  // values of unit i
        const int left = b - a - i * units.len;
        return (double)(left < units.len ? left : units.len) * Cg;
    };
    double s1 = 0.0, s2 = 0.0;
#pragma unroll 4
    for (int i = y; i < cnt; i += 32) s1 = fma(weight(i), (double)p[(size_t)i * G].x, s1);
    const double m = rows_sum(s1, red) * inv;
#pragma unroll 4
    for (int i = y; i < cnt; i += 32) {
        const float2 v = p[(size_t)i * G];
        const double e = (double)v.x - m;
        s2 += fma(weight(i) * e, e, (double)v.y);
    }
    s2 = rows_sum(s2, red);
    if (y == 0 && g < G) {
        mean[(size_t)n * G + g] = (float)m;  // 0 of an empty sequence
        rstd[(size_t)n * G + g] = (float)(1.0 / sqrt(fma(s2, inv, (double)eps)));
    }
}

// The normalisation (forward), or dx from the sums of the kernels below
// (backward; sums[(n G + g) 2 ..] = mean of k and of k xhat).
template <typename T, int V, bool kBwd>
__global__ void __launch_bounds__(256)
kda_norm_apply_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                      T* __restrict__ out, const float* __restrict__ mean, const float* __restrict__ rstd,
                      const T* __restrict__ d_out, const float* __restrict__ sums, float* __restrict__ grad_x,
                      Units units, Layout l, int C, int G, int act)
{
    int n, seg, a, b;
    bool last;
    if (!units.locate(blockIdx.x / l.ngb, n, seg, last, a, b)) return;
    const int g0 = (int)(blockIdx.x % l.ngb) * l.gb;
    const int groups = G - g0 < l.gb ? G - g0 : l.gb;
    const int wide = l.cols > 256;
    const int ty = wide ? 0 : threadIdx.x / l.cols;
    const int cx = wide ? threadIdx.x : threadIdx.x % l.cols;
    if (ty >= l.ty) return;
    for (int c = cx; c < groups * l.cpg; c += wide ? l.threads : l.cols) {
        const int ch = (g0 * l.cpg + c) * V;
        const size_t ng = (size_t)n * G + g0 + c / l.cpg;
        const float m = mean[ng], rs = rstd[ng];
        float w[V], bb[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[j] = weight ? weight[ch + j] : 1.f;
            bb[j] = bias ? bias[ch + j] : 0.f;
        }
        if constexpr (!kBwd) {
            each_token<T, V>(x + ch, a + ty, b, C, l.ty, [&](int t, bool, float (&v)[V]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] = fmaf((v[j] - m) * rs, w[j], bb[j]);
                    if (act) v[j] = silu(v[j]);
                }
                store_vec<V>(out + (size_t)t * C + ch, v);
            }, [] {});
        } else {
            const float k1 = sums[ng * 2], k2 = sums[ng * 2 + 1];
            each_token2<T, V>(x + ch, d_out + ch, a + ty, b, C, l.ty, [&](int t, float (&v)[V], float (&dy)[V]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (v[j] - m) * rs;
                    if (act) dy[j] *= silu_slope(fmaf(xh, w[j], bb[j]));
                    dy[j] = rs * (dy[j] * w[j] - k1 - xh * k2);
                }
                store_vec<V>(grad_x + (size_t)t * C + ch, dy);
            });
        }
    }
}

// Backward sums of a unit: part[unit][0][c] = sum dv xhat, part[unit][1][c] =
// sum dv, and over a group's channels gsum[(unit G + g) 2 ..] = sum k, sum k
// xhat (k = dv w).  A slot without a unit gets zeros in `part`.
template <typename T, int V>
__global__ void __launch_bounds__(256)
kda_norm_bwd_sums_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                         const float* __restrict__ mean, const float* __restrict__ rstd,
                         const T* __restrict__ d_out, float* __restrict__ part, float* __restrict__ gsum,
                         Units units, Layout l, int C, int G, int act)
{
    __shared__ float red[2 * V * 256];  // per thread, then per column of the block
    __shared__ float red_g[2][256];     // per thread: sums of k and k xhat
    int n, seg, a, b;
    bool last;
    const int unit = blockIdx.x / l.ngb;
    const int g0 = (int)(blockIdx.x % l.ngb) * l.gb;
    const int groups = G - g0 < l.gb ? G - g0 : l.gb;
    const int wide = l.cols > 256;
    const int chans = groups * l.cpg * V, ch0 = g0 * l.cpg * V;
    float* pw = part + ((size_t)unit * 2) * C + ch0;
    float* pb = pw + C;
    if (!units.locate(unit, n, seg, last, a, b)) {
        for (int c = threadIdx.x; c < chans; c += l.threads) pw[c] = pb[c] = 0.f;
        return;
    }
    const int ty = wide ? 0 : threadIdx.x / l.cols;
    const int cx = wide ? threadIdx.x : threadIdx.x % l.cols;
    float s1 = 0.f, s2 = 0.f;
    for (int c = cx; c < groups * l.cpg; c += wide ? l.threads : l.cols) {
        if (ty >= l.ty) break;
        const int ch = ch0 + c * V;
        const size_t ng = (size_t)n * G + g0 + c / l.cpg;
        const float m = mean[ng], rs = rstd[ng];
        float w[V], bb[V], dw[V], db[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[j] = weight ? weight[ch + j] : 1.f;
            bb[j] = bias ? bias[ch + j] : 0.f;
            dw[j] = db[j] = 0.f;
        }
        each_token2<T, V>(x + ch, d_out + ch, a + ty, b, C, l.ty, [&](int, float (&v)[V], float (&dy)[V]) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (v[j] - m) * rs;
                if (act) dy[j] *= silu_slope(fmaf(xh, w[j], bb[j]));
                dw[j] = fmaf(dy[j], xh, dw[j]);
                db[j] += dy[j];
            }
        });
        if (wide) {
            store_vec<V>(pw + c * V, dw);
            store_vec<V>(pb + c * V, db);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s1 = fmaf(w[j], db[j], s1);
                s2 = fmaf(w[j], dw[j], s2);
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                red[j * 256 + threadIdx.x] = dw[j];
                red[(V + j) * 256 + threadIdx.x] = db[j];
                s1 = fmaf(w[j], db[j], s1);
                s2 = fmaf(w[j], dw[j], s2);
            }
        }
    }
    if (wide) {  // the whole block agrees
        s1 = block_sum(s1, red);
        s2 = block_sum(s2, red + 8);
        if (threadIdx.x == 0) {
            gsum[((size_t)unit * G + g0) * 2] = s1;
            gsum[((size_t)unit * G + g0) * 2 + 1] = s2;
        }
        return;
    }
    red_g[0][threadIdx.x] = s1;
    red_g[1][threadIdx.x] = s2;
    __syncthreads();
    // over a column's token lanes, and over a group's threads
    for (int q = threadIdx.x; q < 2 * chans; q += l.threads) {
        const int which = q >= chans, c = q - which * chans;
        const float* r = red + (which * V + c % V) * 256 + c / V;
        float t = 0.f;
        for (int y = 0; y < l.ty; ++y) t += r[y * l.cols];
        (which ? pb : pw)[c] = t;
    }
    const int per = l.cpg * l.ty;
    int lg = 32;
    while (lg > 1 && (lg / 2 >= per || lg * groups > l.threads)) lg >>= 1;
    const int sub = threadIdx.x % lg;
    for (int g1 = 0; g1 < groups; g1 += l.threads / lg) {
        const int g = g1 + threadIdx.x / lg;
        float t1 = 0.f, t2 = 0.f;
        if (g < groups)
            for (int i = sub; i < per; i += lg) {
                const int at = (i / l.cpg) * l.cols + g * l.cpg + i % l.cpg;
                t1 += red_g[0][at];
                t2 += red_g[1][at];
            }
        t1 = part_sum(t1, lg);
        t2 = part_sum(t2, lg);
        if (g < groups && sub == 0)
            *reinterpret_cast<float2*>(gsum + ((size_t)unit * G + g0 + g) * 2) = make_float2(t1, t2);
    }
}

// From the parts: the parameters' gradients (the first blocks; 32 channels
// each, 32 warps over the parts), and of every (sequence, group) the means of
// k and k xhat (the others; 32 groups of a sequence each), in 64 bits.
__global__ void __launch_bounds__(1024)
kda_norm_bwd_merge_kernel(const float* __restrict__ part, float* __restrict__ grad_weight,
                          float* __restrict__ grad_bias, long long parts, const float* __restrict__ gsum,
                          float* __restrict__ sums, Units units, int C, int G, int param_blocks, int across)
{
    __shared__ double red[2][32][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    if ((int)blockIdx.x < param_blocks) {
        const int c = blockIdx.x * 32 + lane;
        double sw = 0.0, sb = 0.0;
        if (c < C)
#pragma unroll 4
            for (long long i = y; i < parts; i += 32) {
                sw += part[((size_t)i * 2) * C + c];
                sb += part[((size_t)i * 2 + 1) * C + c];
            }
        red[0][y][lane] = sw;
        red[1][y][lane] = sb;
        __syncthreads();
        if (y < 2 && c < C) {
            double t = 0.0;
#pragma unroll
            for (int k = 0; k < 32; ++k) t += red[y][k][lane];
            if (y == 0 && grad_weight) grad_weight[c] = (float)t;
            if (y == 1 && grad_bias) grad_bias[c] = (float)t;
        }
        return;
    }
    const int at = blockIdx.x - param_blocks, n = at / across;
    const int g = at % across * 32 + lane, gg = g < G ? g : G - 1;
    int a, b;
    units.s.bounds(n, a, b);
    const int cnt = b > a ? units.count_of(a, b) : 0;
    const float2* p = reinterpret_cast<const float2*>(gsum) + (size_t)units.first(n) * G + gg;
    double s1 = 0.0, s2 = 0.0;
#pragma unroll 4
    for (int i = y; i < cnt; i += 32) {
        const float2 v = p[(size_t)i * G];
        s1 += v.x;
        s2 += v.y;
    }
    s1 = rows_sum(s1, red[0]);
    s2 = rows_sum(s2, red[0]);
    if (y == 0 && g < G) {
        const double inv = cnt ? 1.0 / ((double)(b - a) * (C / G)) : 0.0;
        sums[((size_t)n * G + g) * 2] = (float)(s1 * inv);
        sums[((size_t)n * G + g) * 2 + 1] = (float)(s2 * inv);
    }
}

// ---- host -------------------------------------------------------------------

// vector width: the widest of 8 (bf16 only), 4, 2 and 1 that divides a group
int width_of(int Cg, kda_dtype dtype)
{
    if (dtype == KDA_DTYPE_BF16 && Cg % 8 == 0) return 8;
    return Cg % 4 == 0 ? 4 : (Cg % 2 == 0 ? 2 : 1);
}

// Blocks of up to 256 threads; units of 8 to 64 tokens per thread, the longest
// that still give every SM four blocks.
Layout layout_of(int C, int G, int V, long long tokens)
{
    Layout l;
    l.cpg = C / G / V;
    if (l.cpg > 256) {
        l.gb = 1;
        l.cols = l.cpg;
        l.ty = 1;
        const int rounds = (l.cpg + 255) / 256;  // columns of a thread
        l.threads = ((l.cpg + rounds - 1) / rounds + 31) / 32 * 32;
    } else {
        l.gb = 256 / l.cpg < G ? 256 / l.cpg : G;
        l.cols = l.gb * l.cpg;
        l.ty = 256 / l.cols;
        l.threads = (l.cols * l.ty + 31) / 32 * 32;
    }
    l.ngb = (G + l.gb - 1) / l.gb;
    l.len = 64 * l.ty;
    while (l.len > 8 * l.ty && tokens / l.len * l.ngb < 4LL * sm_count()) l.len >>= 1;
    return l;
}

Units units_of(const int32_t* cu, int B, int T, int N, int len)
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
long long slots_of(int B, int T, int N, int packed, int len)
{
    return packed ? ((long long)B * T) / len + N : (long long)N * (T > 0 ? (T + len - 1) / len : 1);
}

// Lanes per row and vectors per lane of the per-token kernel; lanes = 0: rows
// too long for it.
struct RowShape {
    int V, lanes, nv, walkers;
    long long blocks;
};
RowShape row_shape(long long rows, int C, int G, kda_dtype dtype, bool bwd)
{
    RowShape r = {};
    const int Cg = C / G;
    r.V = width_of(Cg, dtype);
    const int vecs = Cg / r.V;
    r.lanes = 1;
    while (r.lanes < 32 && r.lanes < vecs) r.lanes <<= 1;
    if (vecs > 32 * most_vectors(r.V, 32)) r.lanes = 256;
    r.nv = 1;
    while (r.nv * r.lanes < vecs) r.nv <<= 1;
    const bool fits = r.nv <= most_vectors(r.V, r.lanes);
    const int per_block = fits ? 256 / r.lanes : 1;  // rows in flight
    if (!fits) r.lanes = r.nv = 0;
    // as many walkers as the SMs hold at a time, none without a row
    const long long want = (long long)sm_count() * (r.nv ? rows_blocks(r.V * r.nv, r.lanes * r.nv * r.V == Cg, bwd) : 4) * per_block;
    long long w = (want + G - 1) / G;
    if (w > rows) w = rows;
    if (w < 1) w = 1;
    r.walkers = (int)w;
    r.blocks = (w * G + per_block - 1) / per_block;
    return r;
}

template <typename T, int V, int LANES, bool kBwd>
cudaError_t rows_nv(const NormArgs& a, const RowShape& r, cudaStream_t st)
{
    const int rows = a.B * a.T;
    // a power of two of lanes and vectors fills a row with the widest vectors only
    constexpr bool kWhole = LANES == 1 || V == 16 / (int)sizeof(T);
    const bool full = r.lanes * r.nv * V == a.C / a.G;
#define KDA_NORM_ROWS_OF(NV, FULL)                                                                             \
    do {                                                                                                       \
        auto* kernel = &kda_norm_rows_kernel<T, V, LANES, NV, FULL, kBwd>;                                     \
        constexpr int smem = kBwd && kSumsOfSums<T> ? 2 * NV * V * 256 * (int)sizeof(float) : 0;               \
        if constexpr (smem > 32 * 1024)                                                                        \
            if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) \
                return e;                                                                                      \
        kernel<<<(unsigned)r.blocks, 256, smem, st>>>((const T*)a.x, a.weight, a.bias, (T*)a.out, a.mean,      \
            a.rstd, (const T*)a.d_out, a.grad_x, (float*)a.workspace, rows, a.G, a.C / a.G, r.walkers, a.eps,  \
            a.silu);                                                                                           \
    } while (0)
#define KDA_NORM_ROWS(NV)                                                                                      \
    do {                                                                                                       \
        if constexpr (kWhole) {                                                                                \
            if (full) KDA_NORM_ROWS_OF(NV, true);                                                              \
            else KDA_NORM_ROWS_OF(NV, false);                                                                  \
        } else {                                                                                               \
            KDA_NORM_ROWS_OF(NV, false);                                                                       \
        }                                                                                                      \
        return cudaGetLastError();                                                                             \
    } while (0)
    constexpr int kMost = LANES < 32 ? 1 : most_vectors(V, LANES);
    if (r.nv == 1) KDA_NORM_ROWS(1);
    if constexpr (kMost >= 2)
        if (r.nv == 2) KDA_NORM_ROWS(2);
    if constexpr (kMost >= 4)
        if (r.nv == 4) KDA_NORM_ROWS(4);
    if constexpr (kMost >= 8)
        if (r.nv == 8) KDA_NORM_ROWS(8);
    if constexpr (kMost >= 16)
        if (r.nv == 16) KDA_NORM_ROWS(16);
#undef KDA_NORM_ROWS
#undef KDA_NORM_ROWS_OF
    return cudaErrorInvalidConfiguration;
}

template <typename T, int V, bool kBwd>
cudaError_t rows(const NormArgs& a, const RowShape& r, cudaStream_t st)
{
    switch (r.lanes) {
        case 1: return rows_nv<T, V, 1, kBwd>(a, r, st);
        case 2: return rows_nv<T, V, 2, kBwd>(a, r, st);
        case 4: return rows_nv<T, V, 4, kBwd>(a, r, st);
        case 8: return rows_nv<T, V, 8, kBwd>(a, r, st);
        case 16: return rows_nv<T, V, 16, kBwd>(a, r, st);
        case 32: return rows_nv<T, V, 32, kBwd>(a, r, st);
        case 256: return rows_nv<T, V, 256, kBwd>(a, r, st);
    }
    kda_norm_long_rows_kernel<T, V, kBwd><<<(unsigned)r.blocks, 256, 0, st>>>(
        (const T*)a.x, a.weight, a.bias, (T*)a.out, a.mean, a.rstd, (const T*)a.d_out, a.grad_x,
        (float*)a.workspace, (long long)a.B * a.T, a.G, a.C / a.G, r.walkers, a.eps, a.silu);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t forward(const NormArgs& a, kda_dtype dtype, cudaStream_t st)
{
    if (a.per_token) {
        if ((long long)a.B * a.T == 0) return cudaSuccess;
        return rows<T, V, false>(a, row_shape((long long)a.B * a.T, a.C, a.G, dtype, false), st);
    }
    const Layout l = layout_of(a.C, a.G, V, (long long)a.B * a.T);
    const Units u = units_of(a.cu_seqlens, a.B, a.T, a.N, l.len);
    const int across = (a.G + 31) / 32;
    const long long blocks = (long long)u.slots() * l.ngb, merge = (long long)a.N * across;
    if (blocks > INT32_MAX || merge > INT32_MAX) return cudaErrorInvalidConfiguration;
    float* part = (float*)a.workspace;
    if (blocks > 0) {
        kda_norm_stats_kernel<T, V><<<(unsigned)blocks, l.threads, 0, st>>>((const T*)a.x, part, u, l, a.C, a.G);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_norm_merge_kernel<<<(unsigned)merge, 1024, 0, st>>>(part, a.mean, a.rstd, u, a.G, a.C / a.G, across, a.eps);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (blocks > 0)
        kda_norm_apply_kernel<T, V, false><<<(unsigned)blocks, l.threads, 0, st>>>(
            (const T*)a.x, a.weight, a.bias, (T*)a.out, a.mean, a.rstd, nullptr, nullptr, nullptr, u, l, a.C, a.G,
            a.silu);
    return cudaGetLastError();
}

// The backward pass's workspace over sequences: the units' sums per channel
// and per group, and the sequences'.
struct SumSpace {
    size_t part, gsum, sums, total;  // in floats
};
SumSpace sum_space(size_t slots, int C, int G, int N)
{
    SumSpace s;
    s.part = 0;
    s.gsum = slots * 2 * C;
    s.sums = s.gsum + slots * 2 * G;
    s.total = s.sums + (size_t)N * G * 2;
    return s;
}

template <typename T, int V>
cudaError_t backward(const NormArgs& a, kda_dtype dtype, cudaStream_t st)
{
    const long long tokens = (long long)a.B * a.T;
    const int pblocks = (a.C + 31) / 32, across = (a.G + 31) / 32;
    float* part = (float*)a.workspace;
    if (a.per_token) {
        const RowShape r = row_shape(tokens, a.C, a.G, dtype, true);
        if (tokens > 0)
            if (cudaError_t e = rows<T, V, true>(a, r, st)) return e;
        kda_norm_bwd_merge_kernel<<<(unsigned)pblocks, 1024, 0, st>>>(part, a.grad_weight, a.grad_bias,
                                                                      tokens > 0 ? r.walkers : 0, nullptr, nullptr,
                                                                      Units{}, a.C, a.G, pblocks, across);
        return cudaGetLastError();
    }
    const Layout l = layout_of(a.C, a.G, V, tokens);
    const Units u = units_of(a.cu_seqlens, a.B, a.T, a.N, l.len);
    const long long slots = u.slots(), blocks = slots * l.ngb, mblocks = pblocks + (long long)a.N * across;
    if (blocks > INT32_MAX || mblocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const SumSpace s = sum_space((size_t)slots, a.C, a.G, a.N);
    if (blocks > 0) {
        kda_norm_bwd_sums_kernel<T, V><<<(unsigned)blocks, l.threads, 0, st>>>(
            (const T*)a.x, a.weight, a.bias, a.mean, a.rstd, (const T*)a.d_out, part, part + s.gsum, u, l, a.C, a.G,
            a.silu);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_norm_bwd_merge_kernel<<<(unsigned)mblocks, 1024, 0, st>>>(part, a.grad_weight, a.grad_bias, slots,
                                                                  part + s.gsum, part + s.sums, u, a.C, a.G, pblocks,
                                                                  across);
    if (cudaError_t e = cudaGetLastError()) return e;
    if (blocks > 0)
        kda_norm_apply_kernel<T, V, true><<<(unsigned)blocks, l.threads, 0, st>>>(
            (const T*)a.x, a.weight, a.bias, nullptr, a.mean, a.rstd, (const T*)a.d_out, part + s.sums, a.grad_x, u,
            l, a.C, a.G, a.silu);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run(const NormArgs& a, kda_dtype dtype, bool bwd, cudaStream_t st)
{
    return bwd ? backward<T, V>(a, dtype, st) : forward<T, V>(a, dtype, st);
}

cudaError_t dispatch(const NormArgs& a, kda_dtype dtype, bool bwd, cudaStream_t st)
{
    const int V = width_of(a.C / a.G, dtype);
    if (dtype == KDA_DTYPE_F32) {
        if (V == 4) return run<float, 4>(a, dtype, bwd, st);
        if (V == 2) return run<float, 2>(a, dtype, bwd, st);
        return run<float, 1>(a, dtype, bwd, st);
    }
    if (V == 8) return run<__nv_bfloat16, 8>(a, dtype, bwd, st);
    if (V == 4) return run<__nv_bfloat16, 4>(a, dtype, bwd, st);
    if (V == 2) return run<__nv_bfloat16, 2>(a, dtype, bwd, st);
    return run<__nv_bfloat16, 1>(a, dtype, bwd, st);
}

}  // namespace

size_t norm_fwd_workspace(int B, int T, int C, int G, int N, int per_token, int packed, kda_dtype dtype)
{
    if (per_token) return 0;
    const Layout l = layout_of(C, G, width_of(C / G, dtype), (long long)B * T);
    return (size_t)slots_of(B, T, N, packed, l.len) * G * 2 * sizeof(float);
}

size_t norm_bwd_workspace(int B, int T, int C, int G, int N, int per_token, int packed, kda_dtype dtype)
{
    if (per_token) {
        if ((long long)B * T == 0) return 0;
        return (size_t)row_shape((long long)B * T, C, G, dtype, true).walkers * 2 * C * sizeof(float);
    }
    const Layout l = layout_of(C, G, width_of(C / G, dtype), (long long)B * T);
    return sum_space((size_t)slots_of(B, T, N, packed, l.len), C, G, N).total * sizeof(float);
}

cudaError_t launch_norm_fwd(const NormArgs& a, kda_dtype dtype, cudaStream_t st) { return dispatch(a, dtype, false, st); }
cudaError_t launch_norm_bwd(const NormArgs& a, kda_dtype dtype, cudaStream_t st) { return dispatch(a, dtype, true, st); }

}  // namespace kda
