// Short causal depthwise convolution along the tokens, with an optional SiLU:
//
//     v[t, c] = bias[c] + sum_{j < W} w[c, j] x[t - W + 1 + j, c],   y = v or silu(v)
//
// where the W - 1 rows before a sequence come from its window state (or are
// zero).  The new state is the last W - 1 rows of (state ++ x).
//
// Memory-bound: x is read and y written once.  A thread owns V neighbouring
// channels (16 bytes where C allows) and walks a run of tokens with the last
// W - 1 rows in registers, so each row is loaded once but for the W - 1 rows
// in front of a run; four rows are in flight while the four before them are
// worked on.  131072 x 4096 in bf16 with W = 4 and SiLU: 396 us, 5.4 TB/s (84 %
// of the measured copy rate; 5.8 TB/s without the SiLU, whose exponential and
// reciprocal take 55 % of the special function unit).  Tighter register bounds
// for more warps an SM (5 and 6 blocks) cost 8 to 45 %, longer runs nothing
// either way.  Rows whose window reaches before its sequence are left
// to blocks of their own, one sequence per thread row: only those read the
// initial state and write the final one, so the two may be the same memory.
#include "layer.h"
#include "layer_common.cuh"

namespace kda {
namespace {

using namespace layer;

template <int W, int V>
struct Taps {
    float w[W][V];
    float b[V];
    __device__ __forceinline__ void load(const float* weight, const float* bias, int c0)
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float r[W];
            load_vec<W>(weight + (size_t)(c0 + i) * W, r);
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = r[j];
            b[i] = bias ? bias[c0 + i] : 0.f;
        }
    }
    // v of the row `cur` behind the rows h (oldest first)
    __device__ __forceinline__ void dot(const float (&h)[W - 1][V], const float (&cur)[V], float (&v)[V]) const
    {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float s = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][i], h[j][i], s);
            v[i] = fmaf(w[W - 1][i], cur[i], s);
        }
    }
};

template <int W, int V>
__device__ __forceinline__ void push(float (&h)[W - 1][V], const float (&cur)[V])
{
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) h[j][i] = h[j + 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) h[W - 2][i] = cur[i];
}

// Rows of (state ++ x) of sequence n: row r < W - 1 is the state's, row
// W - 1 + p is token p.
template <typename T, int W, int V>
__device__ __forceinline__ void ext_row(const T* x, const T* state, int n, int a, int r, int C,
                                        int c0, float (&v)[V])
{
    if (r >= W - 1) {
        load_vec<V>(x + (size_t)(a + r - (W - 1)) * C + c0, v);
    } else if (state) {
        load_vec<V>(state + ((size_t)n * (W - 1) + r) * C + c0, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <typename T, int W, int V>
__global__ void __launch_bounds__(128)
kda_short_conv_kernel(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                      const T* state, T* __restrict__ out, T* fin, Seqs seqs, int C, int ncb,
                      int tiles, int run, int act)
{
    const int c0 = ((int)(blockIdx.x % ncb) * blockDim.x + threadIdx.x) * V;
    const int item = blockIdx.x / ncb;
    if (c0 >= C) return;
    Taps<W, V> taps;
    taps.load(weight, bias, c0);

    if (item >= tiles) {
        // the first rows of a sequence, and its final state
        const int n = (item - tiles) * blockDim.y + threadIdx.y;
        if (n >= seqs.N) return;
        int a, b;
        seqs.bounds(n, a, b);
        const int L = b - a;
        float h[W - 1][V], last[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            ext_row<T, W, V>(x, state, n, a, j, C, c0, h[j]);
            if (fin) ext_row<T, W, V>(x, state, n, a, L + j, C, c0, last[j]);
        }
#pragma unroll
        for (int p = 0; p < W - 1; ++p) {
            if (p >= L) break;
            float cur[V], v[V];
            load_vec<V>(x + (size_t)(a + p) * C + c0, cur);
            taps.dot(h, cur, v);
            push<W, V>(h, cur);
            if (act) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
            }
            store_vec<V>(out + (size_t)(a + p) * C + c0, v);
        }
        if (fin) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_vec<V>(fin + ((size_t)n * (W - 1) + j) * C + c0, last[j]);
        }
        return;
    }

    int t = (item * blockDim.y + threadIdx.y) * run;
    const int end = t + run < seqs.total ? t + run : seqs.total;
    if (t >= end) return;
    for (int n = seqs.find(t); t < end && n < seqs.N; ++n) {
        int a, b;
        seqs.bounds(n, a, b);
        const int stop = b < end ? b : end;
        if (t < a + W - 1) t = a + W - 1;
        if (t >= stop) {
            t = stop;
            continue;
        }
        float h[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_vec<V>(x + (size_t)(t - (W - 1) + j) * C + c0, h[j]);
        constexpr int U = 4;  // rows per batch; the next batch is in flight meanwhile
        Raw<T, V> next[U];
        if (t + U <= stop)
#pragma unroll
            for (int k = 0; k < U; ++k) next[k].load(x + (size_t)(t + k) * C + c0);
        for (; t + U <= stop; t += U) {
            Raw<T, V> now[U];
#pragma unroll
            for (int k = 0; k < U; ++k) now[k] = next[k];
            if (t + 2 * U <= stop)
#pragma unroll
                for (int k = 0; k < U; ++k) next[k].load(x + (size_t)(t + U + k) * C + c0);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                float cur[V], v[V];
                now[k].get(cur);
                taps.dot(h, cur, v);
                push<W, V>(h, cur);
                if (act) {
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
                }
                store_vec<V>(out + (size_t)(t + k) * C + c0, v);
            }
        }
        for (; t < stop; ++t) {
            float cur[V], v[V];
            load_vec<V>(x + (size_t)t * C + c0, cur);
            taps.dot(h, cur, v);
            push<W, V>(h, cur);
            if (act) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
            }
            store_vec<V>(out + (size_t)t * C + c0, v);
        }
    }
}

// One token for each of N sequences: the window state is read, used and
// shifted by one row in place.  A thread takes its channels of R sequences,
// which share the taps (256 sequences of 4096 channels in bf16: 5.7 us with two
// a thread, 7.8 us with one; 17 MB).
template <typename T, int W, int V, int R>
__global__ void __launch_bounds__(128)
kda_short_conv_step_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                           const float* __restrict__ bias, T* state, T* __restrict__ out, int N, int C, int ncb,
                           int act)
{
    const int c0 = ((int)(blockIdx.x % ncb) * blockDim.x + threadIdx.x) * V;
    const int n0 = ((int)(blockIdx.x / ncb) * blockDim.y + threadIdx.y) * R;
    if (c0 >= C || n0 >= N) return;
    Raw<T, V> rows[R][W];  // the window, then the token
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r < N ? n0 + r : N - 1;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) rows[r][j].load(state + ((size_t)n * (W - 1) + j) * C + c0);
        rows[r][W - 1].load(x + (size_t)n * C + c0);
    }
    Taps<W, V> taps;
    taps.load(weight, bias, c0);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = n0 + r;
        if (n >= N) break;
        float h[W - 1][V], cur[V], v[V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) rows[r][j].get(h[j]);
        rows[r][W - 1].get(cur);
        taps.dot(h, cur, v);
        if (act) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = silu(v[i]);
        }
        store_vec<V>(out + (size_t)n * C + c0, v);
        push<W, V>(h, cur);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_vec<V>(state + ((size_t)n * (W - 1) + j) * C + c0, h[j]);
    }
}

// Backward.  With dv = dy act'(v):
//     dx[p]   = sum_j w[j] dv[p + W - 1 - j]  (+ the final state's adjoint on the last W - 1 rows)
//     dw[j]   = sum_t dv[t] x[t - W + 1 + j],   dbias = sum_t dv[t]
// A thread walks its run of tokens and the W - 1 behind it, with the
// last W - 1 rows of x and the unfinished rows of dx in registers; v is
// computed again from x.  The parameters'
// sums over a block's tokens go to `part` [tile][W + 1][C] and are added up by
// the kernel below in a fixed order.  16384 x 4096 in bf16 with SiLU: 153 us,
// 3.5 TB/s of its 540 MB; bound by issue (68 % of the slots) and the registers
// that W = 4 taps, their sums and rows take (two blocks an SM).
template <typename T, int W, int V>
__global__ void __launch_bounds__(256, 2)
kda_short_conv_bwd_kernel(const T* __restrict__ x, const float* __restrict__ weight,
                          const float* __restrict__ bias, const T* __restrict__ state,
                          const T* __restrict__ d_out, const float* __restrict__ d_fin,
                          float* __restrict__ grad_x, float* __restrict__ grad_state, float* __restrict__ part,
                          Seqs seqs, int C, int ncb, int tiles, int run, int act)
{
    extern __shared__ float red[];  // [blockDim.y][(W + 1) * V][blockDim.x]
    const int c0 = ((int)(blockIdx.x % ncb) * blockDim.x + threadIdx.x) * V;
    const int item = blockIdx.x / ncb;
    const bool mine = c0 < C;
    Taps<W, V> taps;
    if (mine) taps.load(weight, bias, c0);

    if (item >= tiles) {
        // the initial state's gradient
        const int n = (item - tiles) * blockDim.y + threadIdx.y;
        if (!mine || n >= seqs.N) return;
        int a, b;
        seqs.bounds(n, a, b);
        const int L = b - a;
        float h[W - 1][V], dst[W - 1][V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            ext_row<T, W, V>(x, state, n, a, j, C, c0, h[j]);
#pragma unroll
            for (int i = 0; i < V; ++i) dst[j][i] = 0.f;
            if (j >= L && d_fin) load_vec<V>(d_fin + ((size_t)n * (W - 1) + (j - L)) * C + c0, dst[j]);
        }
#pragma unroll
        for (int p = 0; p < W - 1; ++p) {
            if (p >= L) break;
            float cur[V], v[V], dv[V];
            load_vec<V>(x + (size_t)(a + p) * C + c0, cur);
            load_vec<V>(d_out + (size_t)(a + p) * C + c0, dv);
            taps.dot(h, cur, v);
            push<W, V>(h, cur);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (act) dv[i] *= silu_slope(v[i]);
#pragma unroll
                for (int r = p; r < W - 1; ++r) dst[r][i] = fmaf(taps.w[r - p][i], dv[i], dst[r][i]);
            }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_vec<V>(grad_state + ((size_t)n * (W - 1) + j) * C + c0, dst[j]);
        return;
    }

    float dw[W][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][i] = 0.f;
    }
    int t0 = (item * blockDim.y + threadIdx.y) * run;
    const int end = t0 + run < seqs.total ? t0 + run : seqs.total;
    if (mine && t0 < end) {
        for (int n = seqs.find(t0); t0 < end && n < seqs.N; ++n) {
            int a, b;
            seqs.bounds(n, a, b);
            const int stop = b < end ? b : end;
            if (t0 < a) t0 = a;
            if (t0 >= stop) continue;
            float h[W - 1][V], part_dx[W - 1][V];  // part_dx[i]: what row t - (W - 1) + i has so far
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                ext_row<T, W, V>(x, state, n, a, t0 - a + j, C, c0, h[j]);
#pragma unroll
                for (int i = 0; i < V; ++i) part_dx[j][i] = 0.f;
            }
            constexpr int U = 2;  // rows of x and of dy per batch; the next batch is in flight meanwhile
            const int last = stop + W - 1 < b ? stop + W - 1 : b;
            Raw<T, V> nx[U], nd[U];
            auto fetch = [&](int t) {
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    const size_t at = (size_t)(t + k < last ? t + k : last - 1) * C + c0;
                    nx[k].load(x + at);
                    nd[k].load(d_out + at);
                }
            };
            fetch(t0);
            for (int t = t0; t < stop + W - 1; t += U) {
                Raw<T, V> rx[U], rd[U];
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    rx[k] = nx[k];
                    rd[k] = nd[k];
                }
                if (t + U < last) fetch(t + U);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    if (t + k >= stop + W - 1) break;
                    float cur[V], v[V], dv[V];
                    if (t + k < b) {
                        rx[k].get(cur);
                        rd[k].get(dv);
                        taps.dot(h, cur, v);
                        if (act) {
#pragma unroll
                            for (int i = 0; i < V; ++i) dv[i] *= silu_slope(v[i]);
                        }
                    } else {
                        // rows behind the sequence have no adjoint
#pragma unroll
                        for (int i = 0; i < V; ++i) cur[i] = dv[i] = 0.f;
                    }
                    if (t + k < stop) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            db[i] += dv[i];
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) dw[j][i] = fmaf(dv[i], h[j][i], dw[j][i]);
                            dw[W - 1][i] = fmaf(dv[i], cur[i], dw[W - 1][i]);
                        }
                    }
                    push<W, V>(h, cur);
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dx[i] = fmaf(taps.w[0][i], dv[i], part_dx[0][i]);
#pragma unroll
                        for (int j = 0; j + 1 < W - 1; ++j) part_dx[j][i] = fmaf(taps.w[j + 1][i], dv[i], part_dx[j + 1][i]);
                        part_dx[W - 2][i] = taps.w[W - 1][i] * dv[i];
                    }
                    const int p = t + k - (W - 1);
                    if (p >= t0) {
                        const int r = p - b + (W - 1);  // row of the final state
                        if (r >= 0 && d_fin) {
                            float f[V];
                            load_vec<V>(d_fin + ((size_t)n * (W - 1) + r) * C + c0, f);
#pragma unroll
                            for (int i = 0; i < V; ++i) dx[i] += f[i];
                        }
                        store_vec<V>(grad_x + (size_t)p * C + c0, dx);
                    }
                }
            }
            t0 = stop;
        }
    }
    // sum over the block's runs
    const int tx = blockDim.x;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) red[((size_t)threadIdx.y * (W + 1) * V + j * V + i) * tx + threadIdx.x] = dw[j][i];
        red[((size_t)threadIdx.y * (W + 1) * V + W * V + i) * tx + threadIdx.x] = db[i];
    }
    __syncthreads();
    const int per = (W + 1) * V * tx, tid = threadIdx.y * tx + threadIdx.x;
    for (int q = tid; q < per; q += tx * blockDim.y) {
        const int col = q / V, i = q - col * V;  // neighbours write neighbouring channels
        const int j = col / tx, cx = col - j * tx;
        float s = 0.f;
        for (int y = 0; y < (int)blockDim.y; ++y) s += red[((size_t)y * (W + 1) * V + j * V + i) * tx + cx];
        const int c = ((int)(blockIdx.x % ncb) * tx + cx) * V + i;
        if (c < C) part[((size_t)item * (W + 1) + j) * C + c] = s;
    }
}

// grad_weight[c, j] and grad_bias[c] from the tiles' parts: 32 channels of one
// tap per block, eight tile lanes.  In 64 bits: of 131072 tokens, 256 parts in
// fp32 left dweight 2.5e-7 from 64 bits.
__global__ void __launch_bounds__(256)
kda_short_conv_params_kernel(const float* __restrict__ part, float* __restrict__ grad_weight,
                             float* __restrict__ grad_bias, int C, int W, int tiles)
{
    __shared__ double red[8][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, j = blockIdx.y;
    double s = 0.0;
    if (c < C)
        for (int i = y; i < tiles; i += 8) s += part[((size_t)i * (W + 1) + j) * C + c];
    red[y][lane] = s;
    __syncthreads();
    if (y == 0 && c < C) {
        double t = 0.0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += red[k][lane];
        if (j < W) grad_weight[(size_t)c * W + j] = (float)t;
        else if (grad_bias) grad_bias[c] = (float)t;
    }
}

struct Shape {
    int tx, ty, ncb, run;
    long long tiles, edges;
};

// Threads along the channels (a power of two that covers them, at most
// `width`), the rest of the block along the tokens.
Shape shape_of(int C, int V, int threads, int width)
{
    Shape s = {};
    const int cols = (C + V - 1) / V;
    s.tx = 1;
    while (s.tx < cols && s.tx < width) s.tx <<= 1;
    s.ty = threads / s.tx;
    s.ncb = (cols + s.tx - 1) / s.tx;
    return s;
}

void cut_tokens(Shape& s, long long total, int N, int longest)
{
    // the longest run that still gives every SM four blocks: the rows in front
    // of a run and its weights are loaded once per run
    const long long want = 4LL * sm_count();
    s.run = longest;
    while (s.run > 8 && ((total + (long long)s.run * s.ty - 1) / ((long long)s.run * s.ty)) * s.ncb < want) s.run >>= 1;
    s.tiles = (total + (long long)s.run * s.ty - 1) / ((long long)s.run * s.ty);
    s.edges = ((long long)N + s.ty - 1) / s.ty;
}

int fwd_width(int C, kda_dtype dtype)
{
    if (dtype == KDA_DTYPE_F32) return C % 4 == 0 ? 4 : 1;
    return C % 8 == 0 ? 8 : (C % 2 == 0 ? 2 : 1);
}
int bwd_width(int C) { return C % 4 == 0 ? 4 : 1; }

Shape bwd_shape(long long total, int C, int N)
{
    Shape s = shape_of(C, bwd_width(C), 256, 32);
    cut_tokens(s, total, N, 32);
    return s;
}

Seqs seqs_of(const int32_t* cu, int B, int T, int N)
{
    Seqs s;
    s.cu = cu;
    s.N = N;
    s.T = T;
    s.total = B * T;
    return s;
}

template <typename T, int W, int V>
cudaError_t fwd(const ConvArgs& a, cudaStream_t stream)
{
    Shape s = shape_of(a.C, V, 128, 128);
    cut_tokens(s, (long long)a.B * a.T, a.N, 64);
    const long long blocks = (s.tiles + s.edges) * s.ncb;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    kda_short_conv_kernel<T, W, V><<<(unsigned)blocks, dim3(s.tx, s.ty), 0, stream>>>(
        (const T*)a.x, a.weight, a.bias, (const T*)a.initial_state, (T*)a.out, (T*)a.final_state,
        seqs_of(a.cu_seqlens, a.B, a.T, a.N), a.C, s.ncb, (int)s.tiles, s.run, a.silu);
    return cudaGetLastError();
}

template <typename T, int W, int V>
cudaError_t step(const ConvArgs& a, cudaStream_t stream)
{
    const Shape s = shape_of(a.C, V, 128, 128);
    // two sequences a thread once that still gives every SM two blocks
    const int R = (long long)a.N * s.ncb >= 4LL * s.ty * sm_count() ? 2 : 1;
    const long long blocks = ((long long)a.N + s.ty * R - 1) / (s.ty * R) * s.ncb;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto* k = R == 2 ? &kda_short_conv_step_kernel<T, W, V, 2> : &kda_short_conv_step_kernel<T, W, V, 1>;
    k<<<(unsigned)blocks, dim3(s.tx, s.ty), 0, stream>>>((const T*)a.x, a.weight, a.bias, (T*)a.final_state,
                                                         (T*)a.out, a.N, a.C, s.ncb, a.silu);
    return cudaGetLastError();
}

template <typename T, int W, int V>
cudaError_t bwd(const ConvArgs& a, cudaStream_t stream)
{
    Shape s = bwd_shape((long long)a.B * a.T, a.C, a.N);
    const long long edges = a.grad_initial_state ? s.edges : 0;
    const long long blocks = (s.tiles + edges) * s.ncb;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (blocks > 0) {
        const size_t smem = sizeof(float) * (W + 1) * V * s.tx * s.ty;
        kda_short_conv_bwd_kernel<T, W, V><<<(unsigned)blocks, dim3(s.tx, s.ty), smem, stream>>>(
            (const T*)a.x, a.weight, a.bias, (const T*)a.initial_state, (const T*)a.d_out, a.d_final_state,
            a.grad_x, a.grad_initial_state, (float*)a.workspace, seqs_of(a.cu_seqlens, a.B, a.T, a.N), a.C, s.ncb,
            (int)s.tiles, s.run, a.silu);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_short_conv_params_kernel<<<dim3((a.C + 31) / 32, W + (a.grad_bias ? 1 : 0)), 256, 0, stream>>>(
        (const float*)a.workspace, a.grad_weight, a.grad_bias, a.C, W, (int)s.tiles);
    return cudaGetLastError();
}

enum Op { kFwd, kStep, kBwd };

template <Op op, typename T, int V>
cudaError_t by_taps(const ConvArgs& a, cudaStream_t stream)
{
    switch (a.W) {
#define KDA_CONV_W(W)                                                                  \
    case W:                                                                            \
        if constexpr (op == kFwd) return fwd<T, W, V>(a, stream);                      \
        else if constexpr (op == kStep) return step<T, W, V>(a, stream);               \
        else return bwd<T, W, V>(a, stream);
        KDA_CONV_W(2)
        KDA_CONV_W(3)
        KDA_CONV_W(4)
#undef KDA_CONV_W
    }
    return cudaErrorInvalidValue;
}

template <Op op>
cudaError_t by_type(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream)
{
    const int V = op == kBwd ? bwd_width(a.C) : fwd_width(a.C, dtype);
    if (dtype == KDA_DTYPE_F32)
        return V == 4 ? by_taps<op, float, 4>(a, stream) : by_taps<op, float, 1>(a, stream);
    if constexpr (op == kBwd) {
        return V == 4 ? by_taps<op, __nv_bfloat16, 4>(a, stream) : by_taps<op, __nv_bfloat16, 1>(a, stream);
    } else {
        return V == 8 ? by_taps<op, __nv_bfloat16, 8>(a, stream)
                      : V == 2 ? by_taps<op, __nv_bfloat16, 2>(a, stream) : by_taps<op, __nv_bfloat16, 1>(a, stream);
    }
}

}  // namespace

cudaError_t launch_conv_fwd(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream)
{
    return by_type<kFwd>(a, dtype, stream);
}
cudaError_t launch_conv_step(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream)
{
    return by_type<kStep>(a, dtype, stream);
}
cudaError_t launch_conv_bwd(const ConvArgs& a, kda_dtype dtype, cudaStream_t stream)
{
    return by_type<kBwd>(a, dtype, stream);
}

size_t conv_bwd_workspace(int B, int T, int C, int W, int N, kda_dtype)
{
    const Shape s = bwd_shape((long long)B * T, C, N);
    return (size_t)s.tiles * (W + 1) * C * sizeof(float);
}

}  // namespace kda
