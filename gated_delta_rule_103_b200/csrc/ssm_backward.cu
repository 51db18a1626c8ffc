// Backward pass of the selective state-space scan (ssm_scan.cu has the
// forward).  With dy = d_out silu(z) and g_t the adjoint of h_t:
//
//     g_t = C_t dy_t + a_{t+1} g_{t+1}                  (a g of the unit behind, or d_final_state)
//     dC_t = sum_d dy_t h_t           dB_t = sum_d g_t dt u
//     du   = dt (g . B) + skip dy     d dt = u (g . B) + sum_s g_t a_t h_{t-1} A
//     dA   = sum_t g_t a_t h_{t-1} dt
//     dz   = d_out y silu'(z)         d delta = d dt softplus'(delta + bias)
//
// A block walks its unit forward once, leaving the state at every tile's entry
// in the workspace, then backward tile by tile: the tile's states are computed
// again into registers and used up from its last token to its first.  Sums
// over a channel's lanes and over a warp's channels are folded (ssm_common.cuh),
// the warps' in shared memory, the blocks' and units' by kernels in a fixed
// order, so that results do not change from run to run.
//
// Where sequences are cut into units, a pass before it gives every unit its
// end state from zero, its sum of dt, and the adjoint it hands to the unit in
// front, sum_t (prod_{s <= t} a_s) C_t dy_t, all in one walk.
#include "ssm_common.cuh"

namespace kda {
namespace {

using namespace ssm;

constexpr int kThreads = 256;

template <int L>
using BTile = Tile<L, 4, (L == 4 || L == 8) ? 16 : 8, kThreads>;

template <typename T>
struct BwdParams {
    Params<T> f;
    const T* d_out;
    const float* d_fin;
    float *gu, *gdelta, *gz, *ginit;
    float* exits;    // per slot [D][S]: adjoint handed to the unit in front, then the one from behind
    float* entries;  // per tile [D][S]: state at the tile's entry
    float* part_bc;  // [cpb][tokens][G][2][S]
    float* part_A;   // per slot [D][S]
    float* part_d;   // per slot [2][D]: skip, delta_bias
};

// What both passes do to a tile's (token, channel) operands: dt, dt u and dy
// as fp32 in shared memory.
struct Elem {
    float dt, du, dy, pad;
};

template <typename T, typename Tl, bool kY>
struct Feed {
    ChannelRows<T, Tl> u, d, z, o;
    StateRows<T, Tl, kY> bc;
    __device__ __forceinline__ void fetch(const BwdParams<T>& p, int t, int end, int c0, int nch, int g,
                                          int tid)
    {
        const int q4 = (tid % Tl::Q) * 4, nq = nch - q4, D = p.f.D;
        const size_t at = (size_t)(t + tid / Tl::Q) * D + c0 + q4;
        const int left = (end - t < Tl::TT ? end - t : Tl::TT) - tid / Tl::Q;
        u.load(p.f.u, at, D, left, nq, p.f.vec_d, tid);
        d.load(p.f.delta, at, D, left, nq, p.f.vec_d, tid);
        if (kY) {
            if (p.f.z) z.load(p.f.z, at, D, left, nq, p.f.vec_d, tid);
            o.load(p.d_out, at, D, left, nq, p.f.vec_d, tid);
        }
        bc.load(p.f, t, end, g, tid);
    }
    __device__ __forceinline__ void stage(const BwdParams<T>& p, int t, int end, const float (&bias)[4],
                                          Elem* s, float* sB, float* sC, float* dt_sum, int tid)
    {
        const int q4 = (tid % Tl::Q) * 4;
#pragma unroll
        for (int k = 0; k < Tl::IPT; ++k) {
            const int tt = (tid + k * kThreads) / Tl::Q;
            if (tt >= Tl::TT) break;
            float x[4], dv[4], dy[4] = {0.f, 0.f, 0.f, 0.f}, zz[4];
            u.r[k].get(x);
            d.r[k].get(dv);
            if (kY) {
                o.r[k].get(dy);
                if (p.f.z) {
                    z.r[k].get(zz);
#pragma unroll
                    for (int i = 0; i < 4; ++i) dy[i] *= silu(zz[i]);
                }
            }
            const bool in = t + tt < end;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = dv[i] + bias[i];
                if (p.f.softplus) v = softplus(v);
                if (!in) v = 0.f;
                if (dt_sum) dt_sum[i] += v;
                *reinterpret_cast<float4*>(&s[tt * Tl::CH + q4 + i]) = make_float4(v, v * x[i], dy[i], 0.f);
            }
        }
        bc.put(sB, sC, tid);
    }
};

// End state from zero, sum of dt and handed-on adjoint of every unit.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 2)
kda_ssm_bwd_carry_kernel(BwdParams<T> p)
{
    using Tl = BTile<L>;
    constexpr int CH = Tl::CH, TT = Tl::TT, SP = Tl::SP, Q = Tl::Q;
    extern __shared__ __align__(16) unsigned char smem[];
    Elem* s_e = reinterpret_cast<Elem*>(smem);                      // [2][TT][CH]
    float* s_B = reinterpret_cast<float*>(s_e + 2 * TT * CH);       // [2][TT][SP]
    float* s_C = s_B + 2 * TT * SP;                                 // [2][TT][SP]
    const int tid = threadIdx.x;
    const int across = p.f.G * p.f.cpb;
    const int slot = blockIdx.x / across;
    const int gb = (int)(blockIdx.x % across), g = gb / p.f.cpb;
    int n, seg, t0, end;
    bool last;
    if (!p.f.units.locate(slot, n, seg, last, t0, end)) return;
    if (seg == 0 && last) return;
    const int cg = (gb % p.f.cpb) * CH;
    const int nch = p.f.Dg - cg < CH ? p.f.Dg - cg : CH;
    const int c0 = g * p.f.Dg + cg;
    const int ch = tid / L, s0 = (tid % L) * 4;
    const bool chan = ch < nch;
    const size_t row = (size_t)(c0 + (chan ? ch : 0)) * p.f.S;
    float A[4], bias[4], dt_sum[4];
    const int q4 = (tid % Q) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A[i] = chan && s0 + i < p.f.S ? p.f.A[row + s0 + i] * kLog2e : 0.f;
        dt_sum[i] = 0.f;
        bias[i] = p.f.delta_bias && q4 + i < nch ? p.f.delta_bias[c0 + q4 + i] : 0.f;
    }
    const float2 A01 = make_float2(A[0], A[1]), A23 = make_float2(A[2], A[3]);
    float2 h01 = both(0.f), h23 = h01, R01 = h01, R23 = h01, P01 = both(1.f), P23 = P01;
    Feed<T, Tl, true> feed;
    feed.fetch(p, t0, end, c0, nch, g, tid);
    feed.stage(p, t0, end, bias, s_e, s_B, s_C, dt_sum, tid);
    if (t0 + TT < end) feed.fetch(p, t0 + TT, end, c0, nch, g, tid);
    __syncthreads();
    int buf = 0;
    for (int t = t0; t < end; t += TT, buf ^= 1) {
        if (t + TT < end) {
            const int nb = buf ^ 1;
            feed.stage(p, t + TT, end, bias, s_e + nb * TT * CH, s_B + nb * TT * SP, s_C + nb * TT * SP, dt_sum, tid);
            if (t + 2 * TT < end) feed.fetch(p, t + 2 * TT, end, c0, nch, g, tid);
        }
#pragma unroll 4
        for (int j = 0; j < TT; ++j) {
            const float4 e = *reinterpret_cast<const float4*>(&s_e[(buf * TT + j) * CH + ch]);
            const float4 B = *reinterpret_cast<const float4*>(&s_B[(buf * TT + j) * SP + s0]);
            const float4 C = *reinterpret_cast<const float4*>(&s_C[(buf * TT + j) * SP + s0]);
            const float2 dt = both(e.x), du = both(e.y), dy = both(e.z);
            const float2 a01 = ex2(mul2(dt, A01)), a23 = ex2(mul2(dt, A23));
            h01 = fma2(a01, h01, mul2(du, make_float2(B.x, B.y)));
            h23 = fma2(a23, h23, mul2(du, make_float2(B.z, B.w)));
            P01 = mul2(P01, a01);
            P23 = mul2(P23, a23);
            R01 = fma2(P01, mul2(dy, make_float2(C.x, C.y)), R01);
            R23 = fma2(P23, mul2(dy, make_float2(C.z, C.w)), R23);
        }
        __syncthreads();
    }
    const float h[4] = {h01.x, h01.y, h23.x, h23.y}, R[4] = {R01.x, R01.y, R23.x, R23.y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (chan && s0 + i < p.f.S) {
            p.f.ends[(size_t)slot * p.f.D * p.f.S + row + s0 + i] = h[i];
            p.exits[(size_t)slot * p.f.D * p.f.S + row + s0 + i] = R[i];
        }
    float* red = reinterpret_cast<float*>(smem);
    if (tid / Q < TT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) red[(tid / Q) * CH + q4 + i] = dt_sum[i];
    }
    __syncthreads();
    if (tid < nch) {
        float s = 0.f;
        for (int r = 0; r < Tl::ROWS; ++r) s += red[r * CH + tid];
        p.f.steps[(size_t)slot * p.f.D + c0 + tid] = s;
    }
}

// The adjoint that enters every unit from behind, in place of the one it hands
// on: c <- exp(A sum dt) c + R, from a sequence's last unit to its first.
__global__ void __launch_bounds__(256)
kda_ssm_bwd_chain_kernel(const float* __restrict__ A, const float* __restrict__ d_fin, float* exits,
                         const float* __restrict__ steps, Units units, int D, int S)
{
    const size_t DS = (size_t)D * S;
    const int per = (int)((DS + 255) / 256);
    const int n = (int)(blockIdx.x / per);
    const size_t i = (size_t)(blockIdx.x % per) * 256 + threadIdx.x;
    if (i >= DS) return;
    const float a = A[i] * kLog2e;
    const int first = units.first(n);
    const int cnt = units.count(n);
    float c = d_fin ? d_fin[(size_t)n * DS + i] : 0.f;
    float* e = exits + (size_t)first * DS + i;
    const float* st = steps + (size_t)first * D + i / S;
    constexpr int U = 4;
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
                c = fmaf(ex2(a * dt[j]), c, r[j]);
            }
    }
}

template <typename T, int L>
constexpr size_t bwd_smem()
{
    using Tl = BTile<L>;
    // staged operands, results per (token, channel), warps' sums of dB and dC,
    // entry states of every four tokens
    return sizeof(float) * (2 * Tl::TT * Tl::CH * 4 + 4 * Tl::TT * Tl::SP + 3 * Tl::TT * (Tl::CH + 8) +
                            (kThreads / 32) * Tl::TT * 2 * Tl::SP + Tl::TT * kThreads);
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 2)
kda_ssm_bwd_kernel(BwdParams<T> p)
{
    using Tl = BTile<L>;
    constexpr int CH = Tl::CH, TT = Tl::TT, SP = Tl::SP, Q = Tl::Q, IPT = Tl::IPT;
    constexpr int YP = CH + 8;  // no two of a warp's results in one bank
    constexpr int WARPS = kThreads / 32, NL = 32 / L;               // channels of a warp
    extern __shared__ __align__(16) unsigned char smem[];
    Elem* s_e = reinterpret_cast<Elem*>(smem);                      // [2][TT][CH]
    float* s_B = reinterpret_cast<float*>(s_e + 2 * TT * CH);       // [2][TT][SP]
    float* s_C = s_B + 2 * TT * SP;                                 // [2][TT][SP]
    float* s_o = s_C + 2 * TT * SP;                                 // [3][TT][YP]: g.B, sum g a h A, C.h
    float* s_w = s_o + 3 * TT * YP;                                 // [WARPS][TT][2][SP]
    float4* s_m = reinterpret_cast<float4*>(s_w + WARPS * TT * 2 * SP);  // [TT / 4][threads]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.f.D, S = p.f.S;
    const int across = p.f.G * p.f.cpb;
    const int slot = blockIdx.x / across;
    const int gb = (int)(blockIdx.x % across), g = gb / p.f.cpb;
    const int cg = (gb % p.f.cpb) * CH;
    const int nch = p.f.Dg - cg < CH ? p.f.Dg - cg : CH;
    const int c0 = g * p.f.Dg + cg;
    const int ch = tid / L, s0 = (tid % L) * 4;
    const bool chan = ch < nch;
    const size_t row = (size_t)(c0 + (chan ? ch : 0)) * S;
    const size_t DS = (size_t)D * S;
    int n, seg, t0, end;
    bool last;
    if (!p.f.units.locate(slot, n, seg, last, t0, end)) {
        // an empty slot adds nothing to the parameters' gradients
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (chan && s0 + i < S) p.part_A[(size_t)slot * DS + row + s0 + i] = 0.f;
        if (tid < nch) p.part_d[(size_t)slot * 2 * D + c0 + tid] = p.part_d[((size_t)slot * 2 + 1) * D + c0 + tid] = 0.f;
        return;
    }
    // tiles of all units, numbered so that no count of earlier ones is needed
    const int tile0 = t0 / TT + slot, tiles = (end - t0 + TT - 1) / TT;

    float A[4], h[4], c[4], bias[4], skip[4];
    const int q4 = (tid % Q) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool ok = chan && s0 + i < S;
        const size_t at = row + s0 + i;
        A[i] = ok ? p.f.A[at] * kLog2e : 0.f;
        h[i] = c[i] = 0.f;
        if (ok) {
            if (p.f.ends && seg > 0) h[i] = p.f.ends[(size_t)slot * DS + at];
            else if (p.f.init) h[i] = p.f.init[(size_t)n * DS + at];
            if (p.f.ends && !last) c[i] = p.exits[(size_t)slot * DS + at];
            else if (p.d_fin) c[i] = p.d_fin[(size_t)n * DS + at];
        }
        bias[i] = p.f.delta_bias && q4 + i < nch ? p.f.delta_bias[c0 + q4 + i] : 0.f;
        skip[i] = p.f.skip && q4 + i < nch ? p.f.skip[c0 + q4 + i] : 0.f;
    }

    const float2 A01 = make_float2(A[0], A[1]), A23 = make_float2(A[2], A[3]);
    float2 h01 = make_float2(h[0], h[1]), h23 = make_float2(h[2], h[3]);
    float2 c01 = make_float2(c[0], c[1]), c23 = make_float2(c[2], c[3]);
    float2 dA01 = both(0.f), dA23 = dA01;
    auto advance = [&](int j, float2& x01, float2& x23) {
        const float2 dd = *reinterpret_cast<const float2*>(&s_e[j * CH + ch]);
        const float4 B = *reinterpret_cast<const float4*>(&s_B[j * SP + s0]);
        const float2 dt = both(dd.x), du = both(dd.y);
        x01 = fma2(ex2(mul2(dt, A01)), x01, mul2(du, make_float2(B.x, B.y)));
        x23 = fma2(ex2(mul2(dt, A23)), x23, mul2(du, make_float2(B.z, B.w)));
    };

    // forward: the state at every tile's entry
    {
        Feed<T, Tl, false> feed;
        feed.fetch(p, t0, end, c0, nch, g, tid);
        feed.stage(p, t0, end, bias, s_e, s_B, s_C, nullptr, tid);
        if (t0 + TT < end) feed.fetch(p, t0 + TT, end, c0, nch, g, tid);
        __syncthreads();
        int buf = 0;
        for (int k = 0; k < tiles; ++k, buf ^= 1) {
            const int t = t0 + k * TT;
            if (t + TT < end) {
                const int nb = buf ^ 1;
                feed.stage(p, t + TT, end, bias, s_e + nb * TT * CH, s_B + nb * TT * SP, s_C, nullptr, tid);
                if (t + 2 * TT < end) feed.fetch(p, t + 2 * TT, end, c0, nch, g, tid);
            }
            float* e = p.entries + (size_t)(tile0 + k) * DS + row + s0;
            if (chan) {
                const float x[4] = {h01.x, h01.y, h23.x, h23.y};
                store4(e, x, p.f.vec_s && s0 < S, S - s0);
            }
            if (k + 1 < tiles)
#pragma unroll 4
                for (int j = 0; j < TT; ++j) advance(buf * TT + j, h01, h23);
            __syncthreads();
        }
    }

    // backward, from the last tile (its entry state is in h) to the first
    Feed<T, Tl, true> feed;
    float sum_skip[4] = {0.f, 0.f, 0.f, 0.f}, sum_bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (tiles > 0) feed.fetch(p, t0 + (tiles - 1) * TT, end, c0, nch, g, tid);
    for (int k = tiles - 1; k >= 0; --k) {
        const int t = t0 + k * TT;
        feed.stage(p, t, end, bias, s_e, s_B, s_C, nullptr, tid);
        __syncthreads();
        // The tile goes by in fours: their entry states first (each thread's own
        // in shared memory), then from the last four to the first their states
        // and decays again, held in registers.
#pragma unroll 1
        for (int q = 0; q < TT / 4; ++q) {
            s_m[q * kThreads + tid] = make_float4(h01.x, h01.y, h23.x, h23.y);
            if (q + 1 < TT / 4)
#pragma unroll
                for (int j = 0; j < 4; ++j) advance(q * 4 + j, h01, h23);
        }
        float2 dA01_t = both(0.f), dA23_t = dA01_t;
#pragma unroll 1
        for (int tb = TT - 4; tb >= 0; tb -= 4) {
            const float4 m = s_m[tb / 4 * kThreads + tid];
            const float2 b01 = make_float2(m.x, m.y), b23 = make_float2(m.z, m.w);
            float2 hs[4][2], as[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 dd = *reinterpret_cast<const float2*>(&s_e[(tb + j) * CH + ch]);
                const float4 B = *reinterpret_cast<const float4*>(&s_B[(tb + j) * SP + s0]);
                const float2 dt = both(dd.x), du = both(dd.y);
                as[j][0] = ex2(mul2(dt, A01));
                as[j][1] = ex2(mul2(dt, A23));
                hs[j][0] = fma2(as[j][0], j ? hs[j > 0 ? j - 1 : 0][0] : b01, mul2(du, make_float2(B.x, B.y)));
                hs[j][1] = fma2(as[j][1], j ? hs[j > 0 ? j - 1 : 0][1] : b23, mul2(du, make_float2(B.z, B.w)));
            }
            float o[3][4];  // [what][token]
#pragma unroll
            for (int jj = 3; jj >= 0; --jj) {
                const int tok = tb + jj;
                const float4 e = *reinterpret_cast<const float4*>(&s_e[tok * CH + ch]);
                const float4 B = *reinterpret_cast<const float4*>(&s_B[tok * SP + s0]);
                const float4 C = *reinterpret_cast<const float4*>(&s_C[tok * SP + s0]);
                const float2 dt = both(e.x), du = both(e.y), dy = both(e.z);
                const float2 B01 = make_float2(B.x, B.y), B23 = make_float2(B.z, B.w);
                const float2 C01 = make_float2(C.x, C.y), C23 = make_float2(C.z, C.w);
                const float2 g01 = fma2(C01, dy, c01), g23 = fma2(C23, dy, c23);
                c01 = mul2(as[jj][0], g01);
                c23 = mul2(as[jj][1], g23);
                const float2 w01 = mul2(c01, jj ? hs[jj > 0 ? jj - 1 : 0][0] : b01);
                const float2 w23 = mul2(c23, jj ? hs[jj > 0 ? jj - 1 : 0][1] : b23);
                dA01_t = fma2(w01, dt, dA01_t);
                dA23_t = fma2(w23, dt, dA23_t);
                const float2 gB = fma2(g01, B01, mul2(g23, B23));
                const float2 wA = fma2(w01, A01, mul2(w23, A23));
                const float2 hC = fma2(hs[jj][0], C01, mul2(hs[jj][1], C23));
                o[0][jj] = gB.x + gB.y;
                o[1][jj] = wA.x + wA.y;
                o[2][jj] = hC.x + hC.y;
                const float2 p0 = mul2(g01, du), p1 = mul2(g23, du);
                const float2 p2 = mul2(hs[jj][0], dy), p3 = mul2(hs[jj][1], dy);
                float bc[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
                fold<8, NL, L>(bc, lane);
                constexpr int KEEP = NL >= 8 ? 1 : 8 / NL;
                constexpr int BITS = NL >= 8 ? 3 : (NL == 4 ? 2 : (NL == 2 ? 1 : 0));
                if (lane / L < 8) {
                    const int at = fold_index<BITS>(lane, L) * KEEP;  // of {B: 0..3, C: 4..7}
#pragma unroll
                    for (int i = 0; i < KEEP; ++i) {
                        const int v = at + i;
                        s_w[((warp * TT + tok) * 2 + (v >> 2)) * SP + s0 + (v & 3)] = bc[i];
                    }
                }
            }
            constexpr int KEEP = L >= 4 ? 1 : 4 / L;
            constexpr int BITS = L >= 4 ? 2 : (L == 2 ? 1 : 0);
#pragma unroll
            for (int w = 0; w < 3; ++w) {
                if (w == 2 && !p.f.z) break;  // y is wanted for dz alone
                fold<4, L, 1>(o[w], lane);
                if (tid % L < 4) {
                    const int at = tb + fold_index<BITS>(lane, 1) * KEEP;
#pragma unroll
                    for (int i = 0; i < KEEP; ++i) s_o[(w * TT + at + i) * YP + ch] = o[w][i];
                }
            }
        }
        // a tile's sum first: long sums of small terms keep their digits
        dA01.x += dA01_t.x;
        dA01.y += dA01_t.y;
        dA23.x += dA23_t.x;
        dA23.y += dA23_t.y;
        if (k > 0) {
            float next[4] = {0.f, 0.f, 0.f, 0.f};
            const float* e = p.entries + (size_t)(tile0 + k - 1) * DS + row + s0;
            if (chan) {
                if (p.f.vec_s) {
                    if (s0 < S) load_vec<4>(e, next);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (s0 + i < S) next[i] = e[i];
                }
            }
            h01 = make_float2(next[0], next[1]);
            h23 = make_float2(next[2], next[3]);
        }
        __syncthreads();
        // gradients per (token, channel)
#pragma unroll
        for (int k2 = 0; k2 < IPT; ++k2) {
            const int tt = (tid + k2 * kThreads) / Q;
            if (tt >= TT || t + tt >= end || q4 >= nch) continue;
            float x[4], dl[4], zz[4], dout[4], gb4[4], sa[4], y[4], r[4];
            feed.u.r[k2].get(x);
            feed.d.r[k2].get(dl);
            feed.o.r[k2].get(dout);
            load_vec<4>(&s_o[(0 * TT + tt) * YP + q4], gb4);
            load_vec<4>(&s_o[(1 * TT + tt) * YP + q4], sa);
            const size_t at = (size_t)(t + tt) * D + c0 + q4;
            if (p.f.z) {
                feed.z.r[k2].get(zz);
                load_vec<4>(&s_o[(2 * TT + tt) * YP + q4], y);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float sg = sigmoid(zz[i]);
                    r[i] = dout[i] * fmaf(skip[i], x[i], y[i]) * (sg * fmaf(zz[i], 1.f - sg, 1.f));
                    dout[i] *= zz[i] * sg;
                }
                store4(p.gz + at, r, p.f.vec_d, nch - q4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float dt = s_e[tt * CH + q4 + i].dt;
                r[i] = fmaf(dt, gb4[i], skip[i] * dout[i]);
                sum_skip[i] = fmaf(dout[i], x[i], sum_skip[i]);
            }
            store4(p.gu + at, r, p.f.vec_d, nch - q4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[i] = fmaf(x[i], gb4[i], sa[i] * kLn2);
                if (p.f.softplus) r[i] *= sigmoid(dl[i] + bias[i]);
                sum_bias[i] += r[i];
            }
            store4(p.gdelta + at, r, p.f.vec_d, nch - q4);
        }
        if (k > 0) feed.fetch(p, t - TT, end, c0, nch, g, tid);
        // dB and dC of this block's channels
        for (int q = tid; q < TT * 2 * SP; q += kThreads) {
            const int j = q / (2 * SP), ws = q - j * 2 * SP, s = ws % SP;
            if (t + j >= end || s >= S) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) sum += s_w[w * TT * 2 * SP + q];
            p.part_bc[((((size_t)(gb % p.f.cpb) * p.f.units.s.total + t + j) * p.f.G + g) * 2 + ws / SP) * S + s] = sum;
        }
        __syncthreads();
    }

    if (chan) {
        const float dA[4] = {dA01.x, dA01.y, dA23.x, dA23.y}, c_in[4] = {c01.x, c01.y, c23.x, c23.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s0 + i < S) {
                p.part_A[(size_t)slot * DS + row + s0 + i] = dA[i];
                if (seg == 0 && p.ginit) p.ginit[(size_t)n * DS + row + s0 + i] = c_in[i];
            }
    }
    float* red = reinterpret_cast<float*>(smem);
    if (tid / Q < TT) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            red[(tid / Q) * CH + q4 + i] = sum_skip[i];
            red[(Tl::ROWS + tid / Q) * CH + q4 + i] = sum_bias[i];
        }
    }
    __syncthreads();
    if (tid < nch) {
        float a = 0.f, b = 0.f;
        for (int r = 0; r < Tl::ROWS; ++r) {
            a += red[r * CH + tid];
            b += red[(Tl::ROWS + r) * CH + tid];
        }
        p.part_d[(size_t)slot * 2 * D + c0 + tid] = a;
        p.part_d[((size_t)slot * 2 + 1) * D + c0 + tid] = b;
    }
}

// grad_B and grad_C [tokens][G][S] from the channel blocks' sums
// [cpb][tokens][G][2][S].  Rows in front of the first sequence or behind the
// last belong to none and are left alone.
__global__ void __launch_bounds__(256)
kda_ssm_bwd_bc_kernel(const float* __restrict__ part, float* __restrict__ grad_B, float* __restrict__ grad_C,
                      Seqs seqs, int G, int S, int cpb)
{
    const long long all = (long long)seqs.total * G * 2 * S;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= all) return;
    const long long row = i / (2 * S), t = row / G;
    const int ws = (int)(i - row * 2 * S);
    if (seqs.cu && (t < seqs.start(0) || t >= seqs.start(seqs.N))) return;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < cpb; ++k) s += part[(size_t)k * all + i];
    if (ws < S) grad_B[row * S + ws] = s;
    else grad_C[row * S + ws - S] = s;
}

// grad_A [D][S] (i < DS), then grad_skip and grad_delta_bias [D], from the
// units' sums: 32 values per block, eight lanes over the units.
__global__ void __launch_bounds__(256)
kda_ssm_bwd_params_kernel(const float* __restrict__ part_A, const float* __restrict__ part_d,
                          float* __restrict__ grad_A, float* __restrict__ grad_skip,
                          float* __restrict__ grad_bias, int D, int S, long long slots)
{
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long long DS = (long long)D * S, i = (long long)blockIdx.x * 32 + lane;
    const bool isA = i < DS, live = i < DS + 2 * D;
    const float* src = isA ? part_A + i : part_d + (i - DS);
    const size_t stride = isA ? (size_t)DS : (size_t)2 * D;
    float s = 0.f;
    if (live)
        for (long long k = y; k < slots; k += 8) s += src[(size_t)k * stride];
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

// Another walk over the unit's tokens is a fifth of the whole.
constexpr int kBwdFewWarps = 12, kBwdWantWarps = 12, kBwdShortest = 64;

struct Layout {
    Cut c;
    size_t slots, tiles, ends, exits, steps, entries, bc, A, d, total;
};

// Lanes that share a channel.
int bwd_lanes(int S)
{
    int l = 1;
    while (4 * l < S) l <<= 1;
    return l;
}
int bwd_tile_tokens(int L) { return L == 4 || L == 8 ? 16 : 8; }

Layout layout_of(int B, int T, int D, int S, int G, int N, int packed)
{
    Layout l = {};
    const size_t tokens = (size_t)B * T, DS = (size_t)D * S, L = bwd_lanes(S);
    l.c = cut_of(B, T, N, packed, (double)D * L / 32.0, kBwdFewWarps, kBwdWantWarps, kBwdShortest);
    l.slots = (size_t)slots_of(B, T, N, packed, l.c.len);
    const size_t CH = kThreads / L, cpb = ((size_t)(D / G) + CH - 1) / CH;
    l.tiles = tokens / bwd_tile_tokens((int)L) + l.slots + 1;
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
cudaError_t bwd(const ScanArgs& a, cudaStream_t st)
{
    const Layout l = layout_of(a.B, a.T, a.D, a.S, a.G, a.N, a.cu_seqlens != nullptr);
    char* ws = (char*)a.workspace;
    BwdParams<T> p = {};
    p.f = params_of<T>(a, l.c.len, BTile<L>::CH);
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
    p.entries = (float*)(ws + l.entries);
    p.part_bc = (float*)(ws + l.bc);
    p.part_A = (float*)(ws + l.A);
    p.part_d = (float*)(ws + l.d);
    const long long blocks = (long long)l.slots * p.f.G * p.f.cpb;
    const long long chain = ((long long)a.D * a.S + 255) / 256 * a.N;
    const long long bc = ((long long)a.B * a.T * a.G * 2 * a.S + 255) / 256;
    if (blocks > INT32_MAX || chain > INT32_MAX || bc > INT32_MAX) return cudaErrorInvalidConfiguration;
    constexpr size_t carry_smem = sizeof(float) * (2 * BTile<L>::TT * BTile<L>::CH * 4 + 4 * BTile<L>::TT * BTile<L>::SP);
    constexpr size_t smem = bwd_smem<T, L>();
    if (cudaError_t e = cudaFuncSetAttribute(kda_ssm_bwd_kernel<T, L>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem))
        return e;
    if (blocks > 0) {
        if (l.c.cut) {
            if (cudaError_t e = cudaFuncSetAttribute(kda_ssm_bwd_carry_kernel<T, L>,
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize, (int)carry_smem))
                return e;
            kda_ssm_bwd_carry_kernel<T, L><<<(unsigned)blocks, kThreads, carry_smem, st>>>(p);
            if (cudaError_t e = cudaGetLastError()) return e;
            if (cudaError_t e = launch_ssm_chain(a.A, a.initial_state, p.f.ends, p.f.steps, p.f.units, a.D, a.S, st))
                return e;
            kda_ssm_bwd_chain_kernel<<<(unsigned)chain, 256, 0, st>>>(a.A, a.d_final_state, p.exits, p.f.steps,
                                                                     p.f.units, a.D, a.S);
            if (cudaError_t e = cudaGetLastError()) return e;
        }
        kda_ssm_bwd_kernel<T, L><<<(unsigned)blocks, kThreads, smem, st>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    if (bc > 0) {
        kda_ssm_bwd_bc_kernel<<<(unsigned)bc, 256, 0, st>>>(p.part_bc, a.grad_B, a.grad_C, p.f.units.s, a.G, a.S,
                                                            p.f.cpb);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    kda_ssm_bwd_params_kernel<<<(unsigned)(((long long)a.D * (a.S + 2) + 31) / 32), 256, 0, st>>>(
        p.part_A, p.part_d, a.grad_A, a.grad_skip, a.grad_delta_bias, a.D, a.S, (long long)l.slots);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_states(const ScanArgs& a, cudaStream_t st)
{
    switch (bwd_lanes(a.S)) {
        case 1: return bwd<T, 1>(a, st);
        case 2: return bwd<T, 2>(a, st);
        case 4: return bwd<T, 4>(a, st);
        case 8: return bwd<T, 8>(a, st);
        case 16: return bwd<T, 16>(a, st);
        case 32: return bwd<T, 32>(a, st);
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
    return dtype == KDA_DTYPE_BF16 ? by_states<__nv_bfloat16>(a, st) : by_states<float>(a, st);
}

}  // namespace kda
