// Gated delta rule on the CUDA cores: the one-token step, and the recurrent
// forward and backward over a sequence, in float32 for any sizes and types.
//
// State S [P, N] per (b, h), q and k of group h / (H / G):
//     F = exp(g_t) S_{t-1},  w = v_t - F k_t,  u = beta_t w,
//     S_t = F + u k_t^T,     y_t = scale S_t q_t = scale (F q_t + u (k_t . q_t))
// Every row p of S evolves on its own given k, q, g and beta, so a row is
// owned by a group of 8 lanes: lane j of the group holds the columns
// n = (i 8 + j) VW .. + VW (VW = 4 where N allows 16-byte rows, else 1), and the
// two dots S k and S q are taken in one pass, three shuffles each.
#include "common.cuh"
#include "f32x2.cuh"
#include "launch.h"

namespace ssd {
namespace {

using namespace delta;

constexpr int kThreads = 128, kRowsPass = kThreads / 8;  // rows a block handles at once

__device__ __forceinline__ float group_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    return v;
}

// column of element e of lane j
template <int VW> __device__ __forceinline__ int col_of(int e, int j) {
    return ((e / VW) * 8 + j) * VW + e % VW;
}

template <int VW, int NE, typename T>
__device__ __forceinline__ void load_row(float (&s)[NE], const T *row, int N, int j) {
#pragma unroll
    for (int e = 0; e < NE; e += VW) {
        const int n = col_of<VW>(e, j);
        if constexpr (VW == 4) {
            const float4 v = n < N ? ld4(row + n) : make_float4(0.f, 0.f, 0.f, 0.f);
            s[e] = v.x, s[e + 1] = v.y, s[e + 2] = v.z, s[e + 3] = v.w;
        } else {
            s[e] = n < N ? to_f32(row[n]) : 0.f;
        }
    }
}

template <int VW, int NE>
__device__ __forceinline__ void store_row(const float (&s)[NE], float *row, int N, int j) {
#pragma unroll
    for (int e = 0; e < NE; e += VW) {
        const int n = col_of<VW>(e, j);
        if (n >= N) continue;
        if constexpr (VW == 4)
            *reinterpret_cast<float4 *>(row + n) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
        else
            row[n] = s[e];
    }
}

// The same as pairs of float32.
template <int VW, int NE>
__device__ __forceinline__ void load_pairs(uint64_t (&s)[NE / 2], const float *row, int N, int j) {
    float x[NE];
    load_row<VW, NE>(x, row, N, j);
#pragma unroll
    for (int e = 0; e < NE; e += 2) s[e / 2] = f2(x[e], x[e + 1]);
}
template <int VW, int NE>
__device__ __forceinline__ void store_pairs(const uint64_t (&s)[NE / 2], float *row, int N, int j) {
    float x[NE];
#pragma unroll
    for (int e = 0; e < NE; e += 2) un2(s[e / 2], x[e], x[e + 1]);
    store_row<VW, NE>(x, row, N, j);
}
__device__ __forceinline__ float pair_sum(uint64_t v) {
    float x, y;
    un2(v, x, y);
    return x + y;
}

// ------------------------------------------------------------------- the step
// Bound by HBM: the state is read and written once. A block covers
// rows [p0, p0 + rows_per_block) of one (b, h). With N 128, P 64: 54 us for 64
// rows of 80 heads, 6.2 TB/s (58 us where a row is requested when the one before is
// done); a state of 24 heads takes 1.9 us in a graph, the latency of a launch.
template <typename T, int VW, int NE>
__global__ void __launch_bounds__(kThreads) delta_step_kernel(DeltaStepArgs a, int rows_per_block) {
    pdl_enter();
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.H);
    const int64_t b = bh / a.H;
    const int i = h / (int)(a.H / a.G), N = (int)a.N, P = (int)a.P;
    const int p0 = blockIdx.y * rows_per_block, p1 = imin(P, p0 + rows_per_block);
    T *y = (T *)a.y + bh * P;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    if (slot < 0 || slot >= a.nslots) {  // an idle row: no state, zero output
        for (int p = p0 + threadIdx.x; p < p1; p += kThreads) y[p] = from_f32<T>(0.f);
        return;
    }
    const int j = threadIdx.x & 7, row = threadIdx.x >> 3;
    const int64_t base = (slot * a.H + h) * (int64_t)P * N;
    const T *v = (const T *)a.v + bh * P;
    float next[NE], next_v;  // the next row of this thread, on its way while one is worked on
    auto fetch = [&](int p) {
        load_row<VW, NE>(next, a.state + base + (int64_t)p * N, N, j);
        next_v = to_f32(v[p]);
    };
    fetch(imin(p0 + row, p1 - 1));
    float kv[NE], qv[NE], kq = 0.f;
    load_row<VW, NE>(kv, (const T *)a.k + (b * a.G + i) * N, N, j);
    load_row<VW, NE>(qv, (const T *)a.q + (b * a.G + i) * N, N, j);
#pragma unroll
    for (int e = 0; e < NE; ++e) kq = fmaf(kv[e], qv[e], kq);
    kq = group_sum(kq);
    const float alpha = expf(to_f32(((const T *)a.g)[bh])), beta = to_f32(((const T *)a.beta)[bh]);
    for (int p = p0 + row; p < p1 + row; p += kRowsPass) {  // whole warps stay in for the shuffles
        const bool on = p < p1;
        float s[NE];
#pragma unroll
        for (int e = 0; e < NE; ++e) s[e] = next[e];
        const float vp = next_v;
        if (p + kRowsPass < p1) fetch(p + kRowsPass);
        float sk = 0.f, sq = 0.f;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            s[e] *= alpha;
            sk = fmaf(s[e], kv[e], sk);
            sq = fmaf(s[e], qv[e], sq);
        }
        sk = group_sum(sk);
        sq = group_sum(sq);
        if (!on) continue;
        const float u = beta * (vp - sk);
#pragma unroll
        for (int e = 0; e < NE; ++e) s[e] = fmaf(u, kv[e], s[e]);
        store_row<VW, NE>(s, a.new_state + base + (int64_t)p * N, N, j);
        if (j == 0) y[p] = from_f32<T>(a.scale * fmaf(u, kq, sq));
    }
}

// --------------------------------------------------- recurrent forward
// One block per (b, h, 16 rows): the state stays in registers over the whole
// sequence. What bounds it is the latency of a token, from the old state over
// the sums of 8 lanes to the new state; so everything else is off that way: 16
// tokens are staged in shared memory while the next 16 are on their way to
// registers, a token's k and q are read while the one before it is done, k . q is
// formed at staging, the dots are taken of S_{t-1}, the decay coming after, and y
// leaves once per 16 tokens. float32, 12 heads of P 64, N 64, 777 tokens: 147 us,
// 360 cycles a token, a third of it the three dependent shuffles (310 us with loads of
// each 32 tokens waited for and the decay first).
// With `ckpt` the states entering every ckpt_len-th token are stored for the backward.
constexpr int kStage = kRowsPass;  // tokens staged at once; group t of lanes forms k . q of token t

template <typename T, int VW, int NE>
__global__ void __launch_bounds__(kThreads) delta_recurrent_kernel(DeltaArgs a, float *ckpt, int ckpt_len) {
    pdl_enter();
    extern __shared__ float sm[];
    const int N = (int)a.N, P = (int)a.P;
    float *sk = sm, *sq = sk + kStage * N;
    __shared__ float sv[kStage * kRowsPass], sy[kStage * kRowsPass];
    __shared__ float4 sx[kStage];
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.H);
    const int64_t b = bh / a.H;
    const int i = h / (int)(a.H / a.G);
    const int p0 = blockIdx.y * kRowsPass;
    const int j = threadIdx.x & 7, row = threadIdx.x >> 3, p = p0 + row;
    const bool on = p < P;
    const int64_t len = seq_len(a.seqlens, b, a.L);
    if (a.status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.status = 0;
    const int64_t nck = ckpt ? (a.L + ckpt_len - 1) / ckpt_len : 0;
    uint64_t s[NE / 2] = {};
    if (a.init && on) load_pairs<VW, NE>(s, a.init + (bh * P + p) * N, N, j);
    // Staged element x = e kThreads + thread of [kStage][N] (NE kThreads >= kStage N), of v [kStage][rows].
    T rk[NE], rq[NE], rv[2], rg, rb;
    static_assert(kStage * 8 == kThreads && kStage * kRowsPass == 2 * kThreads, "the shares of a thread");
    auto fetch = [&](int64_t t0) {
        const int nt = (int)imin<int64_t>(kStage, len - t0);
        if (nt <= 0) return;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int x = e * kThreads + threadIdx.x, t = x / N;
            const int64_t at = ((b * a.L + t0 + t) * a.G + i) * N + (x - t * N);
            rk[e] = t < nt ? ((const T *)a.k)[at] : from_f32<T>(0.f);
            rq[e] = t < nt && a.q ? ((const T *)a.q)[at] : from_f32<T>(0.f);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x = e * kThreads + threadIdx.x, t = x / kRowsPass, r = x % kRowsPass;
            rv[e] = t < nt && p0 + r < P ? ((const T *)a.v)[((b * a.L + t0 + t) * a.H + h) * P + p0 + r] : from_f32<T>(0.f);
        }
        if ((int)threadIdx.x < nt) {
            const int64_t at = (b * a.L + t0 + threadIdx.x) * a.H + h;
            rg = ((const T *)a.g)[at];
            rb = ((const T *)a.beta)[at];
        }
    };
    fetch(0);
    for (int64_t t0 = 0; t0 < len; t0 += kStage) {
        const int nt = (int)imin<int64_t>(kStage, len - t0);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int x = e * kThreads + threadIdx.x;
            if (x < kStage * N) sk[x] = to_f32(rk[e]), sq[x] = to_f32(rq[e]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) sv[e * kThreads + threadIdx.x] = to_f32(rv[e]);
        if ((int)threadIdx.x < nt) sx[threadIdx.x] = make_float4(expf(to_f32(rg)), to_f32(rb), 0.f, 0.f);
        __syncthreads();
        fetch(t0 + kStage);
        uint64_t kv[NE / 2], qv[NE / 2];
        {
            uint64_t d = 0;
            load_pairs<VW, NE>(kv, sk + row * N, N, j);
            load_pairs<VW, NE>(qv, sq + row * N, N, j);
#pragma unroll
            for (int e = 0; e < NE / 2; ++e) d = fma2(kv[e], qv[e], d);
            const float kq = group_sum(pair_sum(d));
            if (j == 0) sx[row].z = kq;
        }
        __syncthreads();
        constexpr bool AHEAD = NE <= 16;  // registers for two tokens' k and q
        if (AHEAD) {
            load_pairs<VW, NE>(kv, sk, N, j);
            load_pairs<VW, NE>(qv, sq, N, j);
        }
#pragma unroll 1
        for (int half = 0; half < 16; half += 8) {
            if (ckpt && half < nt && on && (half == 0 || ckpt_len == 8))
                store_pairs<VW, NE>(s, ckpt + (((bh * nck + (t0 + half) / ckpt_len) * P) + p) * N, N, j);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int t = half + x;
                if (t >= nt) break;
                uint64_t nk[NE / 2], nq[NE / 2];
                const int at = AHEAD ? imin(t + 1, kStage - 1) : t;
                load_pairs<VW, NE>(nk, sk + at * N, N, j);
                load_pairs<VW, NE>(nq, sq + at * N, N, j);
                if (!AHEAD)
#pragma unroll
                    for (int e = 0; e < NE / 2; ++e) kv[e] = nk[e], qv[e] = nq[e];
                const float4 f = sx[t];  // exp(g), beta, k . q
                const float v = sv[t * kRowsPass + row];
                const uint64_t alpha = f2(f.x, f.x);
                uint64_t d[2] = {}, o[2] = {};
#pragma unroll
                for (int e = 0; e < NE / 2; ++e) {
                    d[e & 1] = fma2(s[e], kv[e], d[e & 1]);
                    o[e & 1] = fma2(s[e], qv[e], o[e & 1]);
                    s[e] = mul2(s[e], alpha);
                }
                const float sd = group_sum(pair_sum(d[0]) + pair_sum(d[1])), so = group_sum(pair_sum(o[0]) + pair_sum(o[1]));
                const float u = f.y * fmaf(-f.x, sd, v);
                const uint64_t u2 = f2(u, u);
#pragma unroll
                for (int e = 0; e < NE / 2; ++e) {
                    s[e] = fma2(u2, kv[e], s[e]);
                    if (AHEAD) kv[e] = nk[e], qv[e] = nq[e];
                }
                if (j == 0) sy[t * kRowsPass + row] = a.scale * fmaf(u, f.z, f.x * so);
            }
        }
        __syncthreads();
        if (a.y)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int x = e * kThreads + threadIdx.x, t = x / kRowsPass, r = x % kRowsPass;
                if (t < nt && p0 + r < P) ((T *)a.y)[((b * a.L + t0 + t) * a.H + h) * P + p0 + r] = from_f32<T>(sy[x]);
            }
    }
    if (a.final_state && on) store_pairs<VW, NE>(s, a.final_state + (bh * P + p) * N, N, j);
    if (a.y)  // tokens past the sequence's length
        for (int64_t x = threadIdx.x; x < (a.L - len) * kRowsPass; x += kThreads) {
            const int64_t t = len + x / kRowsPass;
            const int r = (int)(x % kRowsPass);
            if (p0 + r < P) ((T *)a.y)[((b * a.L + t) * a.H + h) * P + p0 + r] = from_f32<T>(0.f);
        }
}

// -------------------------------------------------- recurrent backward
// One block per (b, h, 16 rows), segments of CK tokens in reverse: the states
// of a segment are recomputed from its checkpoint into shared memory, then with
// E the cotangent of S_t (rows p, all sums over n within a lane group):
//     dq_t += scale dy_t S_t     E += scale dy_t q_t^T     du = E k_t
//     dv_t = beta du             dbeta_t += du . w         dk_t += u E - beta du F
//     E -= beta du k_t^T         dg_t += <E, F>            E *= exp(g_t)
// Bound by instruction issue: every row's share of dq and dk is summed over the rows of
// a block for every token. float32, 12 heads of P 64, N 64, 777 tokens: 835 us.
// The sums over rows are taken per warp by shuffles and over the four warps in
// shared memory; sums over row blocks and over the heads of a group are left
// to delta_reduce_kernel, in a fixed order.
template <typename T, int VW, int NE, int CK>
__global__ void __launch_bounds__(kThreads) delta_recurrent_bwd_kernel(DeltaBwdArgs a) {
    pdl_enter();
    extern __shared__ float sm[];
    const int N = (int)a.f.N, P = (int)a.f.P;
    constexpr int W = kThreads / 32;
    float *st = sm;                          // [CK][NE][threads]: S_{t-1} of this thread
    float *sk = st + CK * NE * kThreads, *sq = sk + CK * N;
    float *sv = sq + CK * N, *sdy = sv + CK * kRowsPass;
    float *pq = sdy + CK * kRowsPass, *pk = pq + CK * W * N;  // [CK][W][N]
    float *pg = pk + CK * W * N, *pb = pg + CK * W;           // [CK][W]
    float *sa = pb + CK * W, *sb = sa + CK;
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.f.H);
    const int64_t b = bh / a.f.H, L = a.f.L;
    const int i = h / (int)(a.f.H / a.f.G);
    const int nrb = gridDim.y, rb = blockIdx.y, p0 = rb * kRowsPass;
    const int j = threadIdx.x & 7, row = threadIdx.x >> 3, p = p0 + row;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool on = p < P;
    const int64_t len = seq_len(a.f.seqlens, b, L), nck = (L + CK - 1) / CK;
    const float scale = a.f.scale;
    float E[NE];
    if (a.dfinal && on) {
        load_row<VW, NE>(E, a.dfinal + (bh * P + p) * N, N, j);
    } else {
#pragma unroll
        for (int e = 0; e < NE; ++e) E[e] = 0.f;
    }
    for (int64_t c = (len + CK - 1) / CK - 1; c >= 0; --c) {
        const int64_t t0 = c * CK;
        const int nt = (int)imin<int64_t>(CK, len - t0);
        __syncthreads();
        for (int x = threadIdx.x; x < nt * N; x += kThreads) {
            const int t = x / N, n = x - t * N;
            const int64_t at = ((b * L + t0 + t) * a.f.G + i) * N + n;
            sk[x] = to_f32(((const T *)a.f.k)[at]);
            sq[x] = to_f32(((const T *)a.f.q)[at]);
        }
        for (int x = threadIdx.x; x < nt * kRowsPass; x += kThreads) {
            const int t = x / kRowsPass, r = x - t * kRowsPass;
            const int64_t at = ((b * L + t0 + t) * a.f.H + h) * P + p0 + r;
            sv[x] = p0 + r < P ? to_f32(((const T *)a.f.v)[at]) : 0.f;
            sdy[x] = p0 + r < P ? scale * to_f32(((const T *)a.dy)[at]) : 0.f;
        }
        if ((int)threadIdx.x < nt) {
            const int64_t at = (b * L + t0 + threadIdx.x) * a.f.H + h;
            sa[threadIdx.x] = expf(to_f32(((const T *)a.f.g)[at]));
            sb[threadIdx.x] = to_f32(((const T *)a.f.beta)[at]);
        }
        __syncthreads();
        float s[NE], kv[NE];
        if (on) {
            load_row<VW, NE>(s, a.ckpt + ((bh * nck + c) * P + p) * N, N, j);
        } else {
#pragma unroll
            for (int e = 0; e < NE; ++e) s[e] = 0.f;
        }
        for (int t = 0; t < nt; ++t) {
#pragma unroll
            for (int e = 0; e < NE; ++e) st[(t * NE + e) * kThreads + threadIdx.x] = s[e];
            if (t + 1 == nt) break;
            load_row<VW, NE>(kv, sk + t * N, N, j);
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                s[e] *= sa[t];
                d = fmaf(s[e], kv[e], d);
            }
            const float u = sb[t] * (sv[t * kRowsPass + row] - group_sum(d));
#pragma unroll
            for (int e = 0; e < NE; ++e) s[e] = fmaf(u, kv[e], s[e]);
        }
        for (int t = nt - 1; t >= 0; --t) {
            const float alpha = sa[t], beta = sb[t], dy = sdy[t * kRowsPass + row];
            load_row<VW, NE>(kv, sk + t * N, N, j);
            float d = 0.f, du = 0.f, qv[NE];
            load_row<VW, NE>(qv, sq + t * N, N, j);
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                s[e] = alpha * st[(t * NE + e) * kThreads + threadIdx.x];  // F
                d = fmaf(s[e], kv[e], d);
                E[e] = fmaf(dy, qv[e], E[e]);
                du = fmaf(E[e], kv[e], du);
            }
            d = group_sum(d);
            du = group_sum(du);
            const float w = sv[t * kRowsPass + row] - d, u = beta * w, bdu = beta * du;
            float dg = 0.f;
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                float xq = dy * fmaf(u, kv[e], s[e]);
                float xk = u * E[e] - bdu * s[e];
                E[e] = fmaf(-bdu, kv[e], E[e]);
                dg = fmaf(E[e], s[e], dg);
                E[e] *= alpha;
                xq += __shfl_xor_sync(0xffffffffu, xq, 8);
                xk += __shfl_xor_sync(0xffffffffu, xk, 8);
                xq += __shfl_xor_sync(0xffffffffu, xq, 16);
                xk += __shfl_xor_sync(0xffffffffu, xk, 16);
                const int n = col_of<VW>(e, j);
                if (lane < 8 && n < N) {
                    pq[(t * W + warp) * N + n] = xq;
                    pk[(t * W + warp) * N + n] = xk;
                }
            }
            if (on && j == 0) ((T *)a.dv)[((b * L + t0 + t) * a.f.H + h) * P + p] = from_f32<T>(bdu);
            dg = warp_sum(dg);
            float db = j == 0 ? du * w : 0.f;
            db = warp_sum(db);
            if (lane == 0) pg[t * W + warp] = dg, pb[t * W + warp] = db;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < nt * N; x += kThreads) {
            const int t = x / N, n = x - t * N;
            float q = 0.f, k = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                q += pq[(t * W + w) * N + n];
                k += pk[(t * W + w) * N + n];
            }
            const int64_t at = (((b * L + t0 + t) * a.f.H + h) * nrb + rb) * N + n;
            a.dq_part[at] = q;
            a.dk_part[at] = k;
        }
        if ((int)threadIdx.x < nt) {
            float dg = 0.f, db = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) dg += pg[threadIdx.x * W + w], db += pb[threadIdx.x * W + w];
            const int64_t at = ((b * L + t0 + threadIdx.x) * a.f.H + h) * nrb + rb;
            a.dg_part[at] = dg;
            a.db_part[at] = db;
        }
    }
    if (a.dinit && on) store_row<VW, NE>(E, a.dinit + (bh * P + p) * N, N, j);
    for (int64_t x = threadIdx.x; x < (L - len) * kRowsPass; x += kThreads) {
        const int64_t t = len + x / kRowsPass;
        const int r = (int)(x % kRowsPass);
        if (p0 + r < P) ((T *)a.dv)[((b * L + t) * a.f.H + h) * P + p0 + r] = from_f32<T>(0.f);
    }
}

// dq, dk: sums over the heads of a group and the row blocks; dg, dbeta: over
// the row blocks. One block per (b, t); zero past the sequence's length.
template <typename T> __global__ void __launch_bounds__(256) delta_reduce_kernel(DeltaBwdArgs a, int nrb) {
    pdl_enter();
    const int64_t bt = blockIdx.x, b = bt / a.f.L, t = bt - b * a.f.L;
    const bool on = t < seq_len(a.f.seqlens, b, a.f.L);
    const int N = (int)a.f.N, G = (int)a.f.G, H = (int)a.f.H, r = H / G;
    for (int x = threadIdx.x; x < G * N; x += blockDim.x) {
        const int i = x / N, n = x - i * N;
        float q = 0.f, k = 0.f;
        if (on)
            for (int w = 0; w < r * nrb; ++w) {
                const int64_t at = ((bt * H + (int64_t)i * r) * nrb + w) * N + n;
                q += a.dq_part[at];
                k += a.dk_part[at];
            }
        ((T *)a.dq)[bt * G * N + x] = from_f32<T>(q);
        ((T *)a.dk)[bt * G * N + x] = from_f32<T>(k);
    }
    for (int h = threadIdx.x; h < H; h += blockDim.x) {
        float dg = 0.f, db = 0.f;
        if (on)
            for (int w = 0; w < nrb; ++w) {
                dg += a.dg_part[(bt * H + h) * nrb + w];
                db += a.db_part[(bt * H + h) * nrb + w];
            }
        ((T *)a.dg)[bt * H + h] = from_f32<T>(dg);
        ((T *)a.dbeta)[bt * H + h] = from_f32<T>(db);
    }
}

// Calls f(VW, NE) as integral constants for this N (at most 256).
template <int V> using Int = std::integral_constant<int, V>;
template <typename F> cudaError_t for_width(int64_t N, F f) {
    if (N % 4 == 0) {
        if (N <= 32) return f(Int<4>{}, Int<4>{});
        if (N <= 64) return f(Int<4>{}, Int<8>{});
        if (N <= 128) return f(Int<4>{}, Int<16>{});
        return f(Int<4>{}, Int<32>{});
    }
    if (N <= 32) return f(Int<1>{}, Int<4>{});
    if (N <= 128) return f(Int<1>{}, Int<16>{});
    return f(Int<1>{}, Int<32>{});
}

template <typename T> cudaError_t step_t(const DeltaStepArgs &a, cudaStream_t stream) {
    return for_width(a.N, [&](auto vw, auto ne) {
        // rows a block walks: as many passes of 16 as leave the GPU two blocks per SM (64 rows of 80 heads: 69 us
        // with 16 rows a block, 58 with 64; one row of 24 heads: 2.6 us with 16, 4.4 with 64)
        int rows = kRowsPass;
        const int64_t want = 2 * (int64_t)sm_count(1);
        while (rows < a.P && a.B * a.H * ((a.P + 2 * rows - 1) / (2 * rows)) >= want) rows *= 2;
        const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.P + rows - 1) / rows));
        return launch_programmatic(delta_step_kernel<T, vw.value, ne.value>, grid, dim3(kThreads), 0, stream, a, rows);
    });
}

template <typename T>
cudaError_t forward_t(const DeltaArgs &a, float *ckpt, int ckpt_len, cudaStream_t stream) {
    return for_width(a.N, [&](auto vw, auto ne) {
        auto kern = delta_recurrent_kernel<T, vw.value, ne.value>;
        const size_t smem = sizeof(float) * kStage * 2 * a.N;  // at most 32 KB
        const dim3 grid((unsigned)(a.B * a.H), (unsigned)((a.P + kRowsPass - 1) / kRowsPass));
        return launch_programmatic(kern, grid, dim3(kThreads), smem, stream, a, ckpt, ckpt_len);
    });
}

template <typename T> cudaError_t backward_t(const DeltaBwdArgs &a, cudaStream_t stream) {
    const int nrb = (int)((a.f.P + kRowsPass - 1) / kRowsPass);
    DeltaArgs f = a.f;
    f.y = nullptr;
    f.q = nullptr;
    f.final_state = nullptr;
    cudaError_t e = forward_t<T>(f, a.ckpt, delta_ckpt_len(a.f.N), stream);
    if (e != cudaSuccess) return e;
    e = for_width(a.f.N, [&](auto vw, auto ne) {
        constexpr int NE = decltype(ne)::value, CK = NE > 16 ? 8 : 16;
        constexpr auto kern = delta_recurrent_bwd_kernel<T, decltype(vw)::value, NE, CK>;
        auto smem_of = [](int64_t N) {
            return sizeof(float) * (CK * NE * kThreads + CK * (2 * N + 2 * kRowsPass + 2 * 4 * N + 2 * 4 + 2));
        };
        const size_t smem = smem_of(a.f.N);
        cudaError_t r = allow_shared<kern>(smem_of(8 * NE));  // 8 NE columns at most
        if (r != cudaSuccess) return r;
        return launch_programmatic(kern, dim3((unsigned)(a.f.B * a.f.H), (unsigned)nrb), dim3(kThreads), smem, stream,
                                   a);
    });
    if (e != cudaSuccess || a.f.L == 0) return e;
    return launch_programmatic(delta_reduce_kernel<T>, dim3((unsigned)(a.f.B * a.f.L)), dim3(256), 0, stream, a, nrb);
}

}  // namespace

int delta_ckpt_len(int64_t N) { return N > 128 ? 8 : 16; }
int delta_row_blocks(int64_t P) { return (int)((P + kRowsPass - 1) / kRowsPass); }

cudaError_t launch_delta_step(int io, const DeltaStepArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? step_t<__nv_bfloat16>(a, stream) : step_t<float>(a, stream);
}

cudaError_t launch_delta_recurrent(const DeltaArgs &a, cudaStream_t stream) {
    return a.io == IO_BF16 ? forward_t<__nv_bfloat16>(a, nullptr, 1, stream) : forward_t<float>(a, nullptr, 1, stream);
}

cudaError_t launch_delta_recurrent_bwd(const DeltaBwdArgs &a, cudaStream_t stream) {
    return a.f.io == IO_BF16 ? backward_t<__nv_bfloat16>(a, stream) : backward_t<float>(a, stream);
}

}  // namespace ssd
