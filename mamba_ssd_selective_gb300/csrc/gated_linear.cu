// Gated linear recurrence, per sequence and channel, with a weight lam per channel:
//     w_t = c softplus(lam) sigmoid(r_t)     a_t = exp(-w_t)     b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
//     h_t = a_t h_{t-1} + b_t                y_t = h_t
// its backward, and one token of it over a pool of states.
//
// A run of tokens acts on the state as h -> A h + H, A the product of its a and H its result from zero, so runs are formed
// apart and joined in order. A warp holds 32 V channels of a run of tokens in registers: it forms a and b, and its (A, H);
// the warps of a block lie one behind the other in time and exchange (A, H) in shared memory; then each goes over its
// run again from the state that enters it. Tokens past a sequence's end act as a = 1, b = 0 and are not read.
#include "gated_linear.cuh"
#include "launch.h"

namespace ssd {
namespace linear {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kFwdRun = kGroup;          // tokens of a warp in the forward: a group of the 8-bit values
constexpr int kBwdRun = kState / kWarps;  // and in the backward, whose block takes the tokens between two saved states

// ------------------------------------------------------------------ forward

template <typename T, int V, bool PACK> __global__ void __launch_bounds__(kThreads) linear_fwd_kernel(LinearArgs p) {
    pdl_enter();
    constexpr int R = kFwdRun;
    __shared__ float2 run[kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + lane) * V, b = blockIdx.z, D = p.D;
    const bool on = c0 < D;
    const int64_t len = seq_len(p.seqlens, b, p.L);
    float k[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        k[v] = on ? p.c * softplus(p.lam[c0 + v]) : 0.f;
        carry[v] = on && p.init ? p.init[b * D + c0 + v] : 0.f;
    }
    const int64_t n = p.B * p.L * D;
    for (int64_t s0 = 0; s0 < p.L; s0 += (int64_t)warps * R) {
        const int64_t t0 = s0 + warp * R, at = (b * p.L + t0) * D + c0;
        const int live = on ? (int)imax<int64_t>(0, imin<int64_t>(R, len - t0)) : 0;  // tokens of the run that count
        const int rows = on ? (int)imax<int64_t>(0, imin<int64_t>(R, p.L - t0)) : 0;  // and that exist
        Raw<T, V> x[R], r[R], i[R];
#pragma unroll
        for (int t = 0; t < R; ++t)
            if (t < live) {
                x[t] = load<T, V>((const T *)p.x + at + t * D);
                r[t] = load<T, V>((const T *)p.r + at + t * D);
                i[t] = load<T, V>((const T *)p.i + at + t * D);
            }
        if constexpr (PACK) {
            if (rows > 0) {
                const int64_t groups = (p.L + kGroup - 1) / kGroup;
                const Raw<T, V> *src[3] = {x, r, i};
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    To8 to8[V];
                    Raw<uint8_t, V> code;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        uint32_t top = 0;
#pragma unroll
                        for (int t = 0; t < R; ++t) top = max(top, abs_bits(to_f32(src[z][t].v[v])));
                        code.v[v] = (uint8_t)scale_code(top);
                        to8[v] = To8(code.v[v]);
                    }
                    store<uint8_t, V>(p.scales + ((z * p.B + b) * groups + t0 / kGroup) * D + c0, code);
#pragma unroll
                    for (int t = 0; t < R; ++t) {
                        Raw<int8_t, V> q;
#pragma unroll
                        for (int v = 0; v < V; ++v) q.v[v] = to8[v](to_f32(src[z][t].v[v]));
                        if (t < rows) store<int8_t, V>(p.values + z * n + at + t * D, q);
                    }
                }
            }
        }
        float a[R][V], h[R][V], A[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gates g = gates<T>(to_f32(r[t].v[v]), to_f32(i[t].v[v]), k[v]);
                a[t][v] = t < live ? g.a : 1.f;
                h[t][v] = t < live ? g.beta2 * g.rbeta * g.iota * to_f32(x[t].v[v]) : 0.f;
                A[v] *= a[t][v];
                H[v] = fmaf(a[t][v], H[v], h[t][v]);
            }
        __syncthreads();  // the runs of the step before have been read
#pragma unroll
        for (int v = 0; v < V; ++v) run[warp][lane * V + v] = make_float2(A[v], H[v]);
        __syncthreads();
        float e[V];  // the state that enters this run
#pragma unroll
        for (int v = 0; v < V; ++v) {
            e[v] = carry[v];
            for (int w = 0; w < warps; ++w) {
                const float2 m = run[w][lane * V + v];
                carry[v] = fmaf(m.x, carry[v], m.y);
                if (w + 1 == warp) e[v] = carry[v];
            }
        }
        if (rows > 0 && p.states && t0 % kState == 0) {
            float *to = p.states + (b * ((p.L + kState - 1) / kState) + t0 / kState) * D + c0;
#pragma unroll
            for (int v = 0; v < V; ++v) to[v] = e[v];
        }
        if (p.y) {
#pragma unroll
            for (int t = 0; t < R; ++t) {
                float y[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    e[v] = fmaf(a[t][v], e[v], h[t][v]);
                    y[v] = t < live ? e[v] : 0.f;
                }
                if (t < rows) store_f32<T, V>((T *)p.y + at + t * D, y);
            }
        }
    }
    if (on && warp == 0 && p.final_state)
#pragma unroll
        for (int v = 0; v < V; ++v) p.final_state[b * D + c0 + v] = carry[v];
}

// ----------------------------------------------------------------- backward
// dh_t = dy_t + m_{t+1}, m_t = a_t dh_t (m behind the last token the gradient of the final state): the same kind of
// recurrence, backwards, a run acting as m -> A m + M. With psi_t = w_t dL/dw_t:
//     dx = dh beta iota     di = dh b (1 - iota)     psi = dh (a^2 b w / beta^2 - a w h_{t-1})     dr = psi (1 - rho)
//     dlam = sigmoid(lam) / softplus(lam) sum psi
// (psi rather than dL/dw, which has 1 / beta: w / beta goes to zero with w.) h_{t-1} is formed again from the state that
// enters each kState tokens. A block goes over its sequence from the end, kState tokens at a time.
template <typename T, int V, bool PACK> __global__ void __launch_bounds__(kThreads) linear_bwd_kernel(LinearBwdArgs p) {
    pdl_enter();
    constexpr int R = kBwdRun;
    __shared__ float run[3][kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + lane) * V, b = blockIdx.z, D = p.f.D, L = p.f.L;
    const bool on = c0 < D;
    const int64_t len = seq_len(p.f.seqlens, b, L), n = p.f.B * L * D, groups = (L + kGroup - 1) / kGroup;
    float k[V], carry[V], sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        k[v] = on ? p.f.c * softplus(p.f.lam[c0 + v]) : 0.f;
        carry[v] = on && p.dfinal ? p.dfinal[b * D + c0 + v] : 0.f;
        sum[v] = 0.f;
    }
    for (int64_t chunk = (L + kState - 1) / kState - 1; chunk >= 0; --chunk) {
        const int64_t t0 = chunk * kState + warp * R, at = (b * L + t0) * D + c0;
        const int live = on ? (int)imax<int64_t>(0, imin<int64_t>(R, len - t0)) : 0;
        const int rows = on ? (int)imax<int64_t>(0, imin<int64_t>(R, L - t0)) : 0;
        float a[R][V], bb[R][V], rho[R][V], iota[R][V], dy[R][V], A[V], H[V], M[V];
        float scale[3][V];
        if constexpr (PACK) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                Raw<uint8_t, V> code;
                if (live > 0) code = load<uint8_t, V>(p.f.scales + ((z * p.f.B + b) * groups + t0 / kGroup) * D + c0);
#pragma unroll
                for (int v = 0; v < V; ++v) scale[z][v] = scale_of(code.v[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            float x[V], r[V], i[V];
            Raw<T, V> d;
            if (t < live) d = load<T, V>((const T *)p.dy + at + t * D);
            if constexpr (PACK) {
                Raw<int8_t, V> q[3];
#pragma unroll
                for (int z = 0; z < 3; ++z)
                    if (t < live) q[z] = load<int8_t, V>(p.f.values + z * n + at + t * D);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = (float)q[0].v[v] * scale[0][v];
                    r[v] = (float)q[1].v[v] * scale[1][v];
                    i[v] = (float)q[2].v[v] * scale[2][v];
                }
            } else {
                Raw<T, V> q[3];
                if (t < live) {
                    q[0] = load<T, V>((const T *)p.f.x + at + t * D);
                    q[1] = load<T, V>((const T *)p.f.r + at + t * D);
                    q[2] = load<T, V>((const T *)p.f.i + at + t * D);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) x[v] = to_f32(q[0].v[v]), r[v] = to_f32(q[1].v[v]), i[v] = to_f32(q[2].v[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gates g = gates<T>(r[v], i[v], k[v]);
                a[t][v] = t < live ? g.a : 1.f;
                bb[t][v] = t < live ? g.beta2 * g.rbeta * g.iota * x[v] : 0.f;
                rho[t][v] = g.rho, iota[t][v] = g.iota, dy[t][v] = to_f32(d.v[v]);
                A[v] *= a[t][v];
                H[v] = fmaf(a[t][v], H[v], bb[t][v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            M[v] = 0.f;
#pragma unroll
            for (int t = R - 1; t >= 0; --t) M[v] = a[t][v] * (dy[t][v] + M[v]);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            run[0][warp][lane * V + v] = A[v];
            run[1][warp][lane * V + v] = H[v];
            run[2][warp][lane * V + v] = M[v];
        }
        __syncthreads();
        float h[V], m[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = on ? p.f.states[(b * ((L + kState - 1) / kState) + chunk) * D + c0 + v] : 0.f;
            for (int w = 0; w < warp; ++w) h[v] = fmaf(run[0][w][lane * V + v], h[v], run[1][w][lane * V + v]);
            m[v] = carry[v];
            for (int w = warps - 1; w >= 0; --w) {
                if (w == warp) m[v] = carry[v];
                carry[v] = fmaf(run[0][w][lane * V + v], carry[v], run[2][w][lane * V + v]);
            }
        }
        float before[R][V];
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[t][v] = h[v];
                h[v] = fmaf(a[t][v], h[v], bb[t][v]);
            }
#pragma unroll
        for (int t = R - 1; t >= 0; --t) {
            float dx[V], dr[V], di[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float av = a[t][v], w = k[v] * rho[t][v], beta2 = one_minus_a2(w, av);
                const float rb = rsqrt_approx(fmaxf(beta2, 1e-37f));
                const float dh = dy[t][v] + m[v];
                const float psi = dh * av * w * (av * bb[t][v] * rb * rb - before[t][v]);
                dx[v] = dh * beta2 * rb * iota[t][v];
                di[v] = dh * bb[t][v] * (1.f - iota[t][v]);
                dr[v] = psi * (1.f - rho[t][v]);
                if (t < live) {
                    sum[v] += psi;
                } else {
                    dx[v] = dr[v] = di[v] = 0.f;
                }
                m[v] = av * dh;
            }
            if (t < rows) {
                store_f32<T, V>((T *)p.dx + at + t * D, dx);
                store_f32<T, V>((T *)p.dr + at + t * D, dr);
                store_f32<T, V>((T *)p.di + at + t * D, di);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) run[0][warp][lane * V + v] = sum[v];
    __syncthreads();
    if (!on || warp != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += run[0][w][lane * V + v];
        p.part[b * D + c0 + v] = s;
        if (p.dinit) p.dinit[b * D + c0 + v] = carry[v];
    }
}

// dlam from the blocks' sums, in float64: their number grows with the batch.
__global__ void __launch_bounds__(256) linear_dlam_kernel(const float *part, const float *lam, float *dlam, int64_t rows, int64_t D) {
    pdl_enter();
    __shared__ double sum[8][33];
    const int64_t d = (int64_t)blockIdx.x * 32 + threadIdx.x;
    double s = 0.0;
    if (d < D)
        for (int64_t i = threadIdx.y; i < rows; i += 8) s += part[i * D + d];
    sum[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || d >= D) return;
    for (int j = 1; j < 8; ++j) s += sum[j][threadIdx.x];
    dlam[d] = (float)(s * softplus_ratio(lam[d]));
}

// -------------------------------------------------------------------- step
template <typename T, int V> __global__ void __launch_bounds__(256) linear_step_kernel(LinearStepArgs p) {
    pdl_enter();
    const int64_t vecs = p.D / V, j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= p.B * vecs) return;
    const int64_t b = j / vecs, c0 = (j - b * vecs) * V, at = b * p.D + c0;
    const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
    float h[V];
    if (slot < 0 || slot >= p.nslots) {  // an idle row: no state, zero output
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.f;
        store_f32<T, V>((T *)p.y + at, h);
        return;
    }
    const Raw<T, V> x = load<T, V>((const T *)p.x + at), r = load<T, V>((const T *)p.r + at), i = load<T, V>((const T *)p.i + at);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Gates g = gates<T>(to_f32(r.v[v]), to_f32(i.v[v]), p.c * softplus(p.lam[c0 + v]));
        h[v] = fmaf(g.a, p.state[slot * p.D + c0 + v], g.beta2 * g.rbeta * g.iota * to_f32(x.v[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) p.new_state[slot * p.D + c0 + v] = h[v];
    store_f32<T, V>((T *)p.y + at, h);
}

// ------------------------------------------------------------------- 8 bits
// A warp takes 32 V channels of one group of tokens.
template <typename T, int V> __global__ void __launch_bounds__(kThreads) pack8_kernel(Pack8Args p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + (threadIdx.x & 31)) * V, b = blockIdx.z, D = p.D;
    const int64_t groups = (p.L + kGroup - 1) / kGroup, g = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (c0 >= D || g >= groups) return;
    const int64_t t0 = g * kGroup, at = (b * p.L + t0) * D + c0;
    const int rows = (int)imin<int64_t>(kGroup, p.L - t0);
    const int live = (int)imax<int64_t>(0, imin<int64_t>(rows, seq_len(p.seqlens, b, p.L) - t0));
    Raw<T, V> x[kGroup];
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
        if (t < live) x[t] = load<T, V>((const T *)p.x + at + t * D);
    To8 to8[V];
    Raw<uint8_t, V> code;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < kGroup; ++t) top = max(top, abs_bits(to_f32(x[t].v[v])));
        code.v[v] = (uint8_t)scale_code(top);
        to8[v] = To8(code.v[v]);
    }
    store<uint8_t, V>(p.scales + (b * groups + g) * D + c0, code);
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
        Raw<int8_t, V> q;
#pragma unroll
        for (int v = 0; v < V; ++v) q.v[v] = to8[v](to_f32(x[t].v[v]));
        if (t < rows) store<int8_t, V>(p.values + at + t * D, q);
    }
}

template <typename T, int V> __global__ void __launch_bounds__(kThreads) unpack8_kernel(Pack8Args p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + (threadIdx.x & 31)) * V, b = blockIdx.z, D = p.D;
    const int64_t groups = (p.L + kGroup - 1) / kGroup, g = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (c0 >= D || g >= groups) return;
    const int64_t t0 = g * kGroup, at = (b * p.L + t0) * D + c0;
    const int rows = (int)imin<int64_t>(kGroup, p.L - t0);
    const Raw<uint8_t, V> code = load<uint8_t, V>(p.scales + (b * groups + g) * D + c0);
    Raw<int8_t, V> q[kGroup];
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
        if (t < rows) q[t] = load<int8_t, V>(p.values + at + t * D);
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
        float f[V];
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = (float)q[t].v[v] * scale_of(code.v[v]);
        if (t < rows) store_f32<T, V>((T *)p.out + at + t * D, f);
    }
}

// --------------------------------------------------------------------- host

// f(integral_constant V): two channels a thread where rows are a multiple of two.
template <typename F> cudaError_t for_width(int64_t D, F &&f) {
    if (D % 2 == 0) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}
unsigned tiles(int64_t D, int V) { return (unsigned)((D + 32 * V - 1) / (32 * V)); }
// Warps of a block for a sequence of L tokens in runs of R: no more than have a token.
int warps_for(int64_t L, int R) { return (int)imax<int64_t>(1, imin<int64_t>(kWarps, (L + R - 1) / R)); }

template <typename T> cudaError_t forward_t(const LinearArgs &a, cudaStream_t stream) {
    return for_width(a.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        const dim3 grid(1, tiles(a.D, V), (unsigned)a.B), block(32 * warps_for(a.L, kFwdRun));
        return a.values ? launch_programmatic(linear_fwd_kernel<T, V, true>, grid, block, 0, stream, a)
                        : launch_programmatic(linear_fwd_kernel<T, V, false>, grid, block, 0, stream, a);
    });
}

template <typename T> cudaError_t backward_t(const LinearBwdArgs &a, cudaStream_t stream) {
    return for_width(a.f.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        cudaError_t e = cudaSuccess;
        if (a.f.B > 0) {
            const dim3 grid(1, tiles(a.f.D, V), (unsigned)a.f.B), block(32 * warps_for(a.f.L, kBwdRun));
            e = a.f.values ? launch_programmatic(linear_bwd_kernel<T, V, true>, grid, block, 0, stream, a)
                           : launch_programmatic(linear_bwd_kernel<T, V, false>, grid, block, 0, stream, a);
        }
        if (e != cudaSuccess) return e;
        return launch_programmatic(linear_dlam_kernel, dim3((unsigned)((a.f.D + 31) / 32)), dim3(32, 8), 0, stream,
                                   (const float *)a.part, a.f.lam, a.dlam, a.f.B, a.f.D);
    });
}

}  // namespace linear

int64_t linear_bwd_parts(int64_t B) { return B; }

cudaError_t launch_linear(int io, const LinearArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::forward_t<__nv_bfloat16>(a, stream) : linear::forward_t<float>(a, stream);
}

cudaError_t launch_linear_bwd(int io, const LinearBwdArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::backward_t<__nv_bfloat16>(a, stream) : linear::backward_t<float>(a, stream);
}

cudaError_t launch_linear_step(int io, const LinearStepArgs &a, cudaStream_t stream) {
    return linear::for_width(a.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        const dim3 grid((unsigned)((a.B * (a.D / V) + 255) / 256));
        return io == IO_BF16 ? launch_programmatic(linear::linear_step_kernel<__nv_bfloat16, V>, grid, dim3(256), 0, stream, a)
                             : launch_programmatic(linear::linear_step_kernel<float, V>, grid, dim3(256), 0, stream, a);
    });
}

cudaError_t launch_pack8(int io, const Pack8Args &a, cudaStream_t stream) {
    return linear::for_width(a.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        const dim3 grid((unsigned)((a.L + linear::kGroup * linear::kWarps - 1) / (linear::kGroup * linear::kWarps)),
                        linear::tiles(a.D, V), (unsigned)a.B), block(linear::kThreads);
        if (a.out)
            return io == IO_BF16 ? launch_programmatic(linear::unpack8_kernel<__nv_bfloat16, V>, grid, block, 0, stream, a)
                                 : launch_programmatic(linear::unpack8_kernel<float, V>, grid, block, 0, stream, a);
        return io == IO_BF16 ? launch_programmatic(linear::pack8_kernel<__nv_bfloat16, V>, grid, block, 0, stream, a)
                             : launch_programmatic(linear::pack8_kernel<float, V>, grid, block, 0, stream, a);
    });
}

}  // namespace ssd
