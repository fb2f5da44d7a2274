// Block norm: what stands between the output of one block and the input of the
// next, per row, in one pass over the data:
//     u = y silu(z)      n = u rsqrt(mean u^2 + eps) w_post     (no w_post: n = u)
//     r = res + s n      out = r rsqrt(mean r^2 + eps) w_pre
// and its backward. Rows are held in registers in float32 (thread t owns the
// vectors t, t + threads, ... of the row), statistics are float32 sums over a
// fixed tree, and each result is rounded once.
#include "common.cuh"
#include "launch.h"

namespace ssd {
namespace {

constexpr int kMaxWarps = 32;

// V consecutive elements as float32, V * sizeof(T) aligned (at most 16 bytes at once).
template <typename T, int V> __device__ __forceinline__ void ld(float (&f)[V], const T *p) {
    if constexpr (V == 1) {
        f[0] = to_f32(p[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 v = ld4(p + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    }
}
template <typename T, int V> __device__ __forceinline__ void st(T *p, const float (&f)[V]) {
    if constexpr (V == 1) {
        p[0] = from_f32<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < V; k += 4)
            *reinterpret_cast<float4 *>(p + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
    } else {
        T v[V];
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = from_f32<T>(f[k]);
#pragma unroll
        for (int k = 0; k < V; k += 4)
            *reinterpret_cast<uint2 *>(p + k) = *reinterpret_cast<const uint2 *>(v + k);
    }
}

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + __expf(-z)); }

// Sum over the block, the same in every thread; `part` is not used by another
// reduction until a __syncthreads() later.
__device__ __forceinline__ float block_sum(float v, float *part) {
    v = warp_sum(v);
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < nw ? part[lane] : 0.f);
}

template <typename T, typename TR, int V, int RV>
__global__ void __launch_bounds__(1024) block_norm_kernel(BlockNormArgs a) {
    pdl_enter();
    __shared__ float part[2][kMaxWarps];
    const int64_t base = (int64_t)blockIdx.x * a.dim;
    const T *y = (const T *)a.y + base, *z = a.z ? (const T *)a.z + base : nullptr;
    const TR *res = (const TR *)a.res + base;
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    float u[RV][V], r[RV][V], ss = 0.f;
#pragma unroll
    for (int k = 0; k < RV; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv) {
            ld<T, V>(u[k], y + (int64_t)v * V);
            ld<TR, V>(r[k], res + (int64_t)v * V);
            if (z) {
                float zz[V];
                ld<T, V>(zz, z + (int64_t)v * V);
#pragma unroll
                for (int e = 0; e < V; ++e) u[k][e] *= zz[e] * sigmoid_f(zz[e]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(u[k][e], u[k][e], ss);
        }
    }
    float tau = 1.f;
    if (a.post_w) tau = rsqrtf(block_sum(ss, part[0]) * inv + a.eps);
    ss = 0.f;
#pragma unroll
    for (int k = 0; k < RV; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv) {
            float w[V], s[V];
            if (a.post_w) ld<float, V>(w, a.post_w + v * V);
            if (a.scale) ld<float, V>(s, a.scale + v * V);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float n = u[k][e] * tau;
                if (a.post_w) n *= w[e];
                r[k][e] += a.scale ? s[e] * n : n;
                ss = fmaf(r[k][e], r[k][e], ss);
            }
            st<TR, V>((TR *)a.res_out + base + (int64_t)v * V, r[k]);
        }
    }
    const float rho = rsqrtf(block_sum(ss, part[1]) * inv + a.eps);
#pragma unroll
    for (int k = 0; k < RV; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv) {
            float w[V];
            ld<float, V>(w, a.pre_w + v * V);
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] *= r[k][e] * rho;
            st<T, V>((T *)a.out + base + (int64_t)v * V, w);
        }
    }
}

// Backward: r is formed again from the inputs (no saved statistics). Block i
// walks the rows i, i + blocks, ... and keeps its sums of the weights'
// gradients in registers; block_norm_reduce_kernel adds the blocks' sums.
template <typename T, typename TR, int V, int RV>
__global__ void __launch_bounds__(1024) block_norm_bwd_kernel(BlockNormArgs a) {
    pdl_enter();
    __shared__ float part[4][kMaxWarps];
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    float gpre[RV][V] = {}, gpost[RV][V] = {}, gscale[RV][V] = {};
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t base = row * a.dim;
        float u[RV][V], r[RV][V], d[RV][V], ss = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                const int64_t at = base + (int64_t)v * V;
                ld<T, V>(u[k], (const T *)a.y + at);
                ld<TR, V>(r[k], (const TR *)a.res + at);
                ld<T, V>(d[k], (const T *)a.dout + at);
                if (a.z) {
                    float zz[V];
                    ld<T, V>(zz, (const T *)a.z + at);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[k][e] *= zz[e] * sigmoid_f(zz[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(u[k][e], u[k][e], ss);
            }
        }
        float tau = 1.f;
        if (a.post_w) tau = rsqrtf(block_sum(ss, part[0]) * inv + a.eps);
        ss = 0.f;
        float ar = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                float w[V], s[V], p[V];
                if (a.post_w) ld<float, V>(w, a.post_w + v * V);
                if (a.scale) ld<float, V>(s, a.scale + v * V);
                ld<float, V>(p, a.pre_w + v * V);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float n = u[k][e] * tau;
                    if (a.post_w) n *= w[e];
                    r[k][e] += a.scale ? s[e] * n : n;
                    ss = fmaf(r[k][e], r[k][e], ss);
                    ar = fmaf(d[k][e] * p[e], r[k][e], ar);
                }
            }
        }
        const float rho = rsqrtf(block_sum(ss, part[1]) * inv + a.eps);
        const float c = block_sum(ar, part[2]) * inv * rho * rho;
        float bu = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                const int64_t at = base + (int64_t)v * V;
                float w[V], s[V], p[V], dr[V];
                if (a.post_w) ld<float, V>(w, a.post_w + v * V);
                if (a.scale) ld<float, V>(s, a.scale + v * V);
                ld<float, V>(p, a.pre_w + v * V);
                if (a.dres_out) ld<TR, V>(dr, (const TR *)a.dres_out + at);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    gpre[k][e] = fmaf(d[k][e], r[k][e] * rho, gpre[k][e]);
                    const float x = rho * (d[k][e] * p[e] - r[k][e] * c);
                    dr[e] = a.dres_out ? dr[e] + x : x;
                    float n = u[k][e] * tau;
                    if (a.post_w) n *= w[e];
                    gscale[k][e] = fmaf(dr[e], n, gscale[k][e]);
                    const float dn = a.scale ? dr[e] * s[e] : dr[e];
                    gpost[k][e] = fmaf(dn, u[k][e] * tau, gpost[k][e]);
                    d[k][e] = a.post_w ? dn * w[e] : dn;
                    bu = fmaf(d[k][e], u[k][e], bu);
                }
                st<TR, V>((TR *)a.dres + at, dr);
            }
        }
        float m = 0.f;
        if (a.post_w) m = block_sum(bu, part[3]) * inv * tau * tau;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                const int64_t at = base + (int64_t)v * V;
#pragma unroll
                for (int e = 0; e < V; ++e) d[k][e] = tau * (d[k][e] - u[k][e] * m);
                if (a.z) {
                    float zz[V], yy[V];
                    ld<T, V>(zz, (const T *)a.z + at);
                    ld<T, V>(yy, (const T *)a.y + at);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float sg = sigmoid_f(zz[e]), x = d[k][e];
                        d[k][e] = x * zz[e] * sg;
                        zz[e] = x * yy[e] * sg * (1.f + zz[e] * (1.f - sg));
                    }
                    st<T, V>((T *)a.dz + at, zz);
                }
                st<T, V>((T *)a.dy + at, d[k]);
            }
        }
        __syncthreads();  // part is free again
    }
    float *o = a.part + (int64_t)blockIdx.x * 3 * a.dim;
#pragma unroll
    for (int k = 0; k < RV; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv) {
            st<float, V>(o + (int64_t)v * V, gpre[k]);
            st<float, V>(o + a.dim + (int64_t)v * V, gpost[k]);
            st<float, V>(o + 2 * a.dim + (int64_t)v * V, gscale[k]);
        }
    }
}

// One warp per 32 columns of one of the three sums; eight warps split the blocks' parts.
__global__ void __launch_bounds__(256) block_norm_reduce_kernel(BlockNormArgs a, int parts) {
    pdl_enter();
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float *dst = which == 0 ? a.dpre_w : which == 1 ? a.dpost_w : a.dscale;
    if (!dst) return;
    float v = 0.f;
    if (col < a.dim)
        for (int i = warp; i < parts; i += 8) v += a.part[((int64_t)i * 3 + which) * a.dim + col];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && col < a.dim) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += s[w][lane];
        dst[col] = v;
    }
}

template <int V> using Int = std::integral_constant<int, V>;

// Vectors of four elements where the row length allows them (the pointers are
// 16-byte aligned), else single elements; vectors per thread so that a block
// of at most 1024 threads holds a row.
template <typename F> cudaError_t for_row(int64_t dim, F f) {
    auto pick = [&](auto v) {
        const int64_t nv = dim / v.value;
        auto threads = [&](int rv) { return (int)(((nv + rv - 1) / rv + 31) / 32 * 32); };
        if (nv <= 1024) return f(v, Int<1>{}, threads(1));
        if (nv <= 2048) return f(v, Int<2>{}, threads(2));
        if (decltype(v)::value == 4 || nv <= 4096) return f(v, Int<4>{}, threads(4));
        if constexpr (decltype(v)::value == 1) return f(v, Int<16>{}, threads(16));
    };
    return dim % 4 == 0 ? pick(Int<4>{}) : pick(Int<1>{});
}

template <typename F> cudaError_t for_types(int io, int res_io, F f) {
    if (io == IO_BF16) return res_io == IO_BF16 ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, 0.f);
    return f(0.f, 0.f);
}

}  // namespace

cudaError_t launch_block_norm(int io, int res_io, const BlockNormArgs &a, cudaStream_t stream) {
    return for_types(io, res_io, [&](auto t, auto tr) {
        return for_row(a.dim, [&](auto v, auto rv, int threads) {
            return launch_programmatic(block_norm_kernel<decltype(t), decltype(tr), decltype(v)::value, decltype(rv)::value>,
                                       dim3((unsigned)a.rows), dim3(threads), 0, stream, a);
        });
    });
}

int block_norm_bwd_parts(int64_t rows, int64_t) { return (int)imin<int64_t>(rows, 2 * (int64_t)sm_count(152)); }

cudaError_t launch_block_norm_bwd(int io, int res_io, const BlockNormArgs &a, cudaStream_t stream) {
    const int parts = block_norm_bwd_parts(a.rows, a.dim);
    cudaError_t e = a.rows == 0 ? cudaSuccess : for_types(io, res_io, [&](auto t, auto tr) {
        return for_row(a.dim, [&](auto v, auto rv, int threads) {
            return launch_programmatic(
                block_norm_bwd_kernel<decltype(t), decltype(tr), decltype(v)::value, decltype(rv)::value>,
                dim3((unsigned)parts), dim3(threads), 0, stream, a);
        });
    });
    if (e != cudaSuccess) return e;
    return launch_programmatic(block_norm_reduce_kernel, dim3((unsigned)((a.dim + 31) / 32), 3), dim3(256), 0, stream, a,
                               parts);
}

}  // namespace ssd
