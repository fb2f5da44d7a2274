// Block norm: what stands between the output of one block and the input of the
// next, per row, in one pass over the data:
//     u = y silu(z)      n = u rsqrt(mean u^2 + eps) w_post     (no w_post: n = u)
//     r = res + s n      out = r rsqrt(mean r^2 + eps) w_pre
// and its backward. Thread t owns the vectors t, t + threads, ... of a row, in
// registers in float32; statistics are float32 sums over a fixed tree, and each
// result is rounded once.
//
// Bound by HBM. A block walks rows (row i, i + blocks, ...): the next row is on its
// way to shared memory (cp.async, each thread copies and reads its own vectors, so
// nothing but the sums crosses threads) while this one is reduced and written.
// 16384 x 2560 bf16: 70 us, 6.0 TB/s; rows that are no multiple of four elements go
// one by one (4096 x 1537 bf16 from cold caches: 83 us, 0.8 TB/s; 38 without a gate).
#include "common.cuh"
#include "launch.h"

namespace ssd {
namespace {

constexpr int kMaxWarps = 32;

// V elements of type T as float32.
template <typename T, int V> __device__ __forceinline__ void ld(float (&f)[V], const T *p) {
    if constexpr (V == 1) {
        f[0] = to_f32(p[0]);
    } else if constexpr (V == 8 && sizeof(T) == 2) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) f[2 * k] = __uint_as_float(w[k] << 16), f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
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
        uint32_t v[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            v[k] = *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (V == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
    }
}

// 1 / (1 + exp(-z)), the quotient within 2 units in the last place. For float32 gates with expf (1 unit): silu(z) within
// 4.5 units for any z. For bf16 gates with __expf, whose error grows as 2 + 1.17 |z| units: at z = -10 silu is off by
// 5e-7 of itself, at -80 by 4e-6, all of it where silu is small (3e-7 of max(1, |z|) at most), far below the 8 bits of
// z; expf there costs 16384 x 2560 70.2 -> 75.0 us and the backward of 8192 x 2560 82.2 -> 88.4 us.
template <typename T> __device__ __forceinline__ float sigmoid_f(float z) {
    return __fdividef(1.f, 1.f + (sizeof(T) == 4 ? expf(-z) : __expf(-z)));
}

// V weights, or ones where there are none.
template <int V> __device__ __forceinline__ void weights(float (&w)[V], const float *p, int v) {
    if (p) {
        ld<float, V>(w, p + v * V);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = 1.f;
    }
}

// Sum over the block, and of two values at once, the same in every thread. `part`
// is not written again before two more __syncthreads().
__device__ __forceinline__ float block_sum(float a, float *part) {
    a = warp_sum(a);
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    return warp_sum(lane < nw ? part[lane] : 0.f);
}
__device__ __forceinline__ float2 block_sum(float a, float b, float *part) {
    a = warp_sum(a);
    b = warp_sum(b);
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) part[threadIdx.x >> 5] = a, part[kMaxWarps + (threadIdx.x >> 5)] = b;
    __syncthreads();
    a = lane < nw ? part[lane] : 0.f;
    b = lane < nw ? part[kMaxWarps + lane] : 0.f;
    return make_float2(warp_sum(a), warp_sum(b));
}

// A thread's vectors of one array of a row, copied ahead into shared memory. Vectors
// of two bytes (V = 1, bf16) cannot be and are read where they lie.
template <typename T, int V, int RV, bool STAGED = true> struct Ahead {
    static constexpr int kBytes = V * sizeof(T);
    static constexpr bool kCopy = STAGED && kBytes >= 4;
    __host__ __device__ static constexpr size_t bytes(int threads) { return kCopy ? (size_t)RV * threads * kBytes : 0; }
    __device__ static __forceinline__ void fetch(uint8_t *buf, const T *row, int nv) {
        if constexpr (kCopy) {
#pragma unroll
            for (int k = 0; k < RV; ++k) {
                const int v = threadIdx.x + k * blockDim.x;
                if (v >= nv) continue;
                const uint32_t d = (uint32_t)__cvta_generic_to_shared(buf + (size_t)v * kBytes);
                const char *s = reinterpret_cast<const char *>(row + (int64_t)v * V);
                if constexpr (kBytes >= 16) {
#pragma unroll
                    for (int e = 0; e < kBytes; e += 16)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + e), "l"(s + e) : "memory");
                } else if constexpr (kBytes == 8) {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(s) : "memory");
                } else {
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(s) : "memory");
                }
            }
        }
    }
    __device__ static __forceinline__ void get(float (&f)[V], const uint8_t *buf, const T *row, int v) {
        if constexpr (kCopy)
            ld<T, V>(f, reinterpret_cast<const T *>(buf) + (size_t)v * V);
        else
            ld<T, V>(f, row + (int64_t)v * V);
    }
};
__device__ __forceinline__ void ahead_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void ahead_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <typename T, typename TR, int V, int RV>
__global__ void __launch_bounds__(256) block_norm_kernel(BlockNormArgs a) {
    pdl_enter();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][2][kMaxWarps];
    using A = Ahead<T, V, RV>;
    using AR = Ahead<TR, V, RV>;
    uint8_t *by = smem, *bz = by + A::bytes(blockDim.x), *br = bz + A::bytes(blockDim.x);
    const T *y = (const T *)a.y, *z = (const T *)a.z;
    const TR *res = (const TR *)a.res;
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    auto fetch = [&](int64_t row) {
        A::fetch(by, y + row * a.dim, nv);
        if (z) A::fetch(bz, z + row * a.dim, nv);
        AR::fetch(br, res + row * a.dim, nv);
        ahead_commit();
    };
    fetch(blockIdx.x);
    int ph = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ph ^= 1) {
        const int64_t base = row * a.dim;
        float u[RV][V], r[RV][V], ss = 0.f;
        ahead_wait<0>();
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                A::get(u[k], by, y + base, v);
                AR::get(r[k], br, res + base, v);
                if (z) {
                    float zz[V];
                    A::get(zz, bz, z + base, v);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[k][e] *= zz[e] * sigmoid_f<T>(zz[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(u[k][e], u[k][e], ss);
            }
        }
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
        float tau = 1.f;
        if (a.post_w) tau = rsqrtf(block_sum(ss, part[ph][0]) * inv + a.eps);
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                float w[V], s[V];
                weights(w, a.post_w, v);
                weights(s, a.scale, v);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    r[k][e] = fmaf(s[e], u[k][e] * tau * w[e], r[k][e]);
                    ss = fmaf(r[k][e], r[k][e], ss);
                }
                st<TR, V>((TR *)a.res_out + base + (int64_t)v * V, r[k]);
            }
        }
        const float rho = rsqrtf(block_sum(ss, part[ph][1]) * inv + a.eps);
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
}

// Backward: r is formed again from the inputs (no saved statistics), which stay in
// shared memory while their row is worked on (with two stages the next row's are on
// their way meanwhile); where a row is too long for that they are read from
// memory each time (STAGED false). A block keeps its sums of the weights' gradients
// in registers; block_norm_reduce_kernel adds the blocks' sums.
// MOST threads at most: 320 (two blocks per SM with one vector per thread: 16384 x
// 2560 bf16 took 187 us, 267 us where 122 registers leave one block), 640 where that
// leaves a thread one vector of eight (8192 x 5120 bf16: 148 us, 203 us with 320 threads and two
// vectors), else 512. 320 and 640 threads are rows of 2560 and 5120; the limits were measured there, and shorter rows take
// the same forms with fewer threads (float32 residual, gate, cold: 16384 x 1024 65 us, 8192 x 2048 72, 4096 x 5120 91).
// 8192 x 2560 bf16 with a float32 residual: 84 us, 5.5 TB/s (110 us with the weights
// read anew for each row and three sums for the three weights).
template <typename T, typename TR, int V, int RV, bool STAGED, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 320 && RV == 1 ? 2 : 1) block_norm_bwd_kernel(BlockNormArgs a, int stages) {
    pdl_enter();
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[2][4][kMaxWarps];
    using A = Ahead<T, V, RV, STAGED>;
    using AR = Ahead<TR, V, RV, STAGED>;
    const size_t na = A::bytes(blockDim.x), nr = AR::bytes(blockDim.x), stage = 3 * na + 2 * nr;
    const T *y = (const T *)a.y, *z = (const T *)a.z, *dout = (const T *)a.dout;
    const TR *res = (const TR *)a.res, *dres_out = (const TR *)a.dres_out;
    const int nv = (int)(a.dim / V);
    const float inv = 1.f / (float)a.dim;
    auto fetch = [&](int64_t row, uint8_t *buf) {
        const int64_t at = row * a.dim;
        A::fetch(buf, y + at, nv);
        if (z) A::fetch(buf + na, z + at, nv);
        A::fetch(buf + 2 * na, dout + at, nv);
        AR::fetch(buf + 3 * na, res + at, nv);
        if (dres_out) AR::fetch(buf + 3 * na + nr, dres_out + at, nv);
        ahead_commit();
    };
    // sums of dout r rho and, with o = dL/dr, of o u tau: that sum times scale is post_w's gradient, times post_w scale's
    float gpre[RV][V] = {}, gsum[RV][V] = {};
    // pre_w, and scale post_w: kept for all rows where there are registers for it
    constexpr bool KEEP = RV * V <= 8;
    float wp[KEEP ? RV : 1][V], ws[KEEP ? RV : 1][V];
    auto read_weights = [&](float (&p)[V], float (&sw)[V], int v) {
        float w[V];
        ld<float, V>(p, a.pre_w + v * V);
        weights(sw, a.scale, v);
        weights(w, a.post_w, v);
#pragma unroll
        for (int e = 0; e < V; ++e) sw[e] *= w[e];
    };
    if constexpr (KEEP)
#pragma unroll
        for (int k = 0; k < RV; ++k)
            if ((int)(threadIdx.x + k * blockDim.x) < nv) read_weights(wp[k], ws[k], threadIdx.x + k * blockDim.x);
    fetch(blockIdx.x, smem);
    int ph = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ph ^= 1) {
        const int64_t base = row * a.dim;
        uint8_t *buf = smem + (stages == 2 && ph ? stage : 0);
        if (stages == 2 && row + gridDim.x < a.rows) {
            fetch(row + gridDim.x, smem + (ph ? 0 : stage));
            ahead_wait<1>();
        } else {
            ahead_wait<0>();
        }
        float u[RV][V], r[RV][V], d[RV][V], ss = 0.f, ar = 0.f, bu = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                A::get(u[k], buf, y + base, v);
                if (z) {
                    float zv[V];
                    A::get(zv, buf + na, z + base, v);
#pragma unroll
                    for (int e = 0; e < V; ++e) u[k][e] *= zv[e] * sigmoid_f<T>(zv[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) ss = fmaf(u[k][e], u[k][e], ss);
            }
        }
        float tau = 1.f;
        if (a.post_w) tau = rsqrtf(block_sum(ss, part[ph][0]) * inv + a.eps);
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                float (&p)[V] = wp[KEEP ? k : 0], (&sw)[V] = ws[KEEP ? k : 0];
                if constexpr (!KEEP) read_weights(p, sw, v);
                AR::get(r[k], buf + 3 * na, res + base, v);
                A::get(d[k], buf + 2 * na, dout + base, v);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    u[k][e] *= tau;
                    r[k][e] = fmaf(sw[e], u[k][e], r[k][e]);
                    ss = fmaf(r[k][e], r[k][e], ss);
                    ar = fmaf(d[k][e] * p[e], r[k][e], ar);
                }
            }
        }
        const float2 sums = block_sum(ss, ar, part[ph][1]);
        const float rho = rsqrtf(sums.x * inv + a.eps), c = sums.y * inv * rho * rho;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                float (&p)[V] = wp[KEEP ? k : 0], (&sw)[V] = ws[KEEP ? k : 0], o[V];
                if constexpr (!KEEP) read_weights(p, sw, v);
                if (dres_out) {
                    AR::get(o, buf + 3 * na + nr, dres_out + base, v);
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {  // u holds u tau
                    gpre[k][e] = fmaf(d[k][e], r[k][e] * rho, gpre[k][e]);
                    o[e] = fmaf(rho, d[k][e] * p[e] - r[k][e] * c, o[e]);
                    gsum[k][e] = fmaf(o[e], u[k][e], gsum[k][e]);
                    d[k][e] = o[e] * sw[e];
                    bu = fmaf(d[k][e], u[k][e], bu);
                }
                st<TR, V>((TR *)a.dres + base + (int64_t)v * V, o);
            }
        }
        float m = 0.f;  // mean of (cotangent of the normed u) . (u tau)
        if (a.post_w) m = block_sum(bu, part[ph][3]) * inv;
#pragma unroll
        for (int k = 0; k < RV; ++k) {
            const int v = threadIdx.x + k * blockDim.x;
            if (v < nv) {
                const int64_t at = base + (int64_t)v * V;
#pragma unroll
                for (int e = 0; e < V; ++e) d[k][e] = tau * fmaf(-u[k][e], m, d[k][e]);
                if (z) {
                    float yv[V], zv[V];
                    A::get(yv, buf, y + base, v);
                    A::get(zv, buf + na, z + base, v);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float sg = sigmoid_f<T>(zv[e]), t = zv[e] * sg;
                        yv[e] *= d[k][e] * fmaf(t, 1.f - sg, sg);
                        d[k][e] *= t;
                    }
                    st<T, V>((T *)a.dz + at, yv);
                }
                st<T, V>((T *)a.dy + at, d[k]);
            }
        }
        if (stages == 1 && row + gridDim.x < a.rows) fetch(row + gridDim.x, smem);
    }
    float *out = a.part + (int64_t)blockIdx.x * 2 * a.dim;
#pragma unroll
    for (int k = 0; k < RV; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v < nv) {
            st<float, V>(out + (int64_t)v * V, gpre[k]);
            st<float, V>(out + a.dim + (int64_t)v * V, gsum[k]);
        }
    }
}

// 32 columns of one of the two sums; sixteen warps split the blocks' parts, few loads after one another.
constexpr int kReduceWarps = 16;
__global__ void __launch_bounds__(32 * kReduceWarps) block_norm_reduce_kernel(BlockNormArgs a, int parts) {
    pdl_enter();
    __shared__ float s[kReduceWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (col < a.dim) {
#pragma unroll 10
        for (int i = warp; i < parts; i += kReduceWarps) v += a.part[((int64_t)i * 2 + which) * a.dim + col];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && col < a.dim) {
#pragma unroll
        for (int w = 1; w < kReduceWarps; ++w) v += s[w][lane];
        if (which == 0) {
            a.dpre_w[col] = v;
        } else {
            if (a.dpost_w) a.dpost_w[col] = a.scale ? v * a.scale[col] : v;
            if (a.dscale) a.dscale[col] = a.post_w ? v * a.post_w[col] : v;
        }
    }
}

template <int V> using Int = std::integral_constant<int, V>;

// Vectors of eight or four elements where the row length allows them (the
// pointers are 16-byte aligned), else single ones; RV of them per thread, the least
// of the given numbers with which a block of at most `most` threads holds a row.
template <typename F, int... RVs> cudaError_t with_rv(int64_t nv, int most, F f, std::integer_sequence<int, RVs...>) {
    cudaError_t e = cudaErrorInvalidValue;
    bool done = false;
    ((done || (nv + RVs - 1) / RVs > most ? void() : (done = true, e = f(Int<RVs>{}, (int)(((nv + RVs - 1) / RVs + 31) / 32 * 32)), void())),
     ...);
    return e;
}
// `RV4` lists the numbers for vectors of four: 16 is for the forward's 256 threads and rows above 8192.
template <typename RV4, typename F> cudaError_t for_row(int64_t dim, int most, F f) {
    if (dim % 8 == 0)
        return with_rv(dim / 8, most, [&](auto rv, int t) { return f(Int<8>{}, rv, t); }, std::integer_sequence<int, 1, 2, 4, 8>{});
    if (dim % 4 == 0)
        return with_rv(dim / 4, most, [&](auto rv, int t) { return f(Int<4>{}, rv, t); }, RV4{});
    return with_rv(dim, most, [&](auto rv, int t) { return f(Int<1>{}, rv, t); }, std::integer_sequence<int, 1, 4, 8, 32, 64>{});
}

template <typename F> cudaError_t for_types(int io, int res_io, F f) {
    if (io == IO_BF16) return res_io == IO_BF16 ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, 0.f);
    return f(0.f, 0.f);
}

// Blocks for `rows` rows: all that are resident at once, and no more. `most` is the largest smem of any call of KERN.
template <auto KERN> cudaError_t resident(int threads, size_t smem, size_t most, int64_t rows, int64_t *grid) {
    if (most > 40 * 1024) {  // with the static part past the 48 KB that need no asking
        cudaError_t e = allow_shared<KERN>(most);
        if (e != cudaSuccess) return e;
    }
    *grid = imin<int64_t>(rows, sm_count(1));
    if (rows > *grid) {
        int per_sm = 0;
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERN, threads, smem);
        if (e != cudaSuccess) return e;
        *grid = imin<int64_t>(rows, (int64_t)sm_count(1) * imax(1, per_sm));
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_block_norm(int io, int res_io, const BlockNormArgs &a, cudaStream_t stream) {
    return for_types(io, res_io, [&](auto t, auto tr) {
        constexpr int kMost = 256;
        return for_row<std::integer_sequence<int, 1, 2, 4, 8, 16>>(a.dim, kMost, [&](auto v, auto rv, int threads) {
            using T = decltype(t);
            using TR = decltype(tr);
            constexpr int V = decltype(v)::value, RV = decltype(rv)::value;
            constexpr auto kern = block_norm_kernel<T, TR, V, RV>;
            auto smem_of = [](int n) { return 2 * Ahead<T, V, RV>::bytes(n) + Ahead<TR, V, RV>::bytes(n); };
            const size_t smem = smem_of(threads);
            int64_t grid = 0;
            cudaError_t e = resident<kern>(threads, smem, smem_of(kMost), a.rows, &grid);
            return e != cudaSuccess ? e : launch_programmatic(kern, dim3((unsigned)grid), dim3(threads), smem, stream, a);
        });
    });
}

// The workspace holds the parts of this many blocks: an SM's registers hold about 640 threads of 8 elements
// (16384 x 768 bf16: 53 us, 57 us with 4 blocks per SM).
int block_norm_bwd_parts(int64_t rows, int64_t dim) {
    return (int)imin<int64_t>(rows, sm_count(152) * imax<int64_t>(4, imin<int64_t>(16, 5120 / imax<int64_t>(1, dim) + 1)));
}

cudaError_t launch_block_norm_bwd(int io, int res_io, const BlockNormArgs &a, cudaStream_t stream) {
    int64_t parts = 0;
    if (a.rows > 0) {
        cudaError_t e = for_types(io, res_io, [&](auto t, auto tr) {
            const int most = a.dim % 8 == 0 && a.dim <= 8 * 640 ? 640 : 512;
            return for_row<std::integer_sequence<int, 1, 2, 4, 8>>(a.dim, most, [&](auto v, auto rv, int threads) {
                using T = decltype(t);
                using TR = decltype(tr);
                constexpr int V = decltype(v)::value, RV = decltype(rv)::value;
                constexpr size_t kMost = 220 * 1024;
                const size_t stage = 3 * Ahead<T, V, RV>::bytes(threads) + 2 * Ahead<TR, V, RV>::bytes(threads);
                auto go = [&](auto staged, auto most, int stages) {
                    constexpr auto kern = block_norm_bwd_kernel<T, TR, V, RV, decltype(staged)::value, decltype(most)::value>;
                    const size_t smem = stages * stage;
                    cudaError_t r = resident<kern>(threads, smem, decltype(staged)::value ? kMost : 0, a.rows, &parts);
                    if (r != cudaSuccess) return r;
                    parts = imin<int64_t>(parts, block_norm_bwd_parts(a.rows, a.dim));
                    return launch_programmatic(kern, dim3((unsigned)parts), dim3(threads), smem, stream, a, stages);
                };
                const int stages = 2 * stage <= kMost ? 2 : 1;
                if (stage > kMost) {
                    if constexpr (RV * V >= 16) return go(std::false_type{}, Int<512>{}, 0);
                    return cudaErrorInvalidValue;
                }
                if constexpr (RV == 1 && V == 8)
                    if (threads > 512) return go(std::true_type{}, Int<640>{}, stages);
                if constexpr (RV <= 2)
                    if (threads <= 320) return go(std::true_type{}, Int<320>{}, stages);
                return go(std::true_type{}, Int<512>{}, stages);
            });
        });
        if (e != cudaSuccess) return e;
    }
    return launch_programmatic(block_norm_reduce_kernel, dim3((unsigned)((a.dim + 31) / 32), 2), dim3(32 * kReduceWarps), 0,
                               stream, a, (int)parts);
}

}  // namespace ssd
