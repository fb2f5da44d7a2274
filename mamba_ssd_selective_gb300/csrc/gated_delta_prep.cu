// T and M T of every chunk of the gated delta rule (gated_delta_tc.cuh), and its
// decays: one block of four warps per (b, chunk, head), bf16 inputs, N <= 128.
//
// Everything is blocks of 16 x 16. Warp w forms row w of the blocks of K K^T and
// Q K^T (mma.sync, K and Q exact, float32 sums) and scales them to A and M in
// registers. The diagonal blocks of I + A are inverted by substitution in
// float32, one warp each; the rest of T follows from
// [[Ta, 0], [-Tb A Ta, Tb]], first for the blocks of 32, then of 64, and M T row
// by row. Operands that were rounded go in as pairs hi + lo of bf16 (2^-17 is
// lost); the fragments of one product are the operands of the next, which
// the tensor-memory path cannot give at this size.
//
// The sums c are taken in float64 and kept as a float32 and its remainder, so
// that a steep decay does not blur the differences of the tokens after it.
//
// Bound by instruction issue (about 5 thousand warp instructions a block); several
// blocks per SM cover the latencies of one.
#include "gated_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kThreads = 128;
// shared memory (bytes): K and Q, 64 rows in panels of 64 columns (128-byte swizzle), later the four tiles; then blocks
// of A of 512 bytes (hi, then lo), the diagonal ones in float32; then the sums' factors
constexpr uint32_t kOffBlk = 32768, kOffSc = kOffBlk + 12 * 512 + 4 * 1024;
enum { S_HI, S_ROW, S_INV, S_N };  // c (base 2) rounded, 2^remainder, beta 2^-remainder
constexpr uint32_t kSmem = kOffSc + S_N * kC * 4;

__device__ __forceinline__ int a_blk(int i, int j) { return (i * (i - 1)) / 2 + j; }
// 16-byte half of a row of a 512-byte block: 32 bytes per row, the halves of rows 4-7 and 12-15 swapped
__device__ __forceinline__ uint32_t in_blk(int row, int half) { return (uint32_t)(row * 32 + ((half ^ ((row >> 2) & 1)) << 4)); }

// 16 bytes from global to shared memory without waiting; zeros where `on` is false
__device__ __forceinline__ void copy16(void *dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}

__global__ void __launch_bounds__(kThreads, 5) delta_prep_kernel(PrepArgs p) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sK = smem, *sQ = smem + 16384, *thi = smem, *mhi = smem + kTile, *tlo = smem + 2 * kTile, *mlo = smem + 3 * kTile;
    uint8_t *blk = smem + kOffBlk;
    constexpr int kLo = 6;
    float *diag = reinterpret_cast<float *>(blk + 12 * 512);
    float *sc = reinterpret_cast<float *>(smem + kOffSc);
    const DeltaArgs &a = p.a;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t2 = 2 * (lane & 3);
    const int H = (int)a.H, N = (int)a.N;
    const int h = (int)(blockIdx.x % H);
    const int64_t bc = blockIdx.x / H, c = bc % p.nc, b = bc / p.nc;
    const int grp = h / (int)(a.H / a.G);
    const int64_t len = seq_len(a.seqlens, b, a.L), t0 = c * kC;
    if (c == 0) {
        const int pb = (int)row_blocks(a.P);
        for (int x = tid; x < 2 * pb; x += kThreads) p.flags[((x / pb) * a.B * H + b * H + h) * pb + x % pb] = 0;
    }
    if (t0 >= len) return;
    const int64_t item = (b * H + h) * p.nc + c;
    const int NK = N <= 64 ? 64 : 128;

    // K and Q, zeros past the length and past N (N is a multiple of 8), all copies in flight at once
    for (int x = tid; x < kC * (NK / 8); x += kThreads) {
        const int row = x / (NK / 8), pc = x - row * (NK / 8);
        const bool on = t0 + row < len && 8 * pc < N;
        const int64_t at = on ? ((b * a.L + t0 + row) * a.G + grp) * N + 8 * pc : 0;
        const uint32_t o = (pc >> 3) * 8192 + piece(row, pc & 7);
        copy16(sK + o, (const __nv_bfloat16 *)a.k + at, on);
        copy16(sQ + o, (const __nv_bfloat16 *)a.q + at, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (w == 0) {
        float gv[2], bv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t t = t0 + 2 * lane + e, at = (b * a.L + t) * H + h;
            gv[e] = t < len ? to_f32(((const __nv_bfloat16 *)a.g)[at]) : 0.f;
            bv[e] = t < len ? to_f32(((const __nv_bfloat16 *)a.beta)[at]) : 0.f;
            // exp is 0 in float32 long before -256: the sums stay finite, the decays the same
            if (gv[e] < -256.f) gv[e] = -256.f;
        }
        double sum = (double)gv[0] + (double)gv[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double u = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += u;
        }
        const double end = __shfl_sync(0xffffffffu, sum, 31) * (double)kLog2e;
        float *o = p.scal + item * kScal + 2 * lane;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const double c2 = (e ? sum : sum - (double)gv[1]) * (double)kLog2e;  // base-2 units
            const float hi = (float)c2, lo = (float)(c2 - (double)hi), eg = exp2f((float)c2);
            const float row = exp2f(lo), inv = bv[e] * exp2f(-lo);
            sc[S_HI * kC + 2 * lane + e] = hi;
            sc[S_ROW * kC + 2 * lane + e] = row;
            sc[S_INV * kC + 2 * lane + e] = inv;
            o[SC_EG * kC + e] = eg;
            o[SC_NEG * kC + e] = -eg;
            o[SC_BETA * kC + e] = bv[e];
            o[SC_BTAIL * kC + e] = bv[e] * exp2f((float)(end - c2));
            o[kScalDecay + e] = hi;
            o[kScalDecay + kC + e] = row;
            o[kScalDecay + 2 * kC + e] = inv;
        }
        if (lane == 0) p.scal[item * kScal + kScalEnd] = exp2f((float)end);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // row w of the blocks of K K^T and Q K^T
    float ak[4][8] = {}, aq[4][8] = {};
    const uint32_t arow = piece(16 * w + (lane & 15), 0), axor = (lane & 7) << 4, ah = (lane >> 4) << 4;
    // for the other operand: rows (lane & 7) + 8 (lane >> 4), piece (lane >> 3) & 1
    const uint32_t brow = piece((lane & 7) + ((lane >> 4) << 3), 0), bh = ((lane >> 3) & 1) << 4;
    const uint32_t k0 = tc::smem_u32(sK), q0 = tc::smem_u32(sQ);
#pragma unroll 1
    for (int ks = 0; ks < NK / 16; ++ks) {
        const uint32_t pan = (ks >> 2) * 8192, col = (ks & 3) << 5;
        // a row's pieces are permuted by row & 7 = lane & 7; piece() above already holds that of piece 0
        uint32_t fk[4], fq[4], fb[4];
        tc::ldm_x4(fk, k0 + pan + ((arow ^ axor) + ((col + ah) ^ axor)));
        tc::ldm_x4(fq, q0 + pan + ((arow ^ axor) + ((col + ah) ^ axor)));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j <= w) {
                tc::ldm_x4(fb, k0 + pan + j * 2048 + ((brow ^ axor) + ((col + bh) ^ axor)));
                tc::mma_block(ak[j], fk, fb);
                tc::mma_block(aq[j], fq, fb);
            }
    }
    // A to shared memory, M to fragments
    uint32_t mh[4][4], ml[4][4];
    const int r0 = 16 * w + g;
    const float hi0 = sc[S_HI * kC + r0], hi1 = sc[S_HI * kC + r0 + 8];
    const float rf0 = sc[S_ROW * kC + r0], rf1 = sc[S_ROW * kC + r0 + 8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j <= w) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int cl = 16 * j + 8 * n + t2;
                const float2 hc = *reinterpret_cast<const float2 *>(sc + S_HI * kC + cl);
                const float2 fc = *reinterpret_cast<const float2 *>(sc + S_INV * kC + cl);
                float d[4] = {rf0 * (tc::ex2(hi0 - hc.x) * fc.x), rf0 * (tc::ex2(hi0 - hc.y) * fc.y),
                              rf1 * (tc::ex2(hi1 - hc.x) * fc.x), rf1 * (tc::ex2(hi1 - hc.y) * fc.y)};
                float av[4], mv[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = r0 + 8 * (e >> 1), col = cl + (e & 1);
                    if (col > row) d[e] = 0.f;
                    av[e] = col < row ? ak[j][4 * n + e] * d[e] : 0.f;
                    mv[e] = col <= row ? aq[j][4 * n + e] * d[e] * a.scale : 0.f;
                }
                split2(mv[0], mv[1], mh[j][2 * n], ml[j][2 * n]);
                split2(mv[2], mv[3], mh[j][2 * n + 1], ml[j][2 * n + 1]);
                if (j == w) {
                    float *o = diag + 256 * w + g * 16 + 8 * n + t2;
                    *reinterpret_cast<float2 *>(o) = make_float2(av[0], av[1]);
                    *reinterpret_cast<float2 *>(o + 128) = make_float2(av[2], av[3]);
                } else {
                    uint32_t hi, lo;
                    uint8_t *o = blk + a_blk(w, j) * 512 + t2 * 2;
                    split2(av[0], av[1], hi, lo);
                    *reinterpret_cast<uint32_t *>(o + in_blk(g, n)) = hi;
                    *reinterpret_cast<uint32_t *>(o + kLo * 512 + in_blk(g, n)) = lo;
                    split2(av[2], av[3], hi, lo);
                    *reinterpret_cast<uint32_t *>(o + in_blk(g + 8, n)) = hi;
                    *reinterpret_cast<uint32_t *>(o + kLo * 512 + in_blk(g + 8, n)) = lo;
                }
            }
        }
    __syncthreads();
    // the tiles take the place of K and Q; zeros above the diagonal
    for (int x = tid; x < 32768 / 16; x += kThreads) reinterpret_cast<uint4 *>(smem)[x] = make_uint4(0, 0, 0, 0);
    // column `lane & 15` of the inverse of diagonal block w, by substitution
    float x[16];
    {
        const float4 *d = reinterpret_cast<const float4 *>(diag + 256 * w);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float acc = i == (lane & 15) ? 1.f : 0.f, ac2 = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * k < i) {
                    const float4 v = d[4 * i + k];
                    acc = fmaf(-v.x, x[4 * k], acc);
                    if (4 * k + 1 < i) ac2 = fmaf(-v.y, x[4 * k + 1], ac2);
                    if (4 * k + 2 < i) acc = fmaf(-v.z, x[4 * k + 2], acc);
                    if (4 * k + 3 < i) ac2 = fmaf(-v.w, x[4 * k + 3], ac2);
                }
            x[i] = acc + ac2;
        }
    }
    __syncthreads();
    {  // both halves of the warp hold the columns: one writes hi, the other lo
        uint8_t *d = (lane < 16 ? thi : tlo) + 16 * w * 128 + (lane & 7) * 2;
        const uint32_t pc = (uint32_t)(2 * w + ((lane >> 3) & 1)) << 4;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float hi = __bfloat162float(__float2bfloat16_rn(x[i]));
            *reinterpret_cast<__nv_bfloat16 *>(d + i * 128 + (pc ^ ((i & 7) << 4))) =
                __float2bfloat16_rn(lane < 16 ? x[i] : x[i] - hi);
        }
    }
    __syncthreads();
    // this lane's row address of a block for ldmatrix: of A, of a tile
    const uint32_t blk_lane = tc::smem_u32(blk) + in_blk(lane & 15, lane >> 4);
    auto tile_addr = [&](const uint8_t *tile, int r, int k) {
        return tc::smem_u32(tile) + piece(16 * r + (lane & 15), 2 * k + (lane >> 4));
    };
    // stores an accumulator block as bf16 in a tile
    auto put_block = [&](const uint32_t (&f)[4], uint8_t *tile, int r, int k) {
        uint8_t *d = tile + (16 * r + g) * 128 + (lane & 3) * 4;
        const int p0 = ((2 * k) ^ (g & 7)) << 4, p1 = ((2 * k + 1) ^ (g & 7)) << 4;
        *reinterpret_cast<uint32_t *>(d + p0) = f[0];
        *reinterpret_cast<uint32_t *>(d + 1024 + p0) = f[1];
        *reinterpret_cast<uint32_t *>(d + p1) = f[2];
        *reinterpret_cast<uint32_t *>(d + 1024 + p1) = f[3];
    };
    // Off the diagonal, T_ij = -sum_k (sum_m T_im A_mk) T_kj: first within the blocks of 32 (warps 1 and 3: i = w,
    // j = w - 1, one k and m each), then the block of 32 below them (i = 2, 3, j = 0, 1, m from 2 to i, k from j to 1)
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
        const int i = level ? 2 + (w >> 1) : w, j = level ? w & 1 : w - 1;
        const int m0 = level ? 2 : i, k1 = level ? 1 : j;
        if (level || (w & 1)) {
            float y[8] = {};
#pragma unroll 1
            for (int k = j; k <= k1; ++k) {
                float acc[8] = {};
                uint32_t xh[4], xl[4], yh[4], yl[4];
#pragma unroll 1
                for (int mm = m0; mm <= i; ++mm) {
                    tc::ldm_x4(xh, tile_addr(thi, i, mm));
                    tc::ldm_x4(xl, tile_addr(tlo, i, mm));
                    tc::ldm_x4_trans(yh, blk_lane + a_blk(mm, k) * 512);
                    tc::ldm_x4_trans(yl, blk_lane + (kLo + a_blk(mm, k)) * 512);
                    tc::mma_block(acc, xh, yh);
                    tc::mma_block(acc, xh, yl);
                    tc::mma_block(acc, xl, yh);
                }
                tc::ldm_x4_trans(yh, tile_addr(thi, k, j));
                tc::ldm_x4_trans(yl, tile_addr(tlo, k, j));
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(-acc[2 * e], -acc[2 * e + 1], xh[e], xl[e]);
                tc::mma_block(y, xh, yh);
                tc::mma_block(y, xh, yl);
                tc::mma_block(y, xl, yh);
            }
            uint32_t yh[4], yl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(y[2 * e], y[2 * e + 1], yh[e], yl[e]);
            put_block(yh, thi, i, j);
            put_block(yl, tlo, i, j);
        }
        __syncthreads();
    }
    // row w of M T
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j <= w) {
            float acc[8] = {};
#pragma unroll
            for (int k = j; k < 4; ++k)
                if (k <= w) {
                    uint32_t yh[4], yl[4];
                    tc::ldm_x4_trans(yh, tile_addr(thi, k, j));
                    tc::ldm_x4_trans(yl, tile_addr(tlo, k, j));
                    tc::mma_block(acc, mh[k], yh);
                    tc::mma_block(acc, mh[k], yl);
                    tc::mma_block(acc, ml[k], yh);
                }
            uint32_t yh[4], yl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split2(acc[2 * e], acc[2 * e + 1], yh[e], yl[e]);
            put_block(yh, mhi, w, j);
            put_block(yl, mlo, w, j);
        }
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
        tc::bulk_store(p.tiles + item * p.tile_bytes, smem, p.tile_bytes);
        tc::bulk_commit();
        tc::bulk_wait_all();
    }
}

}  // namespace

cudaError_t launch_prep(const PrepArgs &p, cudaStream_t stream) {
    return launch_programmatic(delta_prep_kernel, dim3((unsigned)(p.a.B * p.nc * p.a.H)), dim3(kThreads), (size_t)kSmem,
                               stream, p);
}

}  // namespace delta
}  // namespace ssd
