// T and M T of every chunk of the gated delta rule (gated_delta_tc.cuh), and its
// decays: one block of four warps per (b, chunk, head), bf16 inputs, N <= 128.
//
// Everything is blocks of 16 x 16. Warp w forms row 3 - w of the blocks of K K^T and
// row w of Q K^T (mma.sync, K and Q exact, float32 sums), five blocks each, while warp 1
// first takes the sums of g, and scales them to A and M in registers. The diagonal blocks of I + A are inverted by substitution in
// float32, one warp each; the rest of T follows from
// [[Ta, 0], [-Tb A Ta, Tb]], first for the blocks of 32, then of 64, and M T row
// by row. Operands that were rounded go in as pairs hi + lo of bf16 (2^-17 is
// lost); the fragments of one product are the operands of the next, which
// the tensor-memory path cannot give at this size.
//
// The sums c are taken and kept as pairs of float32, value and remainder, so that
// a steep decay does not blur the differences of the tokens after it (float64
// would do, but its additions take a third of the block's time on this GPU).
//
// Bound by nothing alone: 18 thousand cycles a block of loads, products and
// barriers, six blocks per SM (B1 L4096 H24: 124 us, 125 with five, 127 with four), issue
// slots 41 % and shared memory 59 % used; 69 us for the 5120 items of B2 L2048 H80. Of the 470 us of
// B8 L2048 H80 storing the tiles costs 30, the products 29, loading K and Q 18,
// T from the diagonal blocks 10 and M T 5 (each left out in turn).
#include "gated_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kThreads = 128, kLo = 6;  // A's lo blocks begin at block 6
// shared memory (bytes): K and Q, 64 rows in panels of 64 columns (128-byte swizzle), whose place the tiles take once
// their products are formed, and where M T lo will be, and behind it, blocks of A of 512 bytes (hi, then lo) and the
// diagonal ones in float32; then the sums' factors
constexpr uint32_t kOffBlk = 3 * kTile, kOffSc = kOffBlk + 12 * 512 + 4 * 1024;
// c (base 2) rounded, 2^remainder, beta 2^-remainder, and that times exp(c at the end of the block of 16 - c)
enum { S_HI, S_ROW, S_INV, S_COL, S_N };
constexpr uint32_t kOffBar = kOffSc + S_N * kC * 4, kSmem = kOffBar + 16;

__device__ __forceinline__ int a_blk(int i, int j) { return (i * (i - 1)) / 2 + j; }
// 16-byte half of a row of a 512-byte block: 32 bytes per row, the halves of rows 4-7 and 12-15 swapped
__device__ __forceinline__ uint32_t in_blk(int row, int half) { return (uint32_t)(row * 32 + ((half ^ ((row >> 2) & 1)) << 4)); }

// a + b as a sum and its rounding error
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &e) {
    const float v = __fadd_rn(a, b), t = __fsub_rn(v, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(v, t)), __fsub_rn(b, t));
    s = v;
}
// (h + l) log2(e), as a pair
__device__ __forceinline__ void to_base2(float h, float l, float &ch, float &cl) {
    constexpr float kHi = 1.44269504088896341f, kLo = (float)(1.44269504088896340736 - (double)1.44269504088896341f);
    const float p = __fmul_rn(h, kHi);
    two_sum(p, __fmaf_rn(h, kHi, -p) + (h * kLo + l * kHi), ch, cl);
}

struct PrepParams {
    PrepArgs p;
    CUtensorMap mq, mk;
};

// Stores an accumulator block (r, k) of a tile as bf16 and, where lo is not null, its remainder.
__device__ __forceinline__ void put_block(const float (&y)[8], uint8_t *hi, uint8_t *lo, int r, int k, int lane) {
    const int g = lane >> 2;
    const uint32_t o = (uint32_t)(g * 128 + (lane & 3) * 4 + ((g & 7) << 4)) ^ (uint32_t)(32 * k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t h, l;
        split2(y[2 * e], y[2 * e + 1], h, l);
        const uint32_t at = (o ^ (16u * (e >> 1))) + 2048 * r + 1024 * (e & 1);
        *reinterpret_cast<uint32_t *>(hi + at) = h;
        if (lo) *reinterpret_cast<uint32_t *>(lo + at) = l;
    }
}

__device__ __forceinline__ void block_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// Row W of the blocks of Q K^T and row 3 - W of K K^T, five blocks together, scaled: M to fragments, A to shared memory.
// W is a template argument because the blocks are in registers.
template <int W>
__device__ __forceinline__ void rows_of(const PrepArgs &p, uint8_t *smem, int lane, uint32_t (&mh)[4][4], uint32_t (&ml)[4][4]) {
    constexpr int R = 3 - W;
    uint8_t *sK = smem, *sQ = smem + 16384, *blk = smem + kOffBlk;
    float *diag = reinterpret_cast<float *>(blk + 12 * 512);
    const float *sc = reinterpret_cast<const float *>(smem + kOffSc);
    const int g = lane >> 2, t2 = 2 * (lane & 3), NK = p.a.N <= 64 ? 64 : 128;
    // lane parts of addresses: the row (lane & 15) and half lane >> 4 of a block for ldmatrix (the pieces of column
    // block k are those of block 0 with 32 k in their place: xor); for the transposed operand of K K^T
    const uint32_t lt = (uint32_t)((lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4));
    const uint32_t ln = (uint32_t)(((lane & 7) + ((lane >> 4) << 3)) * 128 + ((((lane >> 3) & 1) ^ (lane & 7)) << 4));
    float ak[R + 1][8] = {}, aq[W + 1][8] = {};
    {
        const uint32_t k0 = tc::smem_u32(sK), q0 = tc::smem_u32(sQ);
#pragma unroll 2
        for (int ks = 0; ks < NK / 16; ++ks) {
            const uint32_t pan = (ks >> 2) * 8192, x = (ks & 3) << 5;
            uint32_t fk[4], fq[4];
            tc::ldm_x4(fk, k0 + pan + R * 2048 + (lt ^ x));
            tc::ldm_x4(fq, q0 + pan + W * 2048 + (lt ^ x));
#pragma unroll
            for (int j = 0; j <= (W > R ? W : R); ++j) {
                uint32_t fb[4];
                tc::ldm_x4(fb, k0 + pan + j * 2048 + (ln ^ x));
                if (j <= R) tc::mma_block(ak[j <= R ? j : 0], fk, fb);
                if (j <= W) tc::mma_block(aq[j <= W ? j : 0], fq, fb);
            }
        }
    }
    block_sync();  // the sums of g are there, and K and Q have been read
    // D beta of half n of block (row, j): rows g and g + 8
    auto factors = [&](int row, int j, int n, uint64_t &d0, uint64_t &d1) {
        const int r0 = 16 * row + g, col = 16 * j + 8 * n + t2;
        const float hi0 = sc[S_HI * kC + r0], hi1 = sc[S_HI * kC + r0 + 8];
        const float rf0 = sc[S_ROW * kC + r0], rf1 = sc[S_ROW * kC + r0 + 8];
        if (j < row) {  // exp(c_t - c_j) = exp(c_t - c_e) exp(c_e - c_j), e the block's last token
            const float he = sc[S_HI * kC + 16 * j + 15], re0 = rf0 * tc::ex2(hi0 - he), re1 = rf1 * tc::ex2(hi1 - he);
            const float2 cc = *reinterpret_cast<const float2 *>(sc + S_COL * kC + col);
            d0 = mul2(f2(re0, re0), f2(cc.x, cc.y)), d1 = mul2(f2(re1, re1), f2(cc.x, cc.y));
        } else {  // nothing above the diagonal (where the exponent could overflow)
            const float2 fc = *reinterpret_cast<const float2 *>(sc + S_INV * kC + col);
            const float2 hc = *reinterpret_cast<const float2 *>(sc + S_HI * kC + col);
            const float e00 = col <= r0 ? tc::ex2(hi0 - hc.x) : 0.f, e01 = col + 1 <= r0 ? tc::ex2(hi0 - hc.y) : 0.f;
            const float e10 = col <= r0 + 8 ? tc::ex2(hi1 - hc.x) : 0.f, e11 = col + 1 <= r0 + 8 ? tc::ex2(hi1 - hc.y) : 0.f;
            d0 = mul2(mul2(f2(rf0, rf0), f2(e00, e01)), f2(fc.x, fc.y));
            d1 = mul2(mul2(f2(rf1, rf1), f2(e10, e11)), f2(fc.x, fc.y));
        }
    };
#pragma unroll
    for (int j = 0; j <= R; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint64_t d0, d1;
            factors(R, j, n, d0, d1);
            const uint64_t a0 = mul2(f2(ak[j][4 * n], ak[j][4 * n + 1]), d0), a1 = mul2(f2(ak[j][4 * n + 2], ak[j][4 * n + 3]), d1);
            if (j == R) {  // what lies on and above the diagonal of A is not read
                float *o = diag + 256 * R + g * 16 + 8 * n + t2;
                *reinterpret_cast<uint64_t *>(o) = a0;
                *reinterpret_cast<uint64_t *>(o + 128) = a1;
            } else {
                uint32_t hi, lo;
                uint8_t *o = blk + a_blk(R, j) * 512 + t2 * 2;
                split2(a0, hi, lo);
                *reinterpret_cast<uint32_t *>(o + in_blk(g, n)) = hi;
                *reinterpret_cast<uint32_t *>(o + kLo * 512 + in_blk(g, n)) = lo;
                split2(a1, hi, lo);
                *reinterpret_cast<uint32_t *>(o + in_blk(g + 8, n)) = hi;
                *reinterpret_cast<uint32_t *>(o + kLo * 512 + in_blk(g + 8, n)) = lo;
            }
        }
    const uint64_t s2 = f2(p.a.scale, p.a.scale);
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            uint64_t d0, d1;
            factors(W, j, n, d0, d1);
            split2(mul2(mul2(f2(aq[j][4 * n], aq[j][4 * n + 1]), s2), d0), mh[j][2 * n], ml[j][2 * n]);
            split2(mul2(mul2(f2(aq[j][4 * n + 2], aq[j][4 * n + 3]), s2), d1), mh[j][2 * n + 1], ml[j][2 * n + 1]);
        }
}

// Row W of M T.
template <int W>
__device__ __forceinline__ void m_times_t(const PrepArgs &p, uint8_t *smem, int lane, const uint32_t (&mh)[4][4],
                                          const uint32_t (&ml)[4][4]) {
    const uint32_t lt = (uint32_t)((lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4));
    const uint32_t h0 = tc::smem_u32(smem) + lt, l0 = h0 + 2 * kTile;
    uint8_t *mhi = smem + kTile, *mlo = p.tile_bytes > kTilesFwd ? smem + 3 * kTile : nullptr;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        float acc[8] = {};
#pragma unroll
        for (int k = j; k <= W; ++k) {
            uint32_t yh[4], yl[4];
            tc::ldm_x4_trans(yh, (h0 ^ (32 * j)) + 2048 * k);
            tc::ldm_x4_trans(yl, (l0 ^ (32 * j)) + 2048 * k);
            tc::mma_block(acc, mh[k], yh);
            tc::mma_block(acc, mh[k], yl);
            tc::mma_block(acc, ml[k], yh);
        }
        put_block(acc, mhi, mlo, W, j, lane);
    }
    if (mlo) {  // above the diagonal, where A was
        const float zero[8] = {};
#pragma unroll
        for (int j = W + 1; j < 4; ++j) put_block(zero, mlo, nullptr, W, j, lane);
    }
}

__global__ void __launch_bounds__(kThreads, 6) delta_prep_kernel(const __grid_constant__ PrepParams prm) {
    pdl_wait();
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t &bar = *reinterpret_cast<uint64_t *>(smem + kOffBar);
    const PrepArgs &p = prm.p;
    const DeltaArgs &a = p.a;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int H = (int)a.H;
    const int h = (int)(blockIdx.x % H);
    const int64_t bc = blockIdx.x / H, c = bc % p.nc, b = bc / p.nc;
    const int64_t len = seq_len(a.seqlens, b, a.L), t0 = c * kC;
    if (blockIdx.x == 0 && tid == 0) *a.status = SSD_OK;
    if (c == 0) {
        const int pb = (int)row_blocks(a.P);
        for (int x = tid; x < 2 * pb; x += kThreads) p.flags[((x / pb) * a.B * H + b * H + h) * pb + x % pb] = 0;
    }
    if (t0 >= len) return;
    const int64_t item = (b * H + h) * p.nc + c;

    float gv[2] = {0.f, 0.f}, bv[2] = {0.f, 0.f};
    if (w == 1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int64_t t = t0 + 2 * lane + e, at = (b * a.L + t) * H + h;
            if (t < len) {
                gv[e] = to_f32(((const __nv_bfloat16 *)a.g)[at]);
                bv[e] = to_f32(((const __nv_bfloat16 *)a.beta)[at]);
            }
            // exp is 0 in float32 long before -256: the sums stay finite, the decays the same
            if (gv[e] < -256.f) gv[e] = -256.f;
        }
    }
    if (tid == 0) {
        tc::mbar_init(&bar, 1);
        tc::fence_mbar_init();
        const int grp = h / (int)(a.H / a.G), panels = a.N <= 64 ? 1 : 2;
        tc::mbar_arrive_expect_tx(&bar, panels * 2 * kTile);
        for (int k = 0; k < panels; ++k) {
            tc::tma_load_4d(smem + k * kTile, &prm.mk, &bar, 64 * k, grp, (int)t0, (int)b);
            tc::tma_load_4d(smem + 16384 + k * kTile, &prm.mq, &bar, 64 * k, grp, (int)t0, (int)b);
        }
    }
    __syncthreads();  // the barrier is initialised
    if (w == 1) {  // the sums, while the other warps' products run
        float *sc = reinterpret_cast<float *>(smem + kOffSc);
        float sh, sl;  // the inclusive sum of the lane's two tokens and all before, as a pair
        two_sum(gv[0], gv[1], sh, sl);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float uh = __shfl_up_sync(0xffffffffu, sh, o), ul = __shfl_up_sync(0xffffffffu, sl, o);
            float h2, l2;
            two_sum(sh, uh, h2, l2);
            if (lane >= o) two_sum(h2, l2 + (sl + ul), sh, sl);
        }
        float ch[2], cl[2], eh, el;  // c of the two tokens and at the end, in base-2 units
        to_base2(sh, sl, ch[1], cl[1]);
        two_sum(sh, -gv[1], eh, el);
        to_base2(eh, el + sl, ch[0], cl[0]);
        eh = __shfl_sync(0xffffffffu, ch[1], 31);
        el = __shfl_sync(0xffffffffu, cl[1], 31);
        const float he = __shfl_sync(0xffffffffu, ch[1], lane | 7);  // at the end of the block of 16
        float *o = p.scal + item * kScal + 2 * lane;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float row = tc::ex2(cl[e]), eg = tc::ex2(ch[e]) * row, inv = bv[e] * tc::ex2(-cl[e]);
            sc[S_HI * kC + 2 * lane + e] = ch[e];
            sc[S_ROW * kC + 2 * lane + e] = row;
            sc[S_INV * kC + 2 * lane + e] = inv;
            sc[S_COL * kC + 2 * lane + e] = inv * tc::ex2(he - ch[e]);
            o[SC_EG * kC + e] = eg;
            o[SC_NEG * kC + e] = -eg;
            o[SC_BETA * kC + e] = bv[e];
            o[SC_BTAIL * kC + e] = bv[e] * tc::ex2((eh - ch[e]) + (el - cl[e]));
            o[kScalDecay + e] = ch[e];
            o[kScalDecay + kC + e] = row;
            o[kScalDecay + 2 * kC + e] = inv;
        }
        if (lane == 0) p.scal[item * kScal + kScalEnd] = tc::ex2(eh) * tc::ex2(el);
    }
    const bool ok = tc::mbar_wait(&bar, 0, kWaitNs);
    if (t0 + kC > len && len < a.L) {  // tokens past the sequence's length
        for (int x = (int)(len - t0) * 8 + tid; x < kC * 8; x += kThreads)
            for (int k = 0; k < 4; ++k) reinterpret_cast<uint4 *>(smem + k * kTile)[x] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    uint8_t *thi = smem, *tlo = smem + 2 * kTile, *blk = smem + kOffBlk;
    const float *diag = reinterpret_cast<const float *>(blk + 12 * 512);
    uint32_t mh[4][4], ml[4][4];
    if (w == 0)
        rows_of<0>(p, smem, lane, mh, ml);
    else if (w == 1)
        rows_of<1>(p, smem, lane, mh, ml);
    else if (w == 2)
        rows_of<2>(p, smem, lane, mh, ml);
    else
        rows_of<3>(p, smem, lane, mh, ml);
    __syncthreads();
    // the tiles take the place of K and Q; zeros above the diagonal
    for (int j = w + 1; j < 4; ++j) {
        const float zero[8] = {};
        put_block(zero, thi, tlo, w, j, lane);
        put_block(zero, smem + kTile, nullptr, w, j, lane);
    }
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
    // Off the diagonal, T_ij = -sum_k (sum_m T_im A_mk) T_kj: first within the blocks of 32 (warps 1 and 3: i = w,
    // j = w - 1, one k and m each), then the block of 32 below them (i = 2, 3, j = 0, 1, m from 2 to i, k from j to 1)
    const uint32_t lt = (uint32_t)((lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4));
    const uint32_t h0 = tc::smem_u32(thi) + lt, lb = tc::smem_u32(blk) + in_blk(lane & 15, lane >> 4);
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
                for (int m = m0; m <= i; ++m) {
                    const uint32_t x = (h0 ^ (32 * m)) + 2048 * i, o = lb + a_blk(m, k) * 512;
                    tc::ldm_x4(xh, x);
                    tc::ldm_x4(xl, x + 2 * kTile);
                    tc::ldm_x4_trans(yh, o);
                    tc::ldm_x4_trans(yl, o + kLo * 512);
                    tc::mma_block(acc, xh, yh);
                    tc::mma_block(acc, xh, yl);
                    tc::mma_block(acc, xl, yh);
                }
                const uint32_t x = (h0 ^ (32 * j)) + 2048 * k;
                tc::ldm_x4_trans(yh, x);
                tc::ldm_x4_trans(yl, x + 2 * kTile);
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(-acc[2 * e], -acc[2 * e + 1], xh[e], xl[e]);
                tc::mma_block(y, xh, yh);
                tc::mma_block(y, xh, yl);
                tc::mma_block(y, xl, yh);
            }
            put_block(y, thi, tlo, i, j, lane);
        }
        __syncthreads();
    }
    if (w == 0)
        m_times_t<0>(p, smem, lane, mh, ml);
    else if (w == 1)
        m_times_t<1>(p, smem, lane, mh, ml);
    else if (w == 2)
        m_times_t<2>(p, smem, lane, mh, ml);
    else
        m_times_t<3>(p, smem, lane, mh, ml);
    tc::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
        if (!ok) atomicCAS(a.status, SSD_OK, SSD_ERR_TIMEOUT);
        tc::bulk_store(p.tiles + item * p.tile_bytes, smem, p.tile_bytes);
        tc::bulk_commit();
        tc::bulk_wait_read_all();
    }
}

}  // namespace

cudaError_t launch_prep(const PrepArgs &p, cudaStream_t stream) {
    PrepParams q;
    q.p = p;
    if (!tma_map_heads(&q.mq, p.a.q, p.a.N, p.a.G, p.a.L, p.a.B, 64, kC, true) ||
        !tma_map_heads(&q.mk, p.a.k, p.a.N, p.a.G, p.a.L, p.a.B, 64, kC, true))
        return cudaErrorInvalidValue;
    return launch_programmatic(delta_prep_kernel, dim3((unsigned)(p.a.B * p.nc * p.a.H)), dim3(kThreads), (size_t)kSmem,
                               stream, q);
}

}  // namespace delta
}  // namespace ssd
