// Gated delta rule over a sequence on the tensor cores: bf16 inputs, chunks of
// 64 tokens, state width N <= 128, float32 state.
//
// Within a chunk, with c the inclusive sums of g, S0 the entering state and
// D_tj = exp(c_t - c_j), the recurrence is a triangular solve:
//     A_tj = beta_t D_tj (k_t . k_j), j < t          T = (I + A)^-1
//     R = beta (V - exp(c) K S0^T)                   U = T R
//     Y = scale (exp(c) Q S0^T + M U)                M_tj = D_tj (q_t . k_j), j <= t
//     S1 = exp(c_63) S0 + (exp(c_63 - c) U)^T K
// T and M do not depend on the state, so T and M T are formed ahead of the
// chain, which then has three products per chunk, each waiting for the one
// before (everything transposed: a row of the state is one TMEM lane):
//     [Q S0^T | K S0^T]^T = S0 [Q; K]^T              (M = 128 state rows, N = 128, K = N)
//     [U | M U]^T         = R^T [T; M T]^T           (N = 128, K = 64)
//     S1                  = exp(c_63) S0 + U~^T K    (N = 128, K = 64)
// The A operands (S, R, U~) are written to TMEM by the thread that owns the
// row, so nothing but the barriers of the MMAs crosses threads on the chain.
//
// A CTA owns 128 state rows that share keys: the 64 rows of two heads of one
// group (NH = 2: two T's, R of one head beside zeros for the other, so that both
// products add up in one accumulator), or up to 128 rows of one head (NH = 1).
//
// Precision: the state is float32 in TMEM. S, T, R and U~ enter the products
// as pairs hi + lo of bf16 (2^-17 of the value is lost), K, Q and V are exact, so
// that the state keeps about 17 bits through a chunk; products that only reach
// y (Q S0^T and M U) use hi alone, which is below y's own rounding. The sums c are
// taken in float64 and kept as a float32 and its remainder, so that a steep decay
// does not blur the differences after it.
//
// TMEM (512 columns): QS [0,64) | KS, then U [64,128) | M U [128,192) |
// [Q; K] K^T of the next chunk [192,256) | S float32 [256,384) | operands [384,512):
// S hi 64, lo 64; R of each head hi 32, lo 32; U~ hi 32, lo 32, one after the other.
//
// Warps: 0 TMA loads; 1 MMAs of the chain; 2 the sums of g, decays, and the
// zeroing of tokens past a sequence's length; 3 MMAs of [Q; K] K^T; 4-11 the
// chain's elementwise steps (two warps per 32 rows, half of the tokens or columns
// each); then 4 warps per head for T and M T.
//
// T: the four 16x16 blocks on the diagonal are inverted by substitution in
// float32, one warp each; then warp i forms row i of blocks from the diagonal
// outwards, T_ij = -(sum_{j<k<=i} T_ik A_kj) T_jj, with mma.sync on 16x16
// blocks: the result of one product is the next one's operand in the same
// registers, which the tensor-memory path cannot give at this size.
//
// Every wait is bounded (2 s): a timeout raises a flag, after which no wait
// waits; the copies and products in flight are waited for (bounded too), and the
// status word records SSD_ERR_TIMEOUT.
#include <cuda.h>

#include <cstdint>

#include "common.cuh"
#include "launch.h"
#include "ssd_scan.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kC = 64;         // tokens per chunk
constexpr int kStages = 3;     // chunks of K and Q (and scalars) in flight
constexpr int kVStages = 2;
constexpr int kChainWarp0 = 4, kChainThreads = 256, kPrepWarp0 = 12;
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ constexpr int threads_of(int NH) { return 32 * kPrepWarp0 + 128 * NH; }

struct DeltaTcParams {
    DeltaArgs a;
    CUtensorMap mq, mk, mv, my;
    int units_per_b;  // NH = 2: head pairs; NH = 1: heads times blocks of 128 rows
    int pblocks;      // NH = 1: ceil(P / 128)
};

// per-chunk scalars of one head, one float per token each
enum { SC_HI, SC_ROW, SC_BROW, SC_INV, SC_EG, SC_BETA, SC_BEG, SC_TAIL, SC_ROWS };
constexpr int kScal = SC_ROWS * kC + 4;  // then exp(c_63)

// shared memory carve (bytes from the 1024-aligned base)
constexpr uint32_t kOffKQ = 0;                             // stages of 32 KB: two panels of 64 columns, each
                                                           // 64 rows of Q, then 64 rows of K
constexpr uint32_t kOffV = kOffKQ + kStages * 32768;       // stages of 16 KB: [32-row block][token][row], y in place
constexpr uint32_t kOffT = kOffV + kVStages * 16384;       // per head 16 KB: T hi, M T
__host__ __device__ constexpr uint32_t off_tlo(int NH) { return kOffT + NH * 16384; }
__host__ __device__ constexpr uint32_t off_a(int NH) { return off_tlo(NH) + NH * 8192; }  // per head A hi 8 KB, A lo 8 KB
__host__ __device__ constexpr uint32_t off_scal(int NH) { return off_a(NH) + NH * 16384; }
__host__ __device__ constexpr uint32_t off_bar(int NH) { return off_scal(NH) + kStages * NH * kScal * 4; }
enum {
    BAR_KQ_FULL = 0,                        // [stages] TMA
    BAR_KQ_EMPTY = BAR_KQ_FULL + kStages,   // [stages] last product of the chunk
    BAR_READY = BAR_KQ_EMPTY + kStages,     // [stages] K, Q masked, scalars written
    BAR_SC_EMPTY = BAR_READY + kStages,     // [stages] chain threads
    BAR_V_FULL = BAR_SC_EMPTY + kStages,    // [v stages]
    BAR_V_EMPTY = BAR_V_FULL + kVStages,    // [v stages] chain warps
    BAR_GR_FULL = BAR_V_EMPTY + kVStages,
    BAR_GR_EMPTY,
    BAR_T_FULL,
    BAR_T_EMPTY,
    BAR_S_FULL,
    BAR_A_DONE,
    BAR_R_FULL,
    BAR_B_DONE,
    BAR_U_FULL,
    BAR_C_DONE,
    BAR_DRAIN,                              // [2] the MMA warps' last products
    kBars = BAR_DRAIN + 2
};
constexpr size_t smem_bytes(int NH) { return off_bar(NH) + kBars * 8 + 16 + 1024; }
static_assert(smem_bytes(2) <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
// (x, y) as bf16 pairs hi and lo, hi + lo within 2^-17 of each
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack2(x, y);
    lo = pack2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *fail) {
    const uint32_t addr = tc::smem_u32(bar);
    if (tc::mbar_try_wait(addr, parity)) return true;
    if (*fail) return false;
    const uint64_t t0 = tc::global_ns();
    for (;;) {
        if (tc::mbar_try_wait(addr, parity)) return true;
        if (*fail) return false;
        if (tc::global_ns() - t0 > kWaitNs) {
            *fail = 1;
            return false;
        }
    }
}
__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <int NH> __global__ void __launch_bounds__(threads_of(NH), 1)
delta_chunk_tc(const __grid_constant__ DeltaTcParams prm) {
    const DeltaArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = (int)a.P, N = (int)a.N;
    const int NK = N <= 64 ? 64 : 128;  // state columns the products run over

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sKQ = smem + kOffKQ, *sV = smem + kOffV, *sT = smem + kOffT, *sTlo = smem + off_tlo(NH);
    uint8_t *sA = smem + off_a(NH);
    float *scal = reinterpret_cast<float *>(smem + off_scal(NH));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + off_bar(NH));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int64_t b = blockIdx.x / prm.units_per_b;
    const int un = (int)(blockIdx.x % prm.units_per_b);
    const int h0 = NH == 2 ? 2 * un : un / prm.pblocks;
    const int prow0 = NH == 2 ? 0 : (un % prm.pblocks) * 128;  // state row of lane 0
    const int grp = h0 / (int)(a.H / a.G);

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            int count = 1;
            if (k >= BAR_SC_EMPTY && k < BAR_SC_EMPTY + kStages) count = kChainThreads;
            if (k >= BAR_V_EMPTY && k < BAR_V_EMPTY + kVStages) count = kChainThreads / 32;
            if (k == BAR_GR_EMPTY || k == BAR_T_FULL) count = 128 * NH;
            if (k == BAR_S_FULL || k == BAR_R_FULL || k == BAR_U_FULL) count = kChainThreads;
            tc::mbar_init(bars + k, count);
        }
        tc::fence_mbar_init();
        *fail = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    // the blocks above the diagonal of T and M T stay zero
    for (uint32_t x = tid; x < (uint32_t)NH * 24576 / 16; x += threads_of(NH))
        reinterpret_cast<uint4 *>(sT)[x] = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async_smem();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tQS = tmem, tU = tmem + 64, tO = tmem + 128, tGR = tmem + 192, tS = tmem + 256, tOp = tmem + 384;
    pdl_wait();
    const int64_t len = seq_len(a.seqlens, b, a.L);
    const int nc = (int)((len + kC - 1) / kC);
    if (blockIdx.x == 0 && tid == 0) *a.status = SSD_OK;

    if (warp == 0) {
        // ------------------------------------------------------- TMA loads
        if (lane == 0) {
            auto load_v = [&](int c) -> bool {
                const int s = c % kVStages;
                if (!wait_on(&bars[BAR_V_EMPTY + s], ((c / kVStages) & 1) ^ 1, fail)) return false;
                tc::mbar_arrive_expect_tx(&bars[BAR_V_FULL + s], 16384u);
                for (int k = 0; k < 4; ++k) {
                    const int hh = NH == 2 ? h0 + (k >> 1) : h0, p = NH == 2 ? 32 * (k & 1) : prow0 + 32 * k;
                    tc::tma_load_4d(sV + s * 16384 + k * 4096, &prm.mv, &bars[BAR_V_FULL + s], p, hh, c * kC, (int)b);
                }
                return true;
            };
            int kq_done = 0, v_done = 0;
            for (int c = 0; c <= nc; ++c) {  // K and Q run one chunk ahead of V
                if (c < nc) {
                    const int s = c % kStages;
                    if (!wait_on(&bars[BAR_KQ_EMPTY + s], ((c / kStages) & 1) ^ 1, fail)) break;
                    uint64_t *bar = &bars[BAR_KQ_FULL + s];
                    uint8_t *d = sKQ + s * 32768;
                    tc::mbar_arrive_expect_tx(bar, 32768u);
                    for (int k = 0; k < 2; ++k) {
                        tc::tma_load_4d(d + k * 16384, &prm.mq, bar, 64 * k, grp, c * kC, (int)b);
                        tc::tma_load_4d(d + k * 16384 + 8192, &prm.mk, bar, 64 * k, grp, c * kC, (int)b);
                    }
                    kq_done = c + 1;
                }
                if (c > 0) {
                    if (!load_v(c - 1)) break;
                    v_done = c;
                }
            }
            // no copy outlives the block, even where a wait gave up
            for (int c = imax(0, kq_done - kStages); c < kq_done; ++c)
                tc::mbar_wait(&bars[BAR_KQ_FULL + c % kStages], (c / kStages) & 1, kWaitNs);
            for (int c = imax(0, v_done - kVStages); c < v_done; ++c)
                tc::mbar_wait(&bars[BAR_V_FULL + c % kVStages], (c / kVStages) & 1, kWaitNs);
        }
    } else if (warp == 1) {
        // --------------------------------------------- MMAs of the chain
        if (lane == 0) {
            const uint32_t id128 = tc::idesc_bf16(128, 128, false, false), id64 = tc::idesc_bf16(128, 64, false, false);
            const uint32_t idS = tc::idesc_bf16(128, NK, false, true);
            const uint32_t t0 = tc::smem_u32(sT), tl0 = tc::smem_u32(sTlo);
            for (int c = 0; c < nc; ++c) {
                const int s = c % kStages;
                const uint32_t ph = c & 1, kq = tc::smem_u32(sKQ + s * 32768);
                if (!wait_on(&bars[BAR_KQ_FULL + s], (c / kStages) & 1, fail)) break;
                if (!wait_on(&bars[BAR_READY + s], (c / kStages) & 1, fail)) break;
                if (!wait_on(&bars[BAR_S_FULL], ph, fail)) break;
                tc::tc_fence_after();
                for (int k = 0; k < NK; k += 16)
                    tc::mma_bf16_ts(tQS, tOp + k / 2, tc::sdesc_sw128(kq + (k >> 6) * 16384 + (k & 63) * 2, 16, 1024),
                                    id128, k > 0);
                for (int k = 0; k < NK; k += 16)
                    tc::mma_bf16_ts(tU, tOp + 64 + k / 2,
                                    tc::sdesc_sw128(kq + 8192 + (k >> 6) * 16384 + (k & 63) * 2, 16, 1024), id64, 1);
                tc::mma_commit(&bars[BAR_A_DONE]);
                if (!wait_on(&bars[BAR_T_FULL], ph, fail)) break;
                if (!wait_on(&bars[BAR_R_FULL], ph, fail)) break;
                tc::tc_fence_after();
                for (int hf = 0; hf < NH; ++hf) {
                    const uint32_t r0 = tOp + 64 * hf;
                    for (int k = 0; k < kC; k += 16)
                        tc::mma_bf16_ts(tU, r0 + k / 2, tc::sdesc_sw128(t0 + hf * 16384 + k * 2, 16, 1024), id128,
                                        hf > 0 || k > 0);
                    for (int k = 0; k < kC; k += 16)
                        tc::mma_bf16_ts(tU, r0 + 32 + k / 2, tc::sdesc_sw128(t0 + hf * 16384 + k * 2, 16, 1024), id64, 1);
                    for (int k = 0; k < kC; k += 16)
                        tc::mma_bf16_ts(tU, r0 + k / 2, tc::sdesc_sw128(tl0 + hf * 8192 + k * 2, 16, 1024), id64, 1);
                }
                tc::mma_commit(&bars[BAR_B_DONE]);
                tc::mma_commit(&bars[BAR_T_EMPTY]);
                if (!wait_on(&bars[BAR_U_FULL], ph, fail)) break;
                tc::tc_fence_after();
                for (int k = 0; k < 2 * kC; k += 16)  // U~ hi, then lo
                    tc::mma_bf16_ts(tS, tOp + k / 2, tc::sdesc_sw128(kq + 8192 + (k & 63) * 128, 16384, 1024), idS, 1);
                tc::mma_commit(&bars[BAR_C_DONE]);
                tc::mma_commit(&bars[BAR_KQ_EMPTY + s]);
            }
            tc::mma_commit(&bars[BAR_DRAIN]);
            tc::mbar_wait(&bars[BAR_DRAIN], 0, kWaitNs);
        }
    } else if (warp == 2) {
        // ------------------------ decays of each chunk; tokens past the length
        for (int c = 0; c < nc; ++c) {
            const int s = c % kStages;
            const int64_t t0 = (int64_t)c * kC;
            float gv[NH][2], bv[NH][2];
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t t = t0 + 2 * lane + e, at = (b * a.L + t) * a.H + h0 + hf;
                    gv[hf][e] = t < len ? to_f32(((const __nv_bfloat16 *)a.g)[at]) : 0.f;
                    // exp is 0 in float32 long before -256: the sums stay finite, the decays the same
                    if (gv[hf][e] < -256.f) gv[hf][e] = -256.f;
                    bv[hf][e] = t < len ? to_f32(((const __nv_bfloat16 *)a.beta)[at]) : 0.f;
                }
            wait_on(&bars[BAR_SC_EMPTY + s], ((c / kStages) & 1) ^ 1, fail);
            __syncwarp();
#pragma unroll
            for (int hf = 0; hf < NH; ++hf) {
                double sum = (double)gv[hf][0] + (double)gv[hf][1];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double u = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += u;
                }
                const double end = __shfl_sync(0xffffffffu, sum, 31) * (double)kLog2e;
                float *o = scal + (s * NH + hf) * kScal;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const double c2 = (e ? sum : sum - (double)gv[hf][1]) * (double)kLog2e;  // base-2 units
                    const float hi = (float)c2, lo = (float)(c2 - (double)hi), eg = exp2f(hi), be = bv[hf][e];
                    const int t = 2 * lane + e;
                    o[SC_HI * kC + t] = hi;
                    o[SC_ROW * kC + t] = exp2f(lo);
                    o[SC_BROW * kC + t] = be * exp2f(lo);
                    o[SC_INV * kC + t] = exp2f(-lo);
                    o[SC_EG * kC + t] = eg;
                    o[SC_BETA * kC + t] = be;
                    o[SC_BEG * kC + t] = be * eg;
                    o[SC_TAIL * kC + t] = exp2f((float)(end - c2));
                }
                if (lane == 0) o[SC_ROWS * kC] = exp2f((float)end);
            }
            wait_on(&bars[BAR_KQ_FULL + s], (c / kStages) & 1, fail);
            __syncwarp();
            if (t0 + kC > len && len < a.L) {
                for (int x = (int)(len - t0) * 8 + lane; x < kC * 8; x += 32)
                    for (int k = 0; k < 4; ++k)  // Q and K rows of both panels
                        reinterpret_cast<uint4 *>(sKQ + s * 32768 + k * 8192)[x] = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[BAR_READY + s]);
        }
    } else if (warp == 3) {
        // ------------------------------------------------ [Q; K] K^T, ahead of the chain
        if (lane == 0) {
            const uint32_t id = tc::idesc_bf16(128, 64, false, false);
            for (int c = 0; c < nc; ++c) {
                const int s = c % kStages;
                const uint32_t kq = tc::smem_u32(sKQ + s * 32768);
                if (!wait_on(&bars[BAR_KQ_FULL + s], (c / kStages) & 1, fail)) break;
                if (!wait_on(&bars[BAR_READY + s], (c / kStages) & 1, fail)) break;
                if (!wait_on(&bars[BAR_GR_EMPTY], (c & 1) ^ 1, fail)) break;
                tc::tc_fence_after();
                for (int k = 0; k < NK; k += 16) {
                    const uint32_t at = kq + (k >> 6) * 16384 + (k & 63) * 2;
                    tc::mma_bf16(tGR, tc::sdesc_sw128(at, 16, 1024), tc::sdesc_sw128(at + 8192, 16, 1024), id, k > 0);
                }
                tc::mma_commit(&bars[BAR_GR_FULL]);
            }
            tc::mma_commit(&bars[BAR_DRAIN + 1]);
            tc::mbar_wait(&bars[BAR_DRAIN + 1], 0, kWaitNs);
        }
    } else if (warp < kPrepWarp0) {
        // ---------------------------------------- elementwise steps of the chain
        const int cw = warp - kChainWarp0, q = cw & 3, ch = cw >> 2;
        const int hf = NH == 2 ? q >> 1 : 0, h = h0 + hf;
        const int p32 = NH == 2 ? 32 * (q & 1) : prow0 + 32 * q, p = p32 + lane;  // the warp's first row, this thread's
        const uint32_t lq = (uint32_t)(32 * q) << 16;
        const int64_t srow = ((b * a.H + h) * a.P + p) * a.N;
        // 64 columns of the state as hi + lo operands, and scaled for the next accumulation
        auto put_state = [&](const float (&v)[32], int half, float eq) {
            uint32_t hi[16], lo[16], sc[32];
#pragma unroll
            for (int k = 0; k < 16; ++k) split2(v[2 * k], v[2 * k + 1], hi[k], lo[k]);
#pragma unroll
            for (int k = 0; k < 32; ++k) sc[k] = __float_as_uint(v[k] * eq);
            const int c0 = 64 * ch + 32 * half;
            tc::tmem_st16(tOp + lq + c0 / 2, hi);
            tc::tmem_st16(tOp + 64 + lq + c0 / 2, lo);
            tc::tmem_st32(tS + lq + c0, sc);
        };
        if (nc > 0) {
            wait_on(&bars[BAR_READY], 0, fail);
            __syncwarp();
            const float eq = scal[hf * kScal + SC_ROWS * kC];
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const int n = 64 * ch + 32 * half + k;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (a.init && p < P && n < N) x = *reinterpret_cast<const float4 *>(a.init + srow + n);
                    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
                }
                put_state(v, half, eq);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars[BAR_S_FULL]);
        }
        for (int c = 0; c < nc; ++c) {
            const int s = c % kStages, vs = c % kVStages;
            const uint32_t ph = c & 1;
            const float *sc = scal + (s * NH + hf) * kScal + 32 * ch;
            uint8_t *vt = sV + vs * 16384 + q * 4096 + ch * 2048;  // this warp's [32 tokens][32 rows]
            // R^T = beta v - beta exp(c) (K S0^T)^T
            wait_on(&bars[BAR_V_FULL + vs], (c / kVStages) & 1, fail);
            wait_on(&bars[BAR_A_DONE], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
            {
                float ks[32];
                tc::tmem_ld32(tU + lq + 32 * ch, ks);
                tc::tmem_ld_wait();
                const int valid = (int)imin<int64_t>(32, len - (int64_t)c * kC - 32 * ch);
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 be = *reinterpret_cast<const float4 *>(sc + SC_BETA * kC + k);
                    const float4 bg = *reinterpret_cast<const float4 *>(sc + SC_BEG * kC + k);
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = to_f32(reinterpret_cast<const __nv_bfloat16 *>(vt)[(k + e) * 32 + lane]);
                        if (k + e >= valid) v[e] = 0.f;  // whatever lies past the length
                    }
                    split2(be.x * v[0] - bg.x * ks[k], be.y * v[1] - bg.y * ks[k + 1], hi[k / 2], lo[k / 2]);
                    split2(be.z * v[2] - bg.z * ks[k + 2], be.w * v[3] - bg.w * ks[k + 3], hi[k / 2 + 1], lo[k / 2 + 1]);
                }
                tc::tmem_st16(tOp + lq + 64 * hf + 16 * ch, hi);
                tc::tmem_st16(tOp + lq + 64 * hf + 32 + 16 * ch, lo);
                if (NH == 2) {  // zeros in the other head's operand
#pragma unroll
                    for (int k = 0; k < 16; ++k) hi[k] = 0u;
                    tc::tmem_st16(tOp + lq + 64 * (hf ^ 1) + 16 * ch, hi);
                    tc::tmem_st16(tOp + lq + 64 * (hf ^ 1) + 32 + 16 * ch, hi);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&bars[BAR_R_FULL]);
            }
            if (c > 0) {  // the previous chunk's y has left its buffer
                if (lane == 0) {
                    tc::bulk_wait_read_all();
                    tc::mbar_arrive(&bars[BAR_V_EMPTY + (vs ^ 1)]);
                }
                __syncwarp();
            }
            // U~^T = exp(c_63 - c) U^T
            wait_on(&bars[BAR_B_DONE], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
            {
                float u[32];
                tc::tmem_ld32(tU + lq + 32 * ch, u);
                tc::tmem_ld_wait();
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const float4 tl = *reinterpret_cast<const float4 *>(sc + SC_TAIL * kC + k);
                    split2(u[k] * tl.x, u[k + 1] * tl.y, hi[k / 2], lo[k / 2]);
                    split2(u[k + 2] * tl.z, u[k + 3] * tl.w, hi[k / 2 + 1], lo[k / 2 + 1]);
                }
                tc::tmem_st16(tOp + lq + 16 * ch, hi);
                tc::tmem_st16(tOp + lq + 32 + 16 * ch, lo);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&bars[BAR_U_FULL]);
            }
            // y, under the state's product: the tile of v holds it for the store
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float qs[16], o[16];
                tc::tmem_ld16(tQS + lq + 32 * ch + 16 * half, qs);
                tc::tmem_ld16(tO + lq + 32 * ch + 16 * half, o);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const float4 eg = *reinterpret_cast<const float4 *>(sc + SC_EG * kC + 16 * half + k);
                    __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(vt) + (16 * half + k) * 32 + lane;
                    d[0] = __float2bfloat16_rn(a.scale * fmaf(eg.x, qs[k], o[k]));
                    d[32] = __float2bfloat16_rn(a.scale * fmaf(eg.y, qs[k + 1], o[k + 1]));
                    d[64] = __float2bfloat16_rn(a.scale * fmaf(eg.z, qs[k + 2], o[k + 2]));
                    d[96] = __float2bfloat16_rn(a.scale * fmaf(eg.w, qs[k + 3], o[k + 3]));
                }
            }
            tc::tc_fence_before();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && p32 < P) {
                tc::tma_store_4d(&prm.my, vt, p32, h, c * kC + 32 * ch, (int)b);
                tc::bulk_commit();
            }
            tc::mbar_arrive(&bars[BAR_SC_EMPTY + s]);
            // the state that enters the next chunk
            wait_on(&bars[BAR_C_DONE], ph, fail);
            const int sn = (c + 1) % kStages;
            if (c + 1 < nc) wait_on(&bars[BAR_READY + sn], ((c + 1) / kStages) & 1, fail);
            __syncwarp();
            tc::tc_fence_after();
            if (c + 1 < nc) {
                const float eq = scal[(sn * NH + hf) * kScal + SC_ROWS * kC];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float v[32];
                    tc::tmem_ld32(tS + lq + 64 * ch + 32 * half, v);
                    tc::tmem_ld_wait();
                    put_state(v, half, eq);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&bars[BAR_S_FULL]);
            } else if (a.final_state) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    float v[32];
                    tc::tmem_ld32(tS + lq + 64 * ch + 32 * half, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const int n = 64 * ch + 32 * half + k;
                        if (p < P && n < N)
                            *reinterpret_cast<float4 *>(a.final_state + srow + n) =
                                make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
                tc::tc_fence_before();
            }
        }
        if (nc == 0 && a.final_state && p < P)
            for (int n = 64 * ch; n < imin(N, 64 * ch + 64); n += 4)
                *reinterpret_cast<float4 *>(a.final_state + srow + n) =
                    a.init ? *reinterpret_cast<const float4 *>(a.init + srow + n) : make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < P)  // y is zero past the last chunk
            for (int64_t t = (int64_t)nc * kC + ch; t < a.L; t += 2)
                ((__nv_bfloat16 *)a.y)[((b * a.L + t) * a.H + h) * P + p] = __float2bfloat16_rn(0.f);
        if (lane == 0) tc::bulk_wait_all();
    } else {
        // ------------------------------------------------ T and M T of each head
        const int hf = NH == 2 ? (warp - kPrepWarp0) >> 2 : 0, w = warp & 3;
        const uint32_t lq = (uint32_t)(32 * w) << 16;
        const bool is_k = w >= 2;          // lanes 64-127 of [Q; K] K^T are the rows of K
        const int t = 32 * (w & 1) + lane, bt = t >> 4;
        uint8_t *ahi = sA + hf * 16384, *alo = ahi + 8192, *thi = sT + hf * 16384, *mt = thi + 8192, *tlo = sTlo + hf * 8192;
        // 16-byte piece `pc` of row `row` of a tile of 64 columns
        auto piece = [](int row, int pc) { return (uint32_t)(row * 128 + ((pc ^ (row & 7)) << 4)); };
        // this lane's row address of the 16x16 block (r, k) for ldmatrix
        auto block_addr = [&](const uint8_t *tile, int r, int k) {
            return tc::smem_u32(tile) + piece(16 * r + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4));
        };
        const int g = lane >> 2, cc = 2 * (lane & 3);
        // stores an accumulator block as bf16 (and its remainder)
        auto put_block = [&](const uint32_t (&f)[4], uint8_t *tile, int r, int k) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint32_t *>(tile + piece(16 * r + g + (e & 1) * 8, 2 * k + (e >> 1)) + cc * 2) = f[e];
        };
        for (int c = 0; c < nc; ++c) {
            const int s = c % kStages;
            const float *sc = scal + (s * NH + hf) * kScal;
            wait_on(&bars[BAR_READY + s], (c / kStages) & 1, fail);
            wait_on(&bars[BAR_GR_FULL], c & 1, fail);
            __syncwarp();
            tc::tc_fence_after();
            uint32_t mrow[32];  // rows of Q: M as bf16 pairs
            {
                const float hi_t = sc[SC_HI * kC + t], rf = sc[(is_k ? SC_BROW : SC_ROW) * kC + t];
#pragma unroll
                for (int bj = 0; bj < 4; ++bj) {
                    float x[16];
                    tc::tmem_ld16(tGR + lq + 16 * bj, x);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const int j = 16 * bj + k;
                        const float4 hj = *reinterpret_cast<const float4 *>(sc + SC_HI * kC + j);
                        const float4 fj = *reinterpret_cast<const float4 *>(sc + SC_INV * kC + j);
                        const float hv[4] = {hj.x, hj.y, hj.z, hj.w}, fv[4] = {fj.x, fj.y, fj.z, fj.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool on = is_k ? j + e < t : j + e <= t;
                            x[k + e] = on ? (x[k + e] * rf) * (tc::ex2(hi_t - hv[e]) * fv[e]) : 0.f;
                        }
                    }
                    if (!is_k) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) mrow[8 * bj + k] = pack2(x[2 * k], x[2 * k + 1]);
                    } else if (bj == bt) {  // a diagonal block: float32, in the space of its hi and lo parts
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<float4 *>((k < 2 ? ahi : alo) + piece(t, 2 * bj + (k & 1))) =
                                make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                    } else if (bj < bt) {
                        uint32_t hi[8], lo[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) split2(x[2 * k], x[2 * k + 1], hi[k], lo[k]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            *reinterpret_cast<uint4 *>(ahi + piece(t, 2 * bj + k)) =
                                make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                            *reinterpret_cast<uint4 *>(alo + piece(t, 2 * bj + k)) =
                                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                        }
                    }
                }
            }
            tc::tc_fence_before();
            tc::mbar_arrive(&bars[BAR_GR_EMPTY]);
            named_sync(1 + hf);
            // column `lane & 15` of the inverse of diagonal block w, by substitution
            float x[16];
            {
                const int col = lane & 15;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float acc = i == col ? 1.f : 0.f;
#pragma unroll
                    for (int k = 0; 4 * k < i; ++k) {
                        const float4 v = *reinterpret_cast<const float4 *>((k < 2 ? ahi : alo) +
                                                                           piece(16 * w + i, 2 * w + (k & 1)));
                        const float av[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (4 * k + e < i) acc = fmaf(-av[e], x[4 * k + e], acc);
                    }
                    x[i] = acc;
                }
            }
            // the previous chunk's products have read T and M T
            wait_on(&bars[BAR_T_EMPTY], (c & 1) ^ 1, fail);
            __syncwarp();
            if (!is_k) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k <= 2 * bt + 1)
                        *reinterpret_cast<uint4 *>(mt + piece(t, k)) =
                            make_uint4(mrow[4 * k], mrow[4 * k + 1], mrow[4 * k + 2], mrow[4 * k + 3]);
            }
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t at = piece(16 * w + i, 2 * w + (lane >> 3)) + (lane & 7) * 2;
                    const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
                    *reinterpret_cast<__nv_bfloat16 *>(thi + at) = hi;
                    *reinterpret_cast<__nv_bfloat16 *>(tlo + at) = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
                }
            }
            named_sync(1 + hf);
            // row w of blocks, from the diagonal outwards: block d is T_{w, w-d}
            uint32_t fh[3][4], fl[3][4];
            tc::ldm_x4(fh[0], block_addr(thi, w, w));
            tc::ldm_x4(fl[0], block_addr(tlo, w, w));
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int j = w - d;
                if (j < 0) break;
                float acc[8] = {};
                uint32_t bh[4], bl[4];
#pragma unroll
                for (int e = 0; e < d; ++e) {
                    tc::ldm_x4_trans(bh, block_addr(ahi, w - e, j));
                    tc::ldm_x4_trans(bl, block_addr(alo, w - e, j));
                    tc::mma_block(acc, fh[e], bh);
                    tc::mma_block(acc, fh[e], bl);
                    tc::mma_block(acc, fl[e], bh);
                }
                uint32_t xh[4], xl[4];
                split2(-acc[0], -acc[1], xh[0], xl[0]);
                split2(-acc[2], -acc[3], xh[1], xl[1]);
                split2(-acc[4], -acc[5], xh[2], xl[2]);
                split2(-acc[6], -acc[7], xh[3], xl[3]);
                float y[8] = {};
                tc::ldm_x4_trans(bh, block_addr(thi, j, j));
                tc::ldm_x4_trans(bl, block_addr(tlo, j, j));
                tc::mma_block(y, xh, bh);
                tc::mma_block(y, xh, bl);
                tc::mma_block(y, xl, bh);
                split2(y[0], y[1], xh[0], xl[0]);
                split2(y[2], y[3], xh[1], xl[1]);
                split2(y[4], y[5], xh[2], xl[2]);
                split2(y[6], y[7], xh[3], xl[3]);
                put_block(xh, thi, w, j);
                put_block(xl, tlo, w, j);
                if (d < 3) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) fh[d][e] = xh[e], fl[d][e] = xl[e];
                }
            }
            // row w of M T, in place of M
            uint32_t fm[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k <= w) tc::ldm_x4(fm[k], block_addr(mt, w, k));
            named_sync(1 + hf);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > w) break;
                float acc[8] = {};
#pragma unroll
                for (int k = j; k < 4; ++k) {
                    if (k > w) break;
                    uint32_t bh[4];
                    tc::ldm_x4_trans(bh, block_addr(thi, k, j));
                    tc::mma_block(acc, fm[k], bh);
                }
                const uint32_t f[4] = {pack2(acc[0], acc[1]), pack2(acc[2], acc[3]), pack2(acc[4], acc[5]),
                                       pack2(acc[6], acc[7])};
                put_block(f, mt, w, j);
            }
            tc::fence_proxy_async_smem();
            tc::mbar_arrive(&bars[BAR_T_FULL]);
        }
    }
    __syncthreads();
    if (tid == 0 && *fail) atomicCAS(a.status, SSD_OK, SSD_ERR_TIMEOUT);
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int NH> cudaError_t launch_nh(const DeltaArgs &a, cudaStream_t stream) {
    DeltaTcParams p;
    p.a = a;
    bool ok = tma_map_heads(&p.mq, a.q, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&p.mk, a.k, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&p.mv, a.v, a.P, a.H, a.L, a.B, 32, kC, false);
    ok = ok && tma_map_heads(&p.my, a.y, a.P, a.H, a.L, a.B, 32, 32, false);
    if (!ok) return cudaErrorInvalidValue;
    p.pblocks = (int)((a.P + 127) / 128);
    p.units_per_b = (int)(NH == 2 ? a.H / 2 : a.H * p.pblocks);
    static DeviceOnce configured;
    int dev = 0;
    cudaError_t e = cudaSuccess;
    if (configured.pending(&dev, &e)) {
        e = cudaFuncSetAttribute(delta_chunk_tc<NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(NH));
        if (e != cudaSuccess) return e;
        configured.done(dev);
    } else if (e != cudaSuccess) {
        return e;
    }
    return launch_programmatic(delta_chunk_tc<NH>, dim3((unsigned)(a.B * p.units_per_b)), dim3(threads_of(NH)),
                               smem_bytes(NH), stream, p);
}

}  // namespace

bool delta_tc_supported(int io, int64_t L, int64_t P, int64_t N) {
    return io == IO_BF16 && L > 0 && P % 8 == 0 && N % 8 == 0 && N <= 128 && device_cc_major_cached() == 10;
}

cudaError_t launch_delta_tc(const DeltaArgs &a, cudaStream_t stream) {
    const bool pairs = a.P <= 64 && (a.H / a.G) % 2 == 0 && a.B * (a.H / 2) >= (int64_t)sm_count(152);
    return pairs ? launch_nh<2>(a, stream) : launch_nh<1>(a, stream);
}

}  // namespace ssd
