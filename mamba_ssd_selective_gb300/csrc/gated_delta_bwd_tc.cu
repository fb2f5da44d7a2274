// Backward of the gated delta rule on the tensor cores (the forward's algebra is
// in gated_delta_tc.cuh): bf16 inputs, chunks of 64 tokens, P <= 128, N <= 128.
//
// Four steps: T and M T of every chunk; the forward chain once more, which leaves
// the states S0 entering each chunk and w; the reverse chain below, which leaves dv
// and the cotangent E of the state leaving each chunk; then one block per (b, chunk,
// group) forms dq, dk, dg and dbeta. With E = dS1 of a chunk:
//     z  = beta exp(c_63 - c) K E^T,    dR = T^T z + (M T)^T dY,    dV = dR
//     dS0 = exp(c_63) E + (s exp(c) dY)^T Q - (exp(c) dR)^T K        (the E of the chunk before)
//     G_tj = s (dY_t . w_j) D_tj beta_j, j <= t      X_tj = -(dV_t . w_j) D_tj beta_j, j < t
//     dQ = s exp(c) dY S0 + G K
//     dK = beta exp(c_63 - c) w E - exp(c) dV S0 + G^T Q + (X + X^T) K
// (M T holds the factor s.) The decays' gradient needs no sums of its own: k_t and
// q_t stand beside exp(c_t) or exp(-c_t) wherever they occur, so with dc for the
// chunk's sums of g and dk = dk' + dk", dk' = X K - exp(c) dV S0 the part with exp(c_t):
//     dc_t = q_t . dq_t + k_t . dk'_t - k_t . dk"_t   (+ <S1, E> at the last token),
// dg_t is the sum of dc over the tokens from t on, and beta_t dbeta_t = dV_t . w_t. What a
// pair of tokens adds to dc at one it takes at the other, and what the update adds at
// the last token it takes at its own; both cancel in the sums because both sides
// come from the same rounded operands: <S1, E> is formed as
// exp(c_63) <S0, E> + sum_j beta_j exp(c_63 - c_j) w_j . (E k_j).
#include "gated_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

// ------------------------------------------------------------ reverse chain
// Laid out as the forward chain: a state row of E is one TMEM lane, NH heads of a
// group per CTA. Per chunk, from the last to the first:
//     X = E K^T                            (16 columns of K per product; E hi, E lo)
//     D = dY^T (M T) + z T                 (dY exact, M T hi + lo; z hi, z lo, T hi + lo)
//     E <- exp(c_63) E + (s exp(c) dY)^T Q - (exp(c) dR)^T K
// The products with dY need no E: dY^T (M T) runs under the conversion of E, and
// dY^T Q under that of z. All of E's terms keep hi + lo, so that its gradient of
// the initial state is as exact as the forward's state.
//
// TMEM (512 columns, gated_delta_columns.h): X 64 | D 64 | E float32 128 | operands 128:
// E hi 64, lo 64; z of each head hi 32, lo 32; exp(c) dR hi 32, lo 32 | dY^T of each
// head 32 | s exp(c) dY^T hi 32, lo 32.
//
// Warps: 0 loads; 1 products; 4-11 the chain's elementwise steps; 12-19 the
// operands of dY, and dv.
//
// Bound as the forward chain is; 107 us for the 2560 chunks of B2 L2048 H80.
namespace rev {
constexpr int kChainWarp0 = 4, kOutWarp0 = 12, kThreads = 640;
}  // namespace rev

struct ReverseParams {
    DeltaArgs a;
    CUtensorMap mq, mk, mdy, mdv;
    const uint8_t *tiles;   // kTilesBwd each
    const float *scal;
    const float *dfinal;    // may be null
    float *dinit;           // may be null
    __nv_bfloat16 *cot;     // [B][H][nc][P][N] E of each chunk
    __nv_bfloat16 *dv;
    int *flags;             // per chain
    float *carry;           // [B][H][P][N]
    Pieces pieces;
    int64_t nc;
    int units_per_b, pblocks;
};

namespace rev {
constexpr uint32_t kOffKQ = 0;             // 2 stages of 32 KB, as in the forward chain
constexpr uint32_t kOffDY = 65536;         // 2 stages of 16 KB: [32-row block][token][row]
constexpr uint32_t kOffDV = kOffDY + 32768;
constexpr uint32_t kOffT = kOffDV + 16384; // per head T hi, T lo, then per head M T hi, M T lo (8 KB each)
__host__ __device__ constexpr uint32_t off_scal(int NH) { return kOffT + NH * kTilesBwd; }
__host__ __device__ constexpr uint32_t off_bar(int NH) { return off_scal(NH) + 2 * NH * kScalBytes; }
enum {
    BAR_KQ_FULL = 0,   // [2]
    BAR_KQ_EMPTY = 2,  // [2]
    BAR_DY_FULL = 4,   // [2]
    BAR_DY_EMPTY = 6,  // [2] output warps
    BAR_SC_FULL = 8,   // [2]
    BAR_SC_EMPTY = 10, // [2] chain and output warps
    BAR_E_FULL = 12,   // [2] halves
    BAR_Z_FULL = 14,   // [2]
    BAR_R_FULL = 16,   // [2]
    BAR_T_FULL = 18,
    BAR_T_EMPTY,
    BAR_M_FULL,
    BAR_M_EMPTY,
    BAR_OP_FULL,       // the operands of dY
    BAR_OP_EMPTY,
    BAR_A_DONE,
    BAR_B_DONE,
    BAR_C_DONE,
    BAR_D_READ,        // the output warps have read D
    BAR_DRAIN,
    kBars
};
__host__ __device__ constexpr size_t smem_bytes(int NH) { return off_bar(NH) + kBars * 8 + 16 + 1024; }
}  // namespace rev

template <int NH, int PASS> __global__ void __launch_bounds__(rev::kThreads, 1)
delta_reverse_kernel(const __grid_constant__ ReverseParams prm) {
    using namespace rev;
    static_assert(smem_bytes(NH) <= 232448, "shared memory of one CTA");
    const DeltaArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = (int)a.P, N = (int)a.N;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sKQ = smem + kOffKQ, *sDY = smem + kOffDY, *sDV = smem + kOffDV, *sT = smem + kOffT;
    uint8_t *sM = sT + NH * 2 * kTile;
    float *scal = reinterpret_cast<float *>(smem + off_scal(NH));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + off_bar(NH));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);

    // as in the forward chain; Phi starts from the identity with dY = 0
    const int cut = PASS == FIND ? find_units(prm.pieces.n, prm.pblocks) : prm.pieces.n * prm.pblocks;
    int piece = (blockIdx.x % cut) / prm.pblocks, kind = (blockIdx.x % cut) % prm.pblocks;
    if (PASS == FIND) find_unit(blockIdx.x % cut, prm.pblocks, piece, kind);
    const bool phi = PASS == FIND && kind == prm.pblocks;
    const int R = phi ? N : P, row_warps = NH == 2 || R >= 128 ? 8 : 2 * ((R + 31) / 32);
    __shared__ Segments seg;
    // item k: its steps [c0, c1), step i being chunk nc - 1 - i, and where its rows are
    struct Item {
        int64_t b, len;
        int unit, piece, h0, prow0, grp, c0, c1, nc;
    };
    auto get = [&](int k) {
        Item m;
        if (PASS == WHOLE) {
            seg.item(k, (int)prm.nc, m.unit, m.c0, m.c1);
            m.b = m.unit / prm.units_per_b;
            const int un = m.unit % prm.units_per_b;
            m.h0 = NH == 2 ? 2 * un : un / prm.pblocks;
            m.prow0 = NH == 2 ? 0 : (un % prm.pblocks) * 128;
        } else {
            m.piece = piece;
            m.b = blockIdx.x / cut / a.H;
            m.h0 = (int)(blockIdx.x / cut % a.H);
            m.prow0 = phi ? 0 : kind * 128;
            m.c0 = m.piece * prm.pieces.chunks;
            m.c1 = m.c0 + prm.pieces.chunks;
        }
        m.grp = m.h0 / (int)(a.H / a.G);
        m.len = seq_len(a.seqlens, m.b, a.L);
        m.nc = (int)((m.len + kC - 1) / kC);
        m.c1 = imin(m.c1, m.nc);
        return m;
    };

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) {
            int count = 1;
            if (k == BAR_DY_EMPTY || k == BAR_DY_EMPTY + 1 || k == BAR_D_READ) count = row_warps;
            if (k == BAR_SC_EMPTY || k == BAR_SC_EMPTY + 1) count = 2 * row_warps;
            if ((k >= BAR_E_FULL && k < BAR_R_FULL + 2) || k == BAR_OP_FULL) count = 32 * row_warps;
            tc::mbar_init(bars + k, count);
        }
        tc::fence_mbar_init();
        *fail = 0;
        if (PASS == WHOLE) seg.set(a.B * prm.units_per_b, prm.nc);
    }
    if (warp == 1) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tX = tmem + rev_col::kX, tD = tmem + rev_col::kD, tE = tmem + rev_col::kE;
    const uint32_t tOp = tmem + rev_col::kOp, tY = tmem + rev_col::kY, tYe = tmem + rev_col::kYe;
    pdl_wait();
    const int items = PASS == WHOLE ? seg.items() : 1;

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            int n[4] = {0, 0, 0, 0};  // of K and Q with scalars, M T, dY, T
            int it = 0;
            for (int kk = 0; kk < items && !*fail; ++kk) {
            const Item m = get(kk);
            const int64_t b = m.b;
            const int h0 = m.h0;
            for (int i = m.c0; i < m.c1; ++i, ++it) {
                const int s = it & 1, c = m.nc - 1 - i;
                const uint32_t ph2 = ((it >> 1) & 1) ^ 1, ph = (it & 1) ^ 1;
                const int64_t item0 = (b * a.H + h0) * prm.nc + c;
                if (!wait_on(&bars[BAR_SC_EMPTY + s], ph2, fail) || !wait_on(&bars[BAR_KQ_EMPTY + s], ph2, fail)) break;
                uint64_t *bar = &bars[BAR_KQ_FULL + s];
                uint8_t *d = sKQ + s * 32768;
                tc::mbar_arrive_expect_tx(bar, 32768u);
                for (int k = 0; k < 2; ++k) {
                    tc::tma_load_4d(d + k * 16384, &prm.mq, bar, 64 * k, m.grp, c * kC, (int)b);
                    tc::tma_load_4d(d + k * 16384 + 8192, &prm.mk, bar, 64 * k, m.grp, c * kC, (int)b);
                }
                bar = &bars[BAR_SC_FULL + s];
                tc::mbar_arrive_expect_tx(bar, NH * kScalBytes);
                for (int hf = 0; hf < NH; ++hf)
                    tc::bulk_load(scal + (s * NH + hf) * kScalDecay, prm.scal + (item0 + hf * prm.nc) * kScal, kScalBytes, bar);
                n[0] = it + 1;
                if (!wait_on(&bars[BAR_DY_EMPTY + s], ph2, fail)) break;
                bar = &bars[BAR_DY_FULL + s];
                tc::mbar_arrive_expect_tx(bar, 16384u);
                for (int k = 0; k < 4; ++k) {
                    const int hh = NH == 2 ? h0 + (k >> 1) : h0;
                    const int p = NH == 2 ? 32 * (k & 1) : (phi ? 128 * prm.pblocks : m.prow0) + 32 * k;  // Phi: past P, zeros
                    tc::tma_load_4d(sDY + s * 16384 + k * 4096, &prm.mdy, bar, p, hh, c * kC, (int)b);
                }
                n[2] = it + 1;
                // single stages: a chunk's M T and T are free well before the next chunk's are due
                if (!wait_on(&bars[BAR_M_EMPTY], ph, fail)) break;
                tc::mbar_arrive_expect_tx(&bars[BAR_M_FULL], NH * 2 * kTile);
                for (int hf = 0; hf < NH; ++hf)
                    for (int k = 0; k < 2; ++k)
                        tc::bulk_load(sM + (2 * hf + k) * kTile, prm.tiles + (item0 + hf * prm.nc) * kTilesBwd + (2 * k + 1) * kTile,
                                      kTile, &bars[BAR_M_FULL]);
                n[1] = it + 1;
                if (!wait_on(&bars[BAR_T_EMPTY], ph, fail)) break;
                tc::mbar_arrive_expect_tx(&bars[BAR_T_FULL], NH * 2 * kTile);
                for (int hf = 0; hf < NH; ++hf)
                    for (int k = 0; k < 2; ++k)
                        tc::bulk_load(sT + (2 * hf + k) * kTile, prm.tiles + (item0 + hf * prm.nc) * kTilesBwd + 2 * k * kTile, kTile,
                                      &bars[BAR_T_FULL]);
                n[3] = it + 1;
            }
            }
            // no copy outlives the block, even where a wait gave up
            for (int k = imax(0, n[0] - 2); k < n[0]; ++k) {
                tc::mbar_wait(&bars[BAR_KQ_FULL + (k & 1)], (k >> 1) & 1, kWaitNs);
                tc::mbar_wait(&bars[BAR_SC_FULL + (k & 1)], (k >> 1) & 1, kWaitNs);
            }
            for (int k = imax(0, n[2] - 2); k < n[2]; ++k) tc::mbar_wait(&bars[BAR_DY_FULL + (k & 1)], (k >> 1) & 1, kWaitNs);
            if (n[1]) tc::mbar_wait(&bars[BAR_M_FULL], (n[1] - 1) & 1, kWaitNs);
            if (n[3]) tc::mbar_wait(&bars[BAR_T_FULL], (n[3] - 1) & 1, kWaitNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        const uint32_t one = tc::elect_one();
        const uint32_t idA = tc::idesc_bf16(128, 64, false, false), idB = tc::idesc_bf16(128, 64, false, true);
        const uint32_t idE = tc::idesc_bf16(128, N <= 64 ? 64 : 128, false, true);
        const uint64_t dT = tc::sdesc_sw128(tc::smem_u32(sT), 16, 1024), dM = tc::sdesc_sw128(tc::smem_u32(sM), 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(tc::smem_u32(sKQ) + 8192, 16, 1024);      // rows of K
        const uint64_t dQm = tc::sdesc_sw128(tc::smem_u32(sKQ), 16384, 1024);         // Q and K by columns
        int it = 0;
        for (int kk = 0; kk < items; ++kk) {
        const Item m = get(kk);
        const int64_t len = m.len;
        for (int i = m.c0; i < m.c1; ++i, ++it) {
            const int s = it & 1, c = m.nc - 1 - i;
            const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
            const uint64_t kr = dK + (uint64_t)(s * 2048), qm = dQm + (uint64_t)(s * 2048), km = qm + 512;
            wait_on(&bars[BAR_KQ_FULL + s], ph2, fail);
            __syncwarp();
            if ((int64_t)(c + 1) * kC > len && len < a.L) {  // tokens past the sequence's length
                for (int x = (int)(len - (int64_t)c * kC) * 8 + lane; x < kC * 8; x += 32)
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<uint4 *>(sKQ + s * 32768 + k * 8192)[x] = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
                __syncwarp();
            }
            // D = dY^T (M T)
            wait_on(&bars[BAR_M_FULL], ph, fail);
            wait_on(&bars[BAR_OP_FULL], ph, fail);
            if (it > 0) wait_on(&bars[BAR_D_READ], ph ^ 1, fail);
            __syncwarp();
            tc::tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < NH; ++hf)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma_bf16_ts_if(one, tD, tY + 32 * hf + 8 * (k & 3), dM + (1024 * hf + 512 * (k >> 2) + 128 * (k & 3)), idB,
                                       hf > 0 || k > 0);
            tc::mma_commit_if(one, &bars[BAR_M_EMPTY]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_E_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int pn = 0; pn < 2; ++pn)
                    if (pn == 0 || N > 64)
#pragma unroll
                        for (int k = half; k < 8; k += 2)
                            tc::mma_bf16_ts_if(one, tX, tOp + 64 * (k >> 2) + 32 * pn + 8 * (k & 3), kr + (1024 * pn + 2 * (k & 3)),
                                               idA, half > 0 || pn > 0 || k > 0);
            }
            tc::mma_commit_if(one, &bars[BAR_A_DONE]);
#pragma unroll
            for (int k = 0; k < 8; ++k)  // (s exp(c) dY)^T Q
                tc::mma_bf16_ts_if(one, tE, tYe + 8 * k, qm + 128 * (k & 3), idE, 1);
            tc::mma_commit_if(one, &bars[BAR_OP_EMPTY]);
            wait_on(&bars[BAR_T_FULL], ph, fail);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_Z_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < NH; ++hf) {
#pragma unroll
                    for (int k = half; k < 8; k += 2)  // z hi, z lo with T hi
                        tc::mma_bf16_ts_if(one, tD, tOp + 64 * hf + 8 * k, dT + (1024 * hf + 128 * (k & 3)), idB, 1);
#pragma unroll
                    for (int k = half; k < 4; k += 2)
                        tc::mma_bf16_ts_if(one, tD, tOp + 64 * hf + 8 * k, dT + (1024 * hf + 512 + 128 * k), idB, 1);
                }
            }
            tc::mma_commit_if(one, &bars[BAR_B_DONE]);
            tc::mma_commit_if(one, &bars[BAR_T_EMPTY]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_R_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int k = half; k < 8; k += 2)  // -(exp(c) dR)^T K
                    tc::mma_bf16_ts_if(one, tE, tOp + 8 * k, km + 128 * (k & 3), idE, 1);
            }
            tc::mma_commit_if(one, &bars[BAR_C_DONE]);
            tc::mma_commit_if(one, &bars[BAR_KQ_EMPTY + s]);
        }
        }
        tc::mma_commit_if(one, &bars[BAR_DRAIN]);
        tc::mbar_wait(&bars[BAR_DRAIN], 0, kWaitNs);
        __syncwarp();
    } else if (warp >= kChainWarp0 && warp < kOutWarp0) {
        // ---------------------------------------- elementwise steps of the chain
        const int cw = warp - kChainWarp0, q = cw & 3, ch = cw >> 2;
        const int hf = NH == 2 ? q >> 1 : 0;
        const uint32_t lq = (uint32_t)(32 * q) << 16;
        int it = 0;
        for (int kk = 0; kk < (2 * q < row_warps ? items : 0); ++kk) {
            const Item m = get(kk);
            const int64_t b = m.b;
            const int h = m.h0 + hf, p = (NH == 2 ? 32 * (q & 1) : m.prow0 + 32 * q) + lane;
            const int64_t bh = b * a.H + h, srow = (bh * a.P + p) * a.N;
            // 16 columns of E of chunk c: operands, scaled for the next accumulation, and kept for the gradients
            auto put_state = [&](const float (&v)[16], int c0, float eq, int c) {
                uint32_t hi[8], lo[8], sc[16];
                const uint64_t e2 = f2(eq, eq);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t x = f2(v[2 * k], v[2 * k + 1]);
                    float s0, s1;
                    split2(x, hi[k], lo[k]);
                    un2(mul2(x, e2), s0, s1);
                    sc[2 * k] = __float_as_uint(s0), sc[2 * k + 1] = __float_as_uint(s1);
                }
                tc::tmem_st8(tOp + lq + c0 / 2, hi);
                tc::tmem_st8(tOp + 64 + lq + c0 / 2, lo);
                tc::tmem_st16(tE + lq + c0, sc);
                if (PASS != FIND && p < P) {
                    uint4 *o = reinterpret_cast<uint4 *>(prm.cot + (((b * a.H + h) * prm.nc + c) * P + p) * N + c0);
                    if (c0 < N) o[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (c0 + 8 < N) o[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                }
            };
            auto get_state = [&](float (&v)[16], const float *row, int c0) {
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (row && p < R && c0 + k < N) x = __ldcg(reinterpret_cast<const float4 *>(row + c0 + k));
                    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
                }
                if (phi)
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = c0 + k == p ? 1.f : 0.f;
            };
            auto out_state = [&](const float (&v)[16], float *row, int c0) {
                if (p >= R || !row) return;
#pragma unroll
                for (int k = 0; k < 16; k += 4)
                    if (c0 + k < N) *reinterpret_cast<float4 *>(row + c0 + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            };
            auto row_of = [&](auto *states) { return states ? states + srow : nullptr; };
            if (m.c0 >= m.c1) {  // no token, or none left
                if (PASS != FIND && m.nc == 0 && m.c0 == 0)
                    for (int c0 = 64 * ch; c0 < 64 * ch + 64; c0 += 16) {
                        float v[16];
                        get_state(v, row_of(prm.dfinal), c0);
                        out_state(v, row_of(prm.dinit), c0);
                    }
                continue;
            }
            if (PASS == WHOLE && m.c0 > 0) flag_wait(prm.flags + m.unit, fail);
            const float *from = m.c0 == 0 ? row_of(prm.dfinal) : PASS == WHOLE ? row_of(prm.carry) : nullptr;
            if (PASS == PIECES) from = prm.pieces.in + ((bh * prm.pieces.n + m.piece) * P + p) * N;
            wait_on(&bars[BAR_SC_FULL + (it & 1)], (it >> 1) & 1, fail);
            const float eq0 = scal[((it & 1) * NH + hf) * kScalDecay + kScalEnd];
            __syncwarp();
#pragma unroll 1
            for (int k4 = 0; k4 < 4; ++k4) {
                const int c0 = 64 * ch + 16 * k4;
                float v[16];
                get_state(v, from, c0);
                put_state(v, c0, eq0, m.nc - 1 - m.c0);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars[BAR_E_FULL]);
            tc::mbar_arrive(&bars[BAR_E_FULL + 1]);
            for (int i = m.c0; i < m.c1; ++i, ++it) {
                const int s = it & 1, c = m.nc - 1 - i;
                const uint32_t ph = it & 1;
                const float *sc = scal + (s * NH + hf) * kScalDecay + 32 * ch;
                // z
                float4 f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = *reinterpret_cast<const float4 *>(sc + SC_BTAIL * kC + 4 * k);
                wait_on(&bars[BAR_A_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < 32; t0 += 16) {
                    float x[16];
                    tc::tmem_ld16(tX + lq + 32 * ch + t0, x);
                    tc::tmem_ld_wait();
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 e = f[t0 / 4 + k];
                        split2(mul2(f2(x[4 * k], x[4 * k + 1]), f2(e.x, e.y)), hi[2 * k], lo[2 * k]);
                        split2(mul2(f2(x[4 * k + 2], x[4 * k + 3]), f2(e.z, e.w)), hi[2 * k + 1], lo[2 * k + 1]);
                    }
                    tc::tmem_st8(tOp + lq + 64 * hf + 16 * ch + t0 / 2, hi);
                    tc::tmem_st8(tOp + lq + 64 * hf + 32 + 16 * ch + t0 / 2, lo);
                    if (NH == 2) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) hi[k] = 0u;
                        tc::tmem_st8(tOp + lq + 64 * (hf ^ 1) + 16 * ch + t0 / 2, hi);
                        tc::tmem_st8(tOp + lq + 64 * (hf ^ 1) + 32 + 16 * ch + t0 / 2, hi);
                    }
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars[BAR_Z_FULL + t0 / 16]);
                }
                // -exp(c) dR
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = *reinterpret_cast<const float4 *>(sc + SC_NEG * kC + 4 * k);
                wait_on(&bars[BAR_B_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < 32; t0 += 16) {
                    float x[16];
                    tc::tmem_ld16(tD + lq + 32 * ch + t0, x);
                    tc::tmem_ld_wait();
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 e = f[t0 / 4 + k];
                        split2(mul2(f2(x[4 * k], x[4 * k + 1]), f2(e.x, e.y)), hi[2 * k], lo[2 * k]);
                        split2(mul2(f2(x[4 * k + 2], x[4 * k + 3]), f2(e.z, e.w)), hi[2 * k + 1], lo[2 * k + 1]);
                    }
                    tc::tmem_st8(tOp + lq + 16 * ch + t0 / 2, hi);
                    tc::tmem_st8(tOp + lq + 32 + 16 * ch + t0 / 2, lo);
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars[BAR_R_FULL + t0 / 16]);
                }
                if (lane == 0) tc::mbar_arrive(&bars[BAR_SC_EMPTY + s]);
                // E of the chunk before
                const bool next = i + 1 < m.c1;
                if (next) wait_on(&bars[BAR_SC_FULL + (s ^ 1)], ((it + 1) >> 1) & 1, fail);
                const float eq = next ? scal[((s ^ 1) * NH + hf) * kScalDecay + kScalEnd] : 0.f;
                wait_on(&bars[BAR_C_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
                if (next) {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int c0 = 64 * ch + 16 * half;
                        float v0[16], v1[16];
                        tc::tmem_ld16(tE + lq + c0, v0);
                        tc::tmem_ld16(tE + lq + c0 + 32, v1);
                        tc::tmem_ld_wait();
                        put_state(v0, c0, eq, c - 1);
                        put_state(v1, c0 + 32, eq, c - 1);
                        tc::tmem_st_wait();
                        tc::tc_fence_before();
                        tc::mbar_arrive(&bars[BAR_E_FULL + half]);
                    }
                } else {
                    const bool last = PASS != FIND && m.c1 == m.nc;
                    float *to = PASS == FIND ? (phi ? prm.pieces.phi + ((bh * (prm.pieces.n - 1) + m.piece) * N + p) * N
                                                    : prm.pieces.psi + ((bh * (prm.pieces.n - 1) + m.piece) * P + p) * N)
                                : last       ? row_of(prm.dinit)
                                             : (PASS == WHOLE ? row_of(prm.carry) : nullptr);
#pragma unroll 1
                    for (int c0 = 64 * ch; c0 < 64 * ch + 64; c0 += 16) {
                        float v0[16];
                        tc::tmem_ld16(tE + lq + c0, v0);
                        tc::tmem_ld_wait();
                        out_state(v0, to, c0);
                    }
                    tc::tc_fence_before();
                    if (PASS == WHOLE && !last) {  // handed on to the next CTA
                        __threadfence();
                        asm volatile("bar.sync 1, %0;" ::"r"(32 * row_warps) : "memory");
                        if (cw == 0 && lane == 0) flag_set(prm.flags + m.unit);
                    }
                }
            }
        }
    } else if (warp >= kOutWarp0) {
        // -------------------------------------------- the operands of dY, and dv
        const int cw = warp - kOutWarp0, q = cw & 3, ch = cw >> 2;
        const int hf = NH == 2 ? q >> 1 : 0;
        const uint32_t lq = (uint32_t)(32 * q) << 16;
        if (2 * q < row_warps) {
            if (NH == 2) {  // zeros in the other head's operand, for good
                uint32_t z[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) z[k] = 0u;
                tc::tmem_st16(tY + 32 * (hf ^ 1) + lq + 16 * ch, z);
            }
            // the operands of dY for chunk c, the `it`-th of this CTA
            auto put_dy = [&](int it, int c, int64_t len) {
                const int s = it & 1;
                const float *sc = scal + (s * NH + hf) * kScalDecay + 32 * ch;
                const uint16_t *yt = reinterpret_cast<const uint16_t *>(sDY + s * 16384 + q * 4096 + ch * 2048) + lane;
                const int valid = (int)imin<int64_t>(32, len - (int64_t)c * kC - 32 * ch);
                wait_on(&bars[BAR_DY_FULL + s], (it >> 1) & 1, fail);
                wait_on(&bars[BAR_SC_FULL + s], (it >> 1) & 1, fail);
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const uint32_t y0 = 2 * k < valid ? yt[64 * k] : 0u, y1 = 2 * k + 1 < valid ? yt[64 * k + 32] : 0u;
                    y[k] = y0 | (y1 << 16);
                }
                if (it > 0) wait_on(&bars[BAR_OP_EMPTY], (it & 1) ^ 1, fail);
                __syncwarp();
                tc::tc_fence_after();
                tc::tmem_st16(tY + 32 * hf + lq + 16 * ch, y);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t v = y[8 * half + k];
                        const float2 eg = *reinterpret_cast<const float2 *>(sc + SC_EG * kC + 16 * half + 2 * k);
                        split2(mul2(mul2(f2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)), f2(eg.x, eg.y)),
                                    f2(a.scale, a.scale)),
                               hi[k], lo[k]);
                    }
                    tc::tmem_st8(tYe + lq + 16 * ch + 8 * half, hi);
                    tc::tmem_st8(tYe + 32 + lq + 16 * ch + 8 * half, lo);
                }
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::mbar_arrive(&bars[BAR_OP_FULL]);
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bars[BAR_DY_EMPTY + s]);
                    tc::mbar_arrive(&bars[BAR_SC_EMPTY + s]);
                }
            };
            uint16_t *vt = reinterpret_cast<uint16_t *>(sDV + q * 4096 + ch * 2048) + lane;
            int it = 0;
            for (int kk = 0; kk < items; ++kk) {
                const Item m = get(kk);
                const int h = m.h0 + hf, p32 = NH == 2 ? 32 * (q & 1) : m.prow0 + 32 * q, p = p32 + lane;
                if (m.c0 < m.c1) put_dy(it, m.nc - 1 - m.c0, m.len);
                for (int i = m.c0; i < m.c1; ++i, ++it) {
                    const int c = m.nc - 1 - i;
                    if (i + 1 < m.c1) put_dy(it + 1, c - 1, m.len);
                    wait_on(&bars[BAR_B_DONE], it & 1, fail);
                    __syncwarp();
                    tc::tc_fence_after();
                    if constexpr (PASS == FIND) {
                        if (lane == 0) tc::mbar_arrive(&bars[BAR_D_READ]);
                        __syncwarp();
                        continue;
                    }
                    float x[32];
                    tc::tmem_ld32(tD + lq + 32 * ch, x);
                    tc::tmem_ld_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive(&bars[BAR_D_READ]);
                        tc::bulk_wait_read_all();  // the previous chunk's dv has left the buffer
                    }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const uint32_t y = pack2(x[k], x[k + 1]);
                        vt[32 * k] = (uint16_t)y;
                        vt[32 * k + 32] = (uint16_t)(y >> 16);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && p32 < P) {
                        tc::tma_store_4d(&prm.mdv, vt, p32, h, c * kC + 32 * ch, (int)m.b);
                        tc::bulk_commit();
                    }
                }
                if (PASS != FIND && p < P && m.c0 == 0)  // zero past the last chunk
                    for (int64_t t = (int64_t)m.nc * kC + ch; t < a.L; t += 2)
                        prm.dv[((m.b * a.L + t) * a.H + h) * P + p] = __float2bfloat16_rn(0.f);
            }
            if (lane == 0) tc::bulk_wait_all();
        }
    }
    __syncthreads();
    if (tid == 0 && *fail) atomicCAS(a.status, SSD_OK, SSD_ERR_TIMEOUT);
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// --------------------------------------------------------------- gradients
// One block per (b, chunk, group); the group's heads one after the other add to
// dQ^T and dK^T in TMEM (lanes n, columns tokens), so that the sums over heads
// need no parts in memory and have a fixed order. All products take their
// operands from shared memory: S0, E, K and Q as loaded, read by columns; dY, dV
// and w scaled in place; G and X written by the threads.
//
// 104 KB of shared memory and 256 TMEM columns ([dY; dV] w^T, dQ^T, dk"^T, dk'^T): two
// blocks per SM (P <= 64), one computing while the other loads. G, X, dY, dV and w enter
// the products in bf16 and S0 and E come from memory in bf16; the sums are float32. Together
// these roundings take the error of dq and dk from 1.7e-3 (2-norm), which rounding them to
// bf16 makes alone, to 3.0e-3.
//
// Bound by shared memory and issue slots, which the operands of 40 products (6 KB each) and the
// element steps of a head both want: the sums with q and k and the stores of dq and dk
// as fragments instead of one lane a column took B4 L2048 H80 from 788 to 757 us; products
// issued earlier, under G and X, changed nothing.
namespace grad {
constexpr int kThreads = 288, kElem = 256;  // warps 0-7 elementwise, warp 8 loads and products
constexpr uint32_t kOffKQ = 0;              // 32 KB: two panels of 64 columns, each 64 rows of Q, then 64 of K
constexpr uint32_t kOffG = 32768, kOffX = kOffG + kTile;
constexpr uint32_t kOffPan = kOffX + kTile; // per 64 state rows: S0 16 KB, E 16 KB, [dY; dV] 16 KB, w 8 KB
constexpr uint32_t kPan = 16384 * 3 + kTile;
__host__ __device__ constexpr uint32_t off_scal(int NPAN) { return kOffPan + NPAN * kPan; }
__host__ __device__ constexpr uint32_t off_red(int NPAN) { return off_scal(NPAN) + kScal * 4; }
// sums: [4][64] of dc, [2][64] of dV.w, [64] the previous heads' dc, [64] dbeta where beta is tiny, [8] <S0, E>, [8] scratch
constexpr int kRed = 256 + 4 * kC + 16;
__host__ __device__ constexpr uint32_t columns(int NPAN) { return NPAN == 1 ? 256 : 512; }
__host__ __device__ constexpr uint32_t off_bar(int NPAN) { return off_red(NPAN) + kRed * 4; }
// dbeta is (dV . w) / beta, but dV = beta du is a bf16 operand: where beta is below this, du is formed without it, so that
// du of 1e-18 still keeps dV from falling below the normal numbers (at beta = 2^-120 dbeta was off by 1.3e-2, at 2^-126 by half)
constexpr float kTinyBeta = 0x1p-64f;
enum { BAR_FULL, BAR_READY, BAR_G_DONE, BAR_P_FULL, BAR_DONE, kBars };
__host__ __device__ constexpr size_t smem_bytes(int NPAN) { return off_bar(NPAN) + kBars * 8 + 16 + 1024; }
}  // namespace grad

struct GradParams {
    DeltaArgs a;
    CUtensorMap mq, mk, ms, me, mdy, mdv, mw, mdq, mdk;
    const float *scal;
    const __nv_bfloat16 *w;
    __nv_bfloat16 *dq, *dk, *dg, *dbeta;
    int64_t nc;
};

__device__ __forceinline__ void elem_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// One step of a sum over the lanes of equal lane % 4 that leaves value lane / 4 of eight to each: lanes 4 O apart
// exchange half of their 2 O values.
template <int O> __device__ __forceinline__ void fold(float (&x)[8], int lane) {
    const bool up = lane & (4 * O);
#pragma unroll
    for (int k = 0; k < O; ++k) {
        const float send = up ? x[k] : x[k + O], keep = up ? x[k + O] : x[k];
        x[k] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * O);
    }
}

// 8 bf16 times f, rounded
__device__ __forceinline__ uint4 scaled8(uint4 v, float f) {
    uint32_t o[4] = {v.x, v.y, v.z, v.w};
    const uint64_t f22 = f2(f, f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float x, y;
        un2(mul2(f2(__uint_as_float(o[k] << 16), __uint_as_float(o[k] & 0xffff0000u)), f22), x, y);
        o[k] = pack2(x, y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// sum of the products of 8 bf16 pairs
__device__ __forceinline__ float dot8(uint4 x, uint4 y, float acc) {
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        acc = fmaf(__uint_as_float(xs[k] << 16), __uint_as_float(ys[k] << 16), acc);
        acc = fmaf(__uint_as_float(xs[k] & 0xffff0000u), __uint_as_float(ys[k] & 0xffff0000u), acc);
    }
    return acc;
}

template <int NPAN> __global__ void __launch_bounds__(grad::kThreads, NPAN == 1 ? 2 : 1)
delta_grad_kernel(const __grid_constant__ GradParams prm) {
    using namespace grad;
    static_assert(smem_bytes(1) <= 115712 && smem_bytes(2) <= 232448, "shared memory of two blocks, of one");
    const DeltaArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = (int)a.P, N = (int)a.N, H = (int)a.H, G = (int)a.G, r = H / G;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sKQ = smem + kOffKQ, *sG = smem + kOffG, *sX = smem + kOffX, *sPan = smem + kOffPan;
    float *sc = reinterpret_cast<float *>(smem + off_scal(NPAN));
    float *red = reinterpret_cast<float *>(smem + off_red(NPAN));
    float *r_qk = red, *r_vw = red + 256, *prev = r_vw + 2 * kC, *dbz = prev + kC, *r_se = dbz + kC;
    float *scratch = r_se + 8;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + off_bar(NPAN));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int grp = (int)(blockIdx.x % G);
    const int64_t bc = blockIdx.x / G, c = bc % prm.nc, b = bc / prm.nc, t0 = c * kC;

    if (tid == 0) {
        for (int k = 0; k < kBars; ++k) tc::mbar_init(bars + k, k == BAR_READY || k == BAR_P_FULL ? kElem : 1);
        tc::fence_mbar_init();
        *fail = 0;
    }
    if (warp == 8) {
        tc::tmem_alloc(tmem_slot, columns(NPAN));
        tc::tmem_relinquish();
    }
    if (tid < kC) prev[tid] = 0.f;
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot, tG = tmem, tQ = tmem + 64, tK = tmem + 128, tR = tmem + 192;
    pdl_wait();
    const int64_t len = seq_len(a.seqlens, b, a.L);
    const int rows = (int)imin<int64_t>(kC, a.L - t0);                              // of the outputs
    const int valid = (int)imax<int64_t>(0, imin<int64_t>(kC, len - t0));           // with a token
    const int heads = valid > 0 ? r : 0;

    if (warp == 8) {
        // -------------------------------------------------- loads and products
        const uint32_t one = tc::elect_one();
        const uint32_t idG = tc::idesc_bf16(128, 64, false, false), idK = tc::idesc_bf16(128, 64, true, false);
        const uint32_t idM = tc::idesc_bf16(128, 64, true, true);
        const uint64_t dS = tc::sdesc_sw128(tc::smem_u32(sPan), 8192, 1024);            // S0, and E, by columns
        const uint64_t dP = tc::sdesc_sw128(tc::smem_u32(sPan), 16, 1024);              // tiles by rows
        const uint64_t dQm = tc::sdesc_sw128(tc::smem_u32(sKQ), 16384, 1024), dKm = dQm + 512;
        const uint64_t dKQ = tc::sdesc_sw128(tc::smem_u32(sKQ), 16, 1024);
        const uint64_t dGr = tc::sdesc_sw128(tc::smem_u32(sG), 16, 1024), dXr = tc::sdesc_sw128(tc::smem_u32(sX), 16, 1024);
        for (int i = 0; i < heads; ++i) {
            const int h = grp * r + i;
            const uint32_t ph = i & 1;
            if (i > 0) wait_on(&bars[BAR_DONE], ph ^ 1, fail);
            __syncwarp();
            if (one) {
                uint64_t *bar = &bars[BAR_FULL];
                tc::mbar_arrive_expect_tx(bar, (i ? 0u : 32768u) + NPAN * kPan + kScal * 4);
                if (i == 0)
                    for (int k = 0; k < 2; ++k) {
                        tc::tma_load_4d(sKQ + k * 16384, &prm.mq, bar, 64 * k, grp, (int)t0, (int)b);
                        tc::tma_load_4d(sKQ + k * 16384 + 8192, &prm.mk, bar, 64 * k, grp, (int)t0, (int)b);
                    }
                const int64_t bh = b * H + h, item = bh * prm.nc + c;
                tc::bulk_load(sc, prm.scal + item * kScal, kScal * 4, bar);
                for (int pn = 0; pn < NPAN; ++pn) {
                    uint8_t *d = sPan + pn * kPan;
                    for (int k = 0; k < 2; ++k) {
                        tc::tma_load_4d(d + k * 8192, &prm.ms, bar, 64 * k, 0, 64 * pn, (int)(bh * (prm.nc + 1) + c));
                        tc::tma_load_4d(d + 16384 + k * 8192, &prm.me, bar, 64 * k, 0, 64 * pn, (int)item);
                    }
                    tc::tma_load_4d(d + 32768, &prm.mdy, bar, 64 * pn, h, (int)t0, (int)b);
                    tc::tma_load_4d(d + 40960, &prm.mdv, bar, 64 * pn, h, (int)t0, (int)b);
                    tc::tma_load_4d(d + 49152, &prm.mw, bar, 64 * pn, h, (int)t0, (int)b);
                }
            }
            __syncwarp();
            wait_on(&bars[BAR_FULL], ph, fail);
            wait_on(&bars[BAR_READY], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
#pragma unroll
            for (int pn = 0; pn < NPAN; ++pn)  // [dY; dV] w^T
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc::mma_bf16_if(one, tG, dP + (pn * (kPan / 16) + 2048 + 2 * k), dP + (pn * (kPan / 16) + 3072 + 2 * k), idG,
                                    pn > 0 || k > 0);
            tc::mma_commit_if(one, &bars[BAR_G_DONE]);
            wait_on(&bars[BAR_P_FULL], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
#pragma unroll
            for (int pn = 0; pn < NPAN; ++pn) {
                const uint32_t o = pn * (kPan / 16);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    tc::mma_bf16_if(one, tQ, dS + (o + 128 * k), dP + (o + 2048 + 2 * k), idK, i > 0 || pn > 0 || k > 0);  // S0, dY
                    tc::mma_bf16_if(one, tK, dS + (o + 1024 + 128 * k), dP + (o + 3072 + 2 * k), idK, i > 0 || pn > 0 || k > 0);  // E, w
                    tc::mma_bf16_if(one, tR, dS + (o + 128 * k), dP + (o + 2560 + 2 * k), idK, i > 0 || pn > 0 || k > 0);  // S0, dV
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                tc::mma_bf16_if(one, tQ, dKm + 128 * k, dGr + 2 * k, idK, 1);    // G K
                tc::mma_bf16_if(one, tK, dQm + 128 * k, dGr + 128 * k, idM, 1);  // G^T Q
                tc::mma_bf16_if(one, tR, dKm + 128 * k, dXr + 2 * k, idK, 1);    // X K
                tc::mma_bf16_if(one, tK, dKm + 128 * k, dXr + 128 * k, idM, 1);  // X^T K
            }
            // K E^T of each panel, where [dY; dV] w^T was (and behind the others)
#pragma unroll
            for (int pn = 0; pn < NPAN; ++pn)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma_bf16_if(one, tG + 256 * pn, dKQ + (1024 * (k >> 2) + 2 * (k & 3)),
                                    dP + (pn * (kPan / 16) + 1024 + 512 * (k >> 2) + 2 * (k & 3)), idG, k > 0);
            tc::mma_commit_if(one, &bars[BAR_DONE]);
        }
        if (heads > 0) {  // nothing in flight outlives the block, even where a wait gave up
            tc::mbar_wait(&bars[BAR_FULL], (heads - 1) & 1, kWaitNs);
            tc::mbar_wait(&bars[BAR_DONE], (heads - 1) & 1, kWaitNs);
        }
        __syncwarp();
    } else {
        const int wq = warp & 3, half = warp >> 2;
        const uint32_t lq = (uint32_t)(32 * wq) << 16;
        const bool is_v = wq >= 2;                       // rows of dV: X; rows of dY: G
        const int t = 32 * (wq & 1) + lane;
        for (int i = 0; i < heads; ++i) {
            const int h = grp * r + i;
            const uint32_t ph = i & 1;
            wait_on(&bars[BAR_FULL], ph, fail);
            __syncwarp();
            if (valid < kC && a.seqlens) {  // dY past the length
                for (int x = tid; x < (kC - valid) * 8; x += kElem)
                    for (int pn = 0; pn < NPAN; ++pn)
                        reinterpret_cast<uint4 *>(sPan + pn * kPan + 32768 + valid * 128)[x] = make_uint4(0, 0, 0, 0);
                if (i == 0)  // and K and Q
                    for (int x = tid; x < (kC - valid) * 8; x += kElem)
                        for (int k = 0; k < 4; ++k)
                            reinterpret_cast<uint4 *>(sKQ + k * 8192 + valid * 128)[x] = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
                elem_sync();
            }
            tc::mbar_arrive(&bars[BAR_READY]);
            // under the product: half a row each of dY, or of dV and w, scaled in registers (to be stored over the
            // tiles once the product has read them), dV . w, and <S0, E>, whose tiles have the same layout
            uint4 r1[NPAN][4], r2[NPAN][4];
            {
                const float f1 = is_v ? sc[SC_NEG * kC + t] : sc[SC_EG * kC + t] * a.scale, f2s = sc[SC_BTAIL * kC + t];
                float dot = 0.f;
#pragma unroll
                for (int pn = 0; pn < NPAN; ++pn) {
                    const uint8_t *pan = sPan + pn * kPan;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t o = piece(t, 4 * half + k);
                        const uint4 v = *reinterpret_cast<const uint4 *>(pan + 32768 + (is_v ? kTile : 0) + o);
                        r1[pn][k] = scaled8(v, f1);
                        if (is_v) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(pan + 49152 + o);
                            dot = dot8(v, u, dot);
                            r2[pn][k] = scaled8(u, f2s);
                        } else {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint8_t *at = pan + ((t + 64 * half) + 128 * (2 * k + e)) * 16;
                                dot = dot8(*reinterpret_cast<const uint4 *>(at), *reinterpret_cast<const uint4 *>(at + 16384), dot);
                            }
                        }
                    }
                }
                if (is_v) {
                    r_vw[half * kC + t] = dot;
                } else {
                    dot = warp_sum(dot);
                    if (lane == 0) r_se[(warp & 1) + 2 * half] = dot;
                }
            }
            wait_on(&bars[BAR_G_DONE], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
            const float *hi = sc + kScalDecay, *rowf = hi + kC, *inv = rowf + kC;
            {
                const float hi_t = hi[t];
                // tokens whose beta is too small to divide by: dbeta_j = w_j . du_j with du formed anew
                const uint32_t z0 = __ballot_sync(0xffffffffu, lane < valid && fabsf(sc[SC_BETA * kC + lane]) < kTinyBeta);
                const uint32_t z1 = __ballot_sync(0xffffffffu, lane + 32 < valid && fabsf(sc[SC_BETA * kC + 32 + lane]) < kTinyBeta);
                uint64_t zero = (uint64_t)z1 << 32 | z0;
#pragma unroll 1
                while (zero) {
                    const int j = __ffsll((long long)zero) - 1;
                    zero &= zero - 1;
                    float val = 0.f, y[8];
                    tc::tmem_ld8(tG + lq + (j & 56), y);
                    tc::tmem_ld_wait();
                    if ((j >> 5) == half && (is_v ? t > j : t >= j)) {
                        float kd = 0.f;  // q_t . k_j or k_t . k_j
                        for (int pc = 0; pc < 16; ++pc) {
                            const uint8_t *pan = sKQ + (pc >> 3) * 16384;
                            kd = dot8(*reinterpret_cast<const uint4 *>(pan + (is_v ? 8192 : 0) + piece(t, pc & 7)),
                                      *reinterpret_cast<const uint4 *>(pan + 8192 + piece(j, pc & 7)), kd);
                        }
                        float g = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) g = k == (j & 7) ? y[k] : g;
                        val = g * kd * tc::ex2(hi_t - hi[j]) * (is_v ? -1.f : a.scale);
                    }
                    // exp(c_63 - c_j) w_j . (E k_j): row tid & 63 of each panel, a quarter of the columns
                    const float tail = tc::ex2(hi[kC - 1] - hi[j]);
                    for (int pn = 0; pn < NPAN; ++pn) {
                        const int pr = tid & 63, qd = tid >> 6;
                        if (64 * pn + pr >= P) continue;
                        float ek = 0.f;
                        for (int pc = 4 * qd; pc < 4 * qd + 4; ++pc)
                            ek = dot8(*reinterpret_cast<const uint4 *>(sPan + pn * kPan + 16384 + (pc >> 3) * 8192 + piece(pr, pc & 7)),
                                      *reinterpret_cast<const uint4 *>(sKQ + 8192 + (pc >> 3) * 16384 + piece(j, pc & 7)), ek);
                        val += tail * ek * to_f32(prm.w[((b * a.L + t0 + j) * H + h) * P + 64 * pn + pr]);
                    }
                    val = warp_sum(val);
                    if (lane == 0) scratch[warp] = val;
                    elem_sync();
                    if (tid == 0) {
                        float s = 0.f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) s += scratch[k];
                        dbz[j] = s;
                    }
                    elem_sync();
                }
                float x[32];
                tc::tmem_ld32(tG + lq + 32 * half, x);
                tc::tmem_ld_wait();
                const float rf = rowf[t] * (is_v ? -1.f : a.scale);
                const int last = (is_v ? t - 1 : t) - 32 * half;
                uint8_t *d = is_v ? sX : sG;
                const uint64_t rf2 = f2(rf, rf), ht2 = f2(hi_t, hi_t), m1 = f2(-1.f, -1.f);
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 h4 = *reinterpret_cast<const float4 *>(hi + 32 * half + k + e);
                        const float4 f4 = *reinterpret_cast<const float4 *>(inv + 32 * half + k + e);
                        float e0, e1, e2, e3;
                        un2(fma2(f2(h4.x, h4.y), m1, ht2), e0, e1);
                        un2(fma2(f2(h4.z, h4.w), m1, ht2), e2, e3);
                        // above the diagonal the exponent could overflow
                        e0 = k + e <= last ? tc::ex2(e0) : 0.f, e1 = k + e + 1 <= last ? tc::ex2(e1) : 0.f;
                        e2 = k + e + 2 <= last ? tc::ex2(e2) : 0.f, e3 = k + e + 3 <= last ? tc::ex2(e3) : 0.f;
                        un2(mul2(mul2(f2(x[k + e], x[k + e + 1]), rf2), mul2(f2(e0, e1), f2(f4.x, f4.y))), e0, e1);
                        un2(mul2(mul2(f2(x[k + e + 2], x[k + e + 3]), rf2), mul2(f2(e2, e3), f2(f4.z, f4.w))), e2, e3);
                        o[e / 2] = pack2(e0, e1);
                        o[e / 2 + 1] = pack2(e2, e3);
                    }
                    *reinterpret_cast<uint4 *>(d + piece(t, 4 * half + k / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
#pragma unroll
            for (int pn = 0; pn < NPAN; ++pn)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint8_t *pan = sPan + pn * kPan + piece(t, 4 * half + k);
                    *reinterpret_cast<uint4 *>(pan + 32768 + (is_v ? kTile : 0)) = r1[pn][k];
                    if (is_v) *reinterpret_cast<uint4 *>(pan + 49152) = r2[pn][k];
                }
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            // dc over this and the previous heads
            float bl = 0.f, bh2 = 0.f, eq = 0.f;  // beta of this thread's tokens, exp(c_63), before the scalars are loaded anew
            if (warp == 0) bl = sc[SC_BETA * kC + 2 * lane], bh2 = sc[SC_BETA * kC + 2 * lane + 1], eq = sc[kScalEnd];
            tc::mbar_arrive(&bars[BAR_P_FULL]);
            wait_on(&bars[BAR_DONE], ph, fail);
            __syncwarp();
            tc::tc_fence_after();
            {
                float z = 0.f;
                if (is_v) {
#pragma unroll
                    for (int pn = 0; pn < NPAN; ++pn) {
                        float y[32];
                        tc::tmem_ld32(tG + 256 * pn + lq + 32 * half, y);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t u[4] = {r2[pn][k].x, r2[pn][k].y, r2[pn][k].z, r2[pn][k].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                z = fmaf(__uint_as_float(u[e] << 16), y[8 * k + 2 * e], z);
                                z = fmaf(__uint_as_float(u[e] & 0xffff0000u), y[8 * k + 2 * e + 1], z);
                            }
                        }
                    }
                }
                z = warp_sum(z);
                if (lane == 0) scratch[warp] = z;
            }
            {
                // As fragments: Q and K transposed by ldmatrix give every thread the values that its own stand beside.
                // Lanes 0-15 hold the addresses of the two blocks of 8 columns of Q, 16-31 of K.
                float x[8] = {};  // tokens 8 (v / 2) + 2 (lane % 4) + v % 2 of this half
                const uint32_t at = tc::smem_u32(sKQ) + (wq >> 1) * 16384 + (lane >> 4) * 8192;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float v[16], y[16], z[16];
                    const uint32_t lm = lq + (16u << 16) * m + 32 * half;
                    tc::tmem_ld_frag32(tQ + lm, v);
                    tc::tmem_ld_frag32(tK + lm, y);
                    tc::tmem_ld_frag32(tR + lm, z);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int tb = 0; tb < 4; ++tb) {
                        uint32_t qk[4];
                        tc::ldm_x4_trans(qk, at + piece(32 * half + 8 * tb + (lane & 7), 4 * (wq & 1) + 2 * m + ((lane >> 3) & 1)));
#pragma unroll
                        for (int r8 = 0; r8 < 2; ++r8)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int i4 = 4 * tb + 2 * r8 + e;
                                const float qv = __uint_as_float(e ? qk[r8] & 0xffff0000u : qk[r8] << 16);
                                const float kv = __uint_as_float(e ? qk[2 + r8] & 0xffff0000u : qk[2 + r8] << 16);
                                x[2 * tb + e] = fmaf(qv, v[i4], fmaf(kv, z[i4] - y[i4], x[2 * tb + e]));
                            }
                    }
                }
                tc::tc_fence_before();
                fold<4>(x, lane);
                fold<2>(x, lane);
                fold<1>(x, lane);
                r_qk[wq * kC + 32 * half + 8 * (lane >> 3) + 2 * (lane & 3) + ((lane >> 2) & 1)] = x[0];
            }
            elem_sync();
            if (warp == 0) {
                float d[2], vw[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tt = 2 * lane + e;
                    const float cum = (r_qk[tt] + r_qk[kC + tt]) + (r_qk[2 * kC + tt] + r_qk[3 * kC + tt]);
                    d[e] = cum - prev[tt];
                    prev[tt] = cum;
                    vw[e] = r_vw[tt] + r_vw[kC + tt];
                }
                float se = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) se += r_se[k];
                se *= eq;
#pragma unroll
                for (int k = 0; k < 8; ++k) se += scratch[k];
                float sum = d[0] + d[1];  // suffix sums over the tokens
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float u = __shfl_down_sync(0xffffffffu, sum, o);
                    if (lane + o < 32) sum += u;
                }
                const float be[2] = {bl, bh2};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tt = 2 * lane + e;
                    if (tt >= rows) continue;
                    const int64_t at = (b * a.L + t0 + tt) * H + h;
                    const float dg = (e ? sum - d[0] : sum) + se, db = fabsf(be[e]) < kTinyBeta ? dbz[tt] : vw[e] / be[e];
                    // the first decay scales a zero state where there is no other: the sums leave only their rounding there
                    const bool felt = tt < valid && (t0 + tt > 0 || a.init);
                    prm.dg[at] = __float2bfloat16_rn(felt ? dg : 0.f);
                    prm.dbeta[at] = __float2bfloat16_rn(tt < valid ? db : 0.f);
                }
            }
            elem_sync();  // the sums' space is free again
        }
        if (heads > 0) {
            // [64 tokens][64 columns] tiles (128-byte swizzle) in the panels' space, stored by TMA: the sums as fragments,
            // transposed by stmatrix
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const uint32_t tile = tc::smem_u32(sPan) + which * 16384 + (wq >> 1) * 8192;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float x[16];
                    const uint32_t lm = lq + (16u << 16) * m + 32 * half;
                    tc::tmem_ld_frag32((which ? tK : tQ) + lm, x);
                    if (which) {
                        float y[16];
                        tc::tmem_ld_frag32(tR + lm, y);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] += y[k];
                    }
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int tb = 0; tb < 4; tb += 2) {
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t8 = 32 * half + 8 * (tb + (k >> 1)) + 2 * (lane & 3), i4 = 4 * tb + 2 * k;
                            o[k] = pack2(t8 < valid ? x[i4] : 0.f, t8 + 1 < valid ? x[i4 + 1] : 0.f);
                        }
                        tc::stm_x4_trans(tile + piece(32 * half + 8 * (tb + (lane >> 4)) + (lane & 7),
                                                      4 * (wq & 1) + 2 * m + ((lane >> 3) & 1)), o);
                    }
                }
            }
            tc::tc_fence_before();
            tc::fence_proxy_async_smem();
            elem_sync();
            if (tid == 0) {
                for (int k = 0; k < (N > 64 ? 2 : 1); ++k) {
                    tc::tma_store_4d(&prm.mdq, sPan + k * 8192, 64 * k, grp, (int)t0, (int)b);
                    tc::tma_store_4d(&prm.mdk, sPan + 16384 + k * 8192, 64 * k, grp, (int)t0, (int)b);
                }
                tc::bulk_commit();
                tc::bulk_wait_read_all();
            }
        } else {  // no token here
            for (int x = tid; x < rows * N; x += kElem) {
                const int64_t at = ((b * a.L + t0 + x / N) * G + grp) * N + x % N;
                prm.dq[at] = prm.dk[at] = __float2bfloat16_rn(0.f);
            }
            for (int x = tid; x < rows * r; x += kElem) {
                const int64_t at = (b * a.L + t0 + x / r) * H + grp * r + x % r;
                prm.dg[at] = prm.dbeta[at] = __float2bfloat16_rn(0.f);
            }
        }
    }
    __syncthreads();
    if (tid == 0 && *fail) atomicCAS(a.status, SSD_OK, SSD_ERR_TIMEOUT);
    if (warp == 8) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, columns(NPAN));
    }
}

template <int NH, int PASS> cudaError_t launch_reverse(ReverseParams &p, cudaStream_t stream) {
    const DeltaArgs &a = p.a;
    p.pblocks = (int)row_blocks(a.P);
    p.units_per_b = (int)(NH == 2 ? a.H / 2 : a.H * p.pblocks);
    static DeviceOnce configured;
    int dev = 0;
    cudaError_t e = cudaSuccess;
    if (configured.pending(&dev, &e)) {
        e = cudaFuncSetAttribute(delta_reverse_kernel<NH, PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)rev::smem_bytes(NH));
        if (e != cudaSuccess) return e;
        configured.done(dev);
    } else if (e != cudaSuccess) {
        return e;
    }
    if (PASS != WHOLE) {
        const int64_t grid = a.B * a.H * (PASS == FIND ? find_units(p.pieces.n, p.pblocks) : p.pieces.n * p.pblocks);
        return launch_programmatic(delta_reverse_kernel<NH, PASS>, dim3((unsigned)grid), dim3(rev::kThreads),
                                   rev::smem_bytes(NH), stream, p);
    }
    return launch_chains(delta_reverse_kernel<NH, PASS>, p, a.B * p.units_per_b, p.nc, rev::kThreads, rev::smem_bytes(NH), stream);
}

template <int NPAN> cudaError_t launch_grad(const GradParams &p, cudaStream_t stream) {
    static DeviceOnce configured;
    int dev = 0;
    cudaError_t e = cudaSuccess;
    if (configured.pending(&dev, &e)) {
        e = cudaFuncSetAttribute(delta_grad_kernel<NPAN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)grad::smem_bytes(NPAN));
        if (e != cudaSuccess) return e;
        configured.done(dev);
    } else if (e != cudaSuccess) {
        return e;
    }
    return launch_programmatic(delta_grad_kernel<NPAN>, dim3((unsigned)(p.a.B * p.nc * p.a.G)), dim3(grad::kThreads),
                               grad::smem_bytes(NPAN), stream, p);
}

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

struct BwdWs {
    size_t tiles, scal, flags, carry, pieces, states, cot, w, total;
};
BwdWs bwd_ws(int64_t B, int64_t L, int64_t H, int64_t P, int64_t N) {
    const size_t nc = (size_t)((L + kC - 1) / kC), items = (size_t)(B * H) * nc;
    BwdWs s{};
    s.tiles = 256;
    s.scal = s.tiles + items * kTilesBwd;
    s.flags = s.scal + up256(items * kScal * 4);
    s.carry = s.flags + up256((size_t)(B * H * row_blocks(P)) * 8);
    s.pieces = s.carry + up256((size_t)(B * H * P * N) * 4);
    s.states = s.pieces + up256(plan_pieces(B, H, P, (int64_t)nc, true).bytes(B * H, P, N));
    s.cot = s.states + up256((items + (size_t)(B * H)) * P * N * 2);
    s.w = s.cot + up256(items * P * N * 2);
    s.total = s.w + up256((size_t)(B * L * H * P) * 2);
    return s;
}

}  // namespace
}  // namespace delta

// The recurrent backward against these, N 128: 31 us and 38 for 12 tokens of 4 heads with P 128, 30 and 34
// for 4 tokens of 24 heads with P 64, but 36 and 34 for 8, and 66 and 35 for one token of 80 heads.
bool delta_bwd_tc_supported(int io, int64_t B, int64_t L, int64_t H, int64_t P, int64_t N) {
    return P <= 128 && B * H * ((L + delta::kC - 1) / delta::kC + 1) <= 0x7fffffffLL && delta::tc_takes(io, B, L, H, P, N, 512);
}

size_t delta_bwd_tc_workspace(int64_t B, int64_t L, int64_t H, int64_t P, int64_t N) { return delta::bwd_ws(B, L, H, P, N).total; }

cudaError_t launch_delta_bwd_tc(const DeltaBwdArgs &args, void *workspace, cudaStream_t stream) {
    using namespace delta;
    const DeltaArgs &a = args.f;
    const BwdWs s = bwd_ws(a.B, a.L, a.H, a.P, a.N);
    uint8_t *base = static_cast<uint8_t *>(workspace);
    auto bf = [&](size_t o) { return reinterpret_cast<__nv_bfloat16 *>(base + o); };
    PrepArgs p;
    p.a = a;
    p.a.y = nullptr;
    p.a.final_state = nullptr;
    p.nc = (a.L + kC - 1) / kC;
    p.tiles = base + s.tiles;
    p.scal = reinterpret_cast<float *>(base + s.scal);
    p.tile_bytes = kTilesBwd;
    p.flags = reinterpret_cast<int *>(base + s.flags);
    p.carry = reinterpret_cast<float *>(base + s.carry);
    p.pieces = plan_pieces(a.B, a.H, a.P, p.nc, true);
    p.pieces.carve(base + s.pieces, a.B * a.H, a.P, a.N);
    cudaError_t e = launch_prep(p, stream);
    if (e == cudaSuccess) e = launch_chain(p, bf(s.states), bf(s.w), stream);
    if (e != cudaSuccess) return e;

    ReverseParams rp;
    rp.a = p.a;
    bool ok = tma_map_heads(&rp.mq, a.q, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&rp.mk, a.k, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&rp.mdy, args.dy, a.P, a.H, a.L, a.B, 32, kC, false);
    ok = ok && tma_map_heads(&rp.mdv, args.dv, a.P, a.H, a.L, a.B, 32, 32, false);
    if (!ok) return cudaErrorInvalidValue;
    rp.tiles = p.tiles;
    rp.scal = p.scal;
    rp.dfinal = args.dfinal;
    rp.dinit = args.dinit;
    rp.cot = bf(s.cot);
    rp.dv = static_cast<__nv_bfloat16 *>(args.dv);
    rp.flags = p.flags + a.B * a.H * row_blocks(a.P);
    rp.carry = p.carry;
    rp.nc = p.nc;
    rp.pieces = p.pieces;
    if (p.pieces.n > 1) {
        e = launch_reverse<1, FIND>(rp, stream);
        if (e == cudaSuccess) e = launch_combine(p.pieces, args.dfinal, a.B * a.H, a.P, a.N, stream);
        if (e == cudaSuccess) e = launch_reverse<1, PIECES>(rp, stream);
    } else {
        e = pair_heads(a) ? launch_reverse<2, WHOLE>(rp, stream) : launch_reverse<1, WHOLE>(rp, stream);
    }
    if (e != cudaSuccess) return e;

    GradParams gp;
    gp.a = p.a;
    gp.mq = rp.mq;
    gp.mk = rp.mk;
    ok = tma_map_heads(&gp.ms, bf(s.states), a.N, 1, a.P, a.B * a.H * (p.nc + 1), 64, 64, true);
    ok = ok && tma_map_heads(&gp.me, bf(s.cot), a.N, 1, a.P, a.B * a.H * p.nc, 64, 64, true);
    ok = ok && tma_map_heads(&gp.mdy, args.dy, a.P, a.H, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&gp.mdv, args.dv, a.P, a.H, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&gp.mw, bf(s.w), a.P, a.H, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&gp.mdq, args.dq, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&gp.mdk, args.dk, a.N, a.G, a.L, a.B, 64, kC, true);
    if (!ok) return cudaErrorInvalidValue;
    gp.scal = p.scal;
    gp.w = bf(s.w);
    gp.dq = static_cast<__nv_bfloat16 *>(args.dq);
    gp.dk = static_cast<__nv_bfloat16 *>(args.dk);
    gp.dg = static_cast<__nv_bfloat16 *>(args.dg);
    gp.dbeta = static_cast<__nv_bfloat16 *>(args.dbeta);
    gp.nc = p.nc;
    return a.P <= 64 ? launch_grad<1>(gp, stream) : launch_grad<2>(gp, stream);
}

}  // namespace ssd
