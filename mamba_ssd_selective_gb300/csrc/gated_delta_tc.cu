// The chain of chunks of the gated delta rule on the tensor cores (the algebra is
// in gated_delta_tc.cuh): bf16 inputs, chunks of 64 tokens, N <= 128, float32
// state in TMEM. T and M T come from delta_prep_kernel.
//
// Three products per chunk, each waiting for the one before, everything
// transposed, so that a row of the state is one TMEM lane:
//     [Q S0^T | K S0^T]^T = S0 [Q; K]^T              (M = 128 state rows, N = 128, K = N)
//     [w | M w]^T         = R^T [T; M T]^T           (N = 128, K = 64)
//     S1                  = exp(c_63) S0 + (exp(c_63 - c) beta w)^T K    (N = 128, K = 64)
// The A operands are written to TMEM by the threads that own the rows, so
// nothing but the products' barriers crosses threads on the chain. Each operand
// arrives in two halves, and the first half's products run under the second
// half's writing.
//
// A CTA owns 128 state rows that share keys: the 64 rows of two heads of one
// group (NH = 2: two T's, R of one head beside zeros for the other, so that both
// products add up in one accumulator), or up to 128 rows of one head (NH = 1).
//
// Precision: S, T, R and the update's operand enter the products as pairs hi + lo
// of bf16 (2^-17 of the value is lost; 3.5e-6 of the state in the 2-norm); K, Q and V are
// exact; M T, which only reaches y, is bf16: y's error is 2.3e-3, 1.7e-3 of it from
// rounding y itself.
//
// TMEM (512 columns, gated_delta_columns.h): Q S0^T | K S0^T | w | M w, 64 each; S float32 128;
// operands 128: S hi 64, lo 64; R of each head hi 32, lo 32; the update hi 32, lo 32, one after
// the other. w has columns of its own: its product begins when the first half of R is written, while
// the chain's warps still read the second half of K S0^T.
//
// Warps: 0 loads; 1 products; 4-11 the chain's elementwise steps (two warps per
// 32 rows, half of the tokens or columns each); 12-19 y (and w for the backward).
//
// Where there are more chains than SMs they are cut into equal segments (Segments),
// where there are few into pieces that run at once (Pieces).
//
// Bound by the latency of the chain. A product of 16 columns of K takes 64
// cycles whatever N, 36 of them a chunk (NH = 1); the rest is the elementwise steps
// between them: 4700 cycles a chunk, 5600 for two heads (NH = 2). Tensor pipe 40 % busy, HBM
// 38 %; 98 us for the 2560 chunks of B2 L2048 H80, 469 us the whole call of B8 L2048 H80.
//
// Every wait is bounded (2 s): a timeout raises a flag, after which no wait
// waits; the copies and products in flight are waited for (bounded too), and the
// status word records SSD_ERR_TIMEOUT.
#include "gated_delta_tc.cuh"

namespace ssd {
namespace delta {
namespace {

constexpr int kChainWarp0 = 4, kOutWarp0 = 12, kThreads = 640;

struct ChainParams {
    DeltaArgs a;
    CUtensorMap mq, mk, mv, my, mw;
    const uint8_t *tiles;
    const float *scal;
    uint32_t tile_bytes;
    __nv_bfloat16 *states;  // SAVE: [B][H][nc + 1][P][N] states entering each chunk, then the final one
    int *flags;             // per chain
    float *carry;           // [B][H][P][N]
    Pieces pieces;
    int64_t nc;
    int units_per_b;  // NH = 2: head pairs; NH = 1: heads times blocks of 128 rows
    int pblocks;      // NH = 1: ceil(P / 128)
};

// shared memory carve (bytes from the 1024-aligned base)
constexpr uint32_t kOffKQ = 0;            // 2 stages of 32 KB: two panels of 64 columns, each 64 rows of Q, then 64 of K
constexpr uint32_t kOffV = 65536;         // 2 stages of 16 KB: [32-row block][token][row], y in place
constexpr uint32_t kOffW = kOffV + 32768; // SAVE: w in the same layout
constexpr uint32_t kOffT = kOffW + 16384; // 2 stages of NH x 24 KB: T hi, M T, T lo
__host__ __device__ constexpr uint32_t off_scal(int NH) { return kOffT + 2 * NH * kTilesFwd; }
__host__ __device__ constexpr uint32_t off_bar(int NH) { return off_scal(NH) + 2 * NH * kScalBytes; }
enum {
    BAR_KQ_FULL = 0,   // [2]
    BAR_KQ_EMPTY = 2,  // [2] last product of the chunk
    BAR_V_FULL = 4,    // [2]
    BAR_V_EMPTY = 6,   // [2] y has left the tile
    BAR_T_FULL = 8,    // [2] tiles and scalars
    BAR_T_EMPTY = 10,  // [2] chain and output warps
    BAR_S_FULL = 12,   // [2] halves
    BAR_R_FULL = 14,   // [2]
    BAR_U_FULL = 16,   // [2]
    BAR_A_DONE = 18,
    BAR_B_DONE,
    BAR_C_DONE,
    BAR_O_READ,        // the output warps have read QS, w and M w
    BAR_DRAIN,
    kBars
};
__host__ __device__ constexpr size_t smem_bytes(int NH) { return off_bar(NH) + kBars * 8 + 16 + 1024; }

template <int NH, bool SAVE, int PASS> __global__ void __launch_bounds__(kThreads, 1)
delta_chain_kernel(const __grid_constant__ ChainParams prm) {
    static_assert(smem_bytes(NH) <= 232448, "shared memory of one CTA");
    const DeltaArgs &a = prm.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = (int)a.P, N = (int)a.N;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sKQ = smem + kOffKQ, *sV = smem + kOffV, *sW = smem + kOffW, *sT = smem + kOffT;
    float *scal = reinterpret_cast<float *>(smem + off_scal(NH));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + off_bar(NH));
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *fail = reinterpret_cast<volatile int *>(tmem_slot + 1);

    // a piece's CTA: of its chain's `cut`, the piece and the block of rows, or Phi
    const int cut = PASS == FIND ? find_units(prm.pieces.n, prm.pblocks) : prm.pieces.n * prm.pblocks;
    int piece = (blockIdx.x % cut) / prm.pblocks, kind = (blockIdx.x % cut) % prm.pblocks;
    if (PASS == FIND) find_unit(blockIdx.x % cut, prm.pblocks, piece, kind);
    const bool phi = PASS == FIND && kind == prm.pblocks;
    const int R = phi ? N : P;  // rows of the state
    // warps with rows of the state; those whose rows lie past R take no part
    const int row_warps = NH == 2 || R >= 128 ? 8 : 2 * ((R + 31) / 32);
    __shared__ Segments seg;
    // item k: its chunks [c0, c1) that hold tokens, and where its rows are
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
            m.prow0 = NH == 2 ? 0 : (un % prm.pblocks) * 128;  // state row of lane 0
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
            if (k == BAR_V_EMPTY || k == BAR_V_EMPTY + 1 || k == BAR_O_READ) count = row_warps;
            if (k == BAR_T_EMPTY || k == BAR_T_EMPTY + 1) count = 2 * row_warps;
            if (k >= BAR_S_FULL && k < BAR_U_FULL + 2) count = 32 * row_warps;
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
    const uint32_t tQS = tmem + col::kQS, tKS = tmem + col::kKS, tW = tmem + col::kW, tMW = tmem + col::kMW;
    const uint32_t tS = tmem + col::kS, tOp = tmem + col::kOp;
    pdl_wait();
    const int items = PASS == WHOLE ? seg.items() : 1;

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            int it = 0, done = 0, v_done = 0;
            for (int k = 0; k < items; ++k) {
                const Item m = get(k);
                for (int c = m.c0; c < m.c1; ++c, ++it) {
                    const int s = it & 1;
                    const uint32_t ph = ((it >> 1) & 1) ^ 1;
                    if (!wait_on(&bars[BAR_T_EMPTY + s], ph, fail) || !wait_on(&bars[BAR_KQ_EMPTY + s], ph, fail)) break;
                    uint64_t *bar = &bars[BAR_KQ_FULL + s];
                    uint8_t *d = sKQ + s * 32768;
                    tc::mbar_arrive_expect_tx(bar, 32768u);
                    for (int e = 0; e < 2; ++e) {
                        tc::tma_load_4d(d + e * 16384, &prm.mq, bar, 64 * e, m.grp, c * kC, (int)m.b);
                        tc::tma_load_4d(d + e * 16384 + 8192, &prm.mk, bar, 64 * e, m.grp, c * kC, (int)m.b);
                    }
                    bar = &bars[BAR_T_FULL + s];
                    tc::mbar_arrive_expect_tx(bar, NH * (kTilesFwd + kScalBytes));
                    for (int hf = 0; hf < NH; ++hf) {
                        const int64_t item = (m.b * a.H + m.h0 + hf) * prm.nc + c;
                        tc::bulk_load(sT + (s * NH + hf) * kTilesFwd, prm.tiles + item * prm.tile_bytes, kTilesFwd, bar);
                        tc::bulk_load(scal + (s * NH + hf) * kScalDecay, prm.scal + item * kScal, kScalBytes, bar);
                    }
                    done = it + 1;
                    if (!wait_on(&bars[BAR_V_EMPTY + s], ph, fail)) break;  // y of the stage's last chunk has left
                    bar = &bars[BAR_V_FULL + s];
                    tc::mbar_arrive_expect_tx(bar, 16384u);
                    for (int e = 0; e < 4; ++e) {
                        const int hh = NH == 2 ? m.h0 + (e >> 1) : m.h0;
                        const int p = NH == 2 ? 32 * (e & 1) : (phi ? 128 * prm.pblocks : m.prow0) + 32 * e;  // Phi: past P, zeros
                        tc::tma_load_4d(sV + s * 16384 + e * 4096, &prm.mv, bar, p, hh, c * kC, (int)m.b);
                    }
                    v_done = it + 1;
                }
                if (*fail) break;
            }
            // no copy outlives the block, even where a wait gave up
            for (int c = imax(0, done - 2); c < done; ++c) {
                tc::mbar_wait(&bars[BAR_T_FULL + (c & 1)], (c >> 1) & 1, kWaitNs);
                tc::mbar_wait(&bars[BAR_KQ_FULL + (c & 1)], (c >> 1) & 1, kWaitNs);
            }
            for (int c = imax(0, v_done - 2); c < v_done; ++c)
                tc::mbar_wait(&bars[BAR_V_FULL + (c & 1)], (c >> 1) & 1, kWaitNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- products
        const uint32_t one = tc::elect_one();
        const uint32_t id128 = tc::idesc_bf16(128, 128, false, false), id64 = tc::idesc_bf16(128, 64, false, false);
        const uint32_t idS = tc::idesc_bf16(128, N <= 64 ? 64 : 128, false, true);
        // descriptors of the tiles' first bytes; a step adds its byte offset / 16
        const uint64_t dT = tc::sdesc_sw128(tc::smem_u32(sT), 16, 1024);
        const uint64_t dKQ = tc::sdesc_sw128(tc::smem_u32(sKQ), 16, 1024);
        const uint64_t dK = tc::sdesc_sw128(tc::smem_u32(sKQ) + 8192, 16384, 1024);  // K's rows, columns contiguous
        int it = 0;
        for (int k = 0; k < items; ++k) {
        const Item m = get(k);
        const int64_t len = m.len;
        for (int c = m.c0; c < m.c1; ++c, ++it) {
            const int s = it & 1;
            const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
            const uint64_t kq = dKQ + (uint64_t)(s * 2048), kk = dK + (uint64_t)(s * 2048);
            wait_on(&bars[BAR_KQ_FULL + s], ph2, fail);
            __syncwarp();
            if ((int64_t)(c + 1) * kC > len && len < a.L) {  // tokens past the sequence's length
                for (int x = (int)(len - (int64_t)c * kC) * 8 + lane; x < kC * 8; x += 32)
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<uint4 *>(sKQ + s * 32768 + k * 8192)[x] = make_uint4(0, 0, 0, 0);
                tc::fence_proxy_async_smem();
                __syncwarp();
            }
            if (it > 0) wait_on(&bars[BAR_O_READ], ph ^ 1, fail);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_S_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int pn = 0; pn < 2; ++pn)  // panels of 64 columns; S hi, S lo
                    if (pn == 0 || N > 64)
#pragma unroll
                        for (int k = half; k < 8; k += 2)
                            tc::mma_bf16_ts_if(one, tQS, tOp + 64 * (k >> 2) + 32 * pn + 8 * (k & 3),
                                               kq + (1024 * pn + 2 * (k & 3)), id128, half > 0 || pn > 0 || k > 0);
            }
            tc::mma_commit_if(one, &bars[BAR_A_DONE]);
            wait_on(&bars[BAR_T_FULL + s], ph2, fail);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_R_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int hf = 0; hf < NH; ++hf) {
                    const uint32_t r0 = tOp + 64 * hf;
                    const uint64_t dt = dT + (uint64_t)((s * NH + hf) * (kTilesFwd / 16)), dl = dt + 1024;
#pragma unroll
                    for (int k = half; k < 8; k += 2)  // R hi, R lo with [T hi; M T]
                        tc::mma_bf16_ts_if(one, tW, r0 + 8 * k, dt + 2 * (k & 3), id128, half > 0 || hf > 0 || k > 0);
#pragma unroll
                    for (int k = half; k < 4; k += 2) tc::mma_bf16_ts_if(one, tW, r0 + 8 * k, dl + 2 * k, id64, 1);
                }
            }
            tc::mma_commit_if(one, &bars[BAR_B_DONE]);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait_on(&bars[BAR_U_FULL + half], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int k = half; k < 8; k += 2)  // the update hi, lo
                    tc::mma_bf16_ts_if(one, tS, tOp + 8 * k, kk + 128 * (k & 3), idS, 1);
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
            const int64_t b = m.b, len = m.len;
            const int h = m.h0 + hf, p = (NH == 2 ? 32 * (q & 1) : m.prow0 + 32 * q) + lane;  // this thread's row
            const int64_t bh = b * a.H + h, srow = (bh * a.P + p) * a.N;  // this thread's row of [B][H][P][N]
            // 16 columns of the state as hi + lo operands, and scaled for the next accumulation
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
                tc::tmem_st16(tS + lq + c0, sc);
                if (SAVE && p < P) {
                    uint4 *o = reinterpret_cast<uint4 *>(prm.states + (((b * a.H + h) * (prm.nc + 1) + c) * P + p) * N + c0);
                    if (c0 < N) o[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if (c0 + 8 < N) o[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                }
            };
            // 16 columns of the state from this thread's float32 row, which may be null (zero; Phi: the identity)
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
            // and to them; with SAVE the final state in bf16 as well
            auto out_state = [&](const float (&v)[16], float *row, int c0, bool last) {
                if (p >= R) return;
                if (row)
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (c0 + k < N)
                            *reinterpret_cast<float4 *>(row + c0 + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                if (SAVE && last) {
                    uint4 *o = reinterpret_cast<uint4 *>(prm.states + (((b * a.H + h) * (prm.nc + 1) + m.nc) * P + p) * N + c0);
                    if (c0 < N) o[0] = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
                    if (c0 + 8 < N)
                        o[1] = make_uint4(pack2(v[8], v[9]), pack2(v[10], v[11]), pack2(v[12], v[13]), pack2(v[14], v[15]));
                }
            };
            auto row_of = [&](auto *states) { return states ? states + srow : nullptr; };
            if (m.c0 >= m.c1) {  // no token, or none left
                if (PASS != FIND && m.nc == 0 && m.c0 == 0)
                    for (int c0 = 64 * ch; c0 < 64 * ch + 64; c0 += 16) {
                        float v[16];
                        get_state(v, row_of(a.init), c0);
                        out_state(v, row_of(a.final_state), c0, true);
                    }
                continue;
            }
            if (PASS == WHOLE && m.c0 > 0) flag_wait(prm.flags + m.unit, fail);
            const float *from = m.c0 == 0 ? row_of(a.init) : PASS == WHOLE ? row_of(prm.carry) : nullptr;
            if (PASS == PIECES) from = prm.pieces.in + ((bh * prm.pieces.n + m.piece) * P + p) * N;
            wait_on(&bars[BAR_T_FULL + (it & 1)], (it >> 1) & 1, fail);
            const float eq0 = scal[((it & 1) * NH + hf) * kScalDecay + kScalEnd];
            __syncwarp();
#pragma unroll 1
            for (int k4 = 0; k4 < 4; ++k4) {
                const int c0 = 64 * ch + 16 * k4;
                float v[16];
                get_state(v, from, c0);
                put_state(v, c0, eq0, m.c0);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::mbar_arrive(&bars[BAR_S_FULL]);
            tc::mbar_arrive(&bars[BAR_S_FULL + 1]);
            for (int c = m.c0; c < m.c1; ++c, ++it) {
                const int s = it & 1;
                const uint32_t ph = it & 1, ph2 = (it >> 1) & 1;
                const float *sc = scal + (s * NH + hf) * kScalDecay + 32 * ch;
                // R^T = v - exp(c) (K S0^T)^T; vt is this thread's column of the warp's [32 tokens][32 rows]
                __nv_bfloat16 *vt = reinterpret_cast<__nv_bfloat16 *>(sV + s * 16384 + q * 4096 + ch * 2048) + lane;
                wait_on(&bars[BAR_V_FULL + s], ph2, fail);
                const int valid = (int)imin<int64_t>(32, len - (int64_t)c * kC - 32 * ch);
                for (int k = imax(0, valid); k < 32; ++k) vt[32 * k] = __float2bfloat16_rn(0.f);  // past the length
                uint64_t v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = f2(to_f32(vt[64 * k]), to_f32(vt[64 * k + 32]));
                wait_on(&bars[BAR_A_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < 32; t0 += 16) {
                    float ks[16];
                    tc::tmem_ld16(tKS + lq + 32 * ch + t0, ks);
                    float4 ng[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) ng[k] = *reinterpret_cast<const float4 *>(sc + SC_NEG * kC + t0 + 4 * k);
                    tc::tmem_ld_wait();
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        split2(fma2(f2(ng[k].x, ng[k].y), f2(ks[4 * k], ks[4 * k + 1]), v[t0 / 2 + 2 * k]), hi[2 * k], lo[2 * k]);
                        split2(fma2(f2(ng[k].z, ng[k].w), f2(ks[4 * k + 2], ks[4 * k + 3]), v[t0 / 2 + 2 * k + 1]),
                               hi[2 * k + 1], lo[2 * k + 1]);
                    }
                    tc::tmem_st8(tOp + lq + 64 * hf + 16 * ch + t0 / 2, hi);
                    tc::tmem_st8(tOp + lq + 64 * hf + 32 + 16 * ch + t0 / 2, lo);
                    if (NH == 2) {  // zeros in the other head's operand
#pragma unroll
                        for (int k = 0; k < 8; ++k) hi[k] = 0u;
                        tc::tmem_st8(tOp + lq + 64 * (hf ^ 1) + 16 * ch + t0 / 2, hi);
                        tc::tmem_st8(tOp + lq + 64 * (hf ^ 1) + 32 + 16 * ch + t0 / 2, hi);
                    }
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars[BAR_R_FULL + t0 / 16]);
                }
                // the update's operand, exp(c_63 - c) beta w
                float4 tl[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) tl[k] = *reinterpret_cast<const float4 *>(sc + SC_BTAIL * kC + 4 * k);
                wait_on(&bars[BAR_B_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
#pragma unroll
                for (int t0 = 0; t0 < 32; t0 += 16) {
                    float u[16];
                    tc::tmem_ld16(tW + lq + 32 * ch + t0, u);
                    tc::tmem_ld_wait();
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 f = tl[t0 / 4 + k];
                        split2(mul2(f2(u[4 * k], u[4 * k + 1]), f2(f.x, f.y)), hi[2 * k], lo[2 * k]);
                        split2(mul2(f2(u[4 * k + 2], u[4 * k + 3]), f2(f.z, f.w)), hi[2 * k + 1], lo[2 * k + 1]);
                    }
                    tc::tmem_st8(tOp + lq + 16 * ch + t0 / 2, hi);
                    tc::tmem_st8(tOp + lq + 32 + 16 * ch + t0 / 2, lo);
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    tc::mbar_arrive(&bars[BAR_U_FULL + t0 / 16]);
                }
                if (lane == 0) tc::mbar_arrive(&bars[BAR_T_EMPTY + s]);
                // the state that enters the next chunk
                const bool next = c + 1 < m.c1;
                if (next) wait_on(&bars[BAR_T_FULL + (s ^ 1)], ((it + 1) >> 1) & 1, fail);
                const float eqn = next ? scal[((s ^ 1) * NH + hf) * kScalDecay + kScalEnd] : 0.f;
                wait_on(&bars[BAR_C_DONE], ph, fail);
                __syncwarp();
                tc::tc_fence_after();
                if (next) {
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
                        const int c0 = 64 * ch + 16 * half;
                        float v0[16], v1[16];
                        tc::tmem_ld16(tS + lq + c0, v0);
                        tc::tmem_ld16(tS + lq + c0 + 32, v1);
                        tc::tmem_ld_wait();
                        put_state(v0, c0, eqn, c + 1);
                        put_state(v1, c0 + 32, eqn, c + 1);
                        tc::tmem_st_wait();
                        tc::tc_fence_before();
                        tc::mbar_arrive(&bars[BAR_S_FULL + half]);
                    }
                } else {
                    const bool last = PASS != FIND && m.c1 == m.nc;
                    float *to = PASS == FIND ? (phi ? prm.pieces.phi + ((bh * (prm.pieces.n - 1) + m.piece) * N + p) * N
                                                    : prm.pieces.psi + ((bh * (prm.pieces.n - 1) + m.piece) * P + p) * N)
                                : last       ? row_of(a.final_state)
                                             : (PASS == WHOLE ? row_of(prm.carry) : nullptr);
#pragma unroll 1
                    for (int c0 = 64 * ch; c0 < 64 * ch + 64; c0 += 16) {
                        float v0[16];
                        tc::tmem_ld16(tS + lq + c0, v0);
                        tc::tmem_ld_wait();
                        out_state(v0, to, c0, last);
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
        // ------------------------------------------------------------ y, and w
        const int cw = warp - kOutWarp0, q = cw & 3, ch = cw >> 2;
        const int hf = NH == 2 ? q >> 1 : 0;
        const uint32_t lq = (uint32_t)(32 * q) << 16;
        int it = 0;
        for (int kk = 0; kk < (2 * q < row_warps ? items : 0); ++kk) {
            const Item m = get(kk);
            const int64_t b = m.b;
            const int h = m.h0 + hf, p32 = NH == 2 ? 32 * (q & 1) : m.prow0 + 32 * q, p = p32 + lane;
            for (int c = m.c0; c < m.c1; ++c, ++it) {
                const int s = it & 1;
                const float *sc = scal + (s * NH + hf) * kScalDecay + 32 * ch;
                uint16_t *vt = reinterpret_cast<uint16_t *>(sV + s * 16384 + q * 4096 + ch * 2048) + lane;
                uint16_t *wt = reinterpret_cast<uint16_t *>(sW + q * 4096 + ch * 2048) + lane;
                wait_on(&bars[BAR_B_DONE], it & 1, fail);
                __syncwarp();
                tc::tc_fence_after();
                if constexpr (PASS == FIND) {  // no outputs: the buffers are free at once
                    if (lane == 0) {
                        tc::mbar_arrive(&bars[BAR_O_READ]);
                        tc::mbar_arrive(&bars[BAR_T_EMPTY + s]);
                        tc::mbar_arrive(&bars[BAR_V_EMPTY + s]);
                    }
                    __syncwarp();
                    continue;
                }
                float qs[32], o[32];
                if (SAVE) {
                    tc::tmem_ld32(tW + lq + 32 * ch, qs);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const uint32_t y = pack2(qs[k], qs[k + 1]);
                        wt[32 * k] = (uint16_t)y;
                        wt[32 * k + 32] = (uint16_t)(y >> 16);
                    }
                }
                tc::tmem_ld32(tQS + lq + 32 * ch, qs);
                tc::tmem_ld32(tMW + lq + 32 * ch, o);
                tc::tmem_ld_wait();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[BAR_O_READ]);
                wait_on(&bars[BAR_T_FULL + s], (it >> 1) & 1, fail);
                const uint64_t s2 = f2(a.scale, a.scale);
                float4 eg[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) eg[k] = *reinterpret_cast<const float4 *>(sc + SC_EG * kC + 4 * k);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float4 e = eg[k / 4];
                    float y0, y1;
                    un2(fma2(mul2(k & 2 ? f2(e.z, e.w) : f2(e.x, e.y), s2), f2(qs[k], qs[k + 1]), f2(o[k], o[k + 1])), y0, y1);
                    const uint32_t y = pack2(y0, y1);
                    vt[32 * k] = (uint16_t)y;
                    vt[32 * k + 32] = (uint16_t)(y >> 16);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::mbar_arrive(&bars[BAR_T_EMPTY + s]);
                    if (p32 < P) {
                        if (a.y) tc::tma_store_4d(&prm.my, vt, p32, h, c * kC + 32 * ch, (int)b);
                        if (SAVE) tc::tma_store_4d(&prm.mw, wt, p32, h, c * kC + 32 * ch, (int)b);
                        tc::bulk_commit();
                        tc::bulk_wait_read_all();
                    }
                    tc::mbar_arrive(&bars[BAR_V_EMPTY + s]);
                }
                __syncwarp();
            }
            if (PASS != FIND && a.y && p < P && m.c0 == 0)  // y is zero past the last chunk
                for (int64_t t = (int64_t)m.nc * kC + ch; t < a.L; t += 2)
                    ((__nv_bfloat16 *)a.y)[((b * a.L + t) * a.H + h) * P + p] = __float2bfloat16_rn(0.f);
        }
        if (lane == 0) tc::bulk_wait_all();
    }
    __syncthreads();
    if (tid == 0 && *fail) atomicCAS(a.status, SSD_OK, SSD_ERR_TIMEOUT);
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int NH, bool SAVE, int PASS> cudaError_t launch_form(ChainParams &p, cudaStream_t stream) {
    const DeltaArgs &a = p.a;
    p.pblocks = (int)row_blocks(a.P);
    p.units_per_b = (int)(NH == 2 ? a.H / 2 : a.H * p.pblocks);
    static DeviceOnce configured;
    int dev = 0;
    cudaError_t e = cudaSuccess;
    if (configured.pending(&dev, &e)) {
        e = cudaFuncSetAttribute(delta_chain_kernel<NH, SAVE, PASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes(NH));
        if (e != cudaSuccess) return e;
        configured.done(dev);
    } else if (e != cudaSuccess) {
        return e;
    }
    if (PASS != WHOLE) {
        const int64_t grid = a.B * a.H * (PASS == FIND ? find_units(p.pieces.n, p.pblocks) : p.pieces.n * p.pblocks);
        return launch_programmatic(delta_chain_kernel<NH, SAVE, PASS>, dim3((unsigned)grid), dim3(kThreads), smem_bytes(NH),
                                   stream, p);
    }
    return launch_chains(delta_chain_kernel<NH, SAVE, PASS>, p, a.B * p.units_per_b, p.nc, kThreads, smem_bytes(NH), stream);
}

}  // namespace

cudaError_t launch_chain(const PrepArgs &pr, __nv_bfloat16 *states, __nv_bfloat16 *w, cudaStream_t stream) {
    const DeltaArgs &a = pr.a;
    ChainParams p;
    p.a = a;
    bool ok = tma_map_heads(&p.mq, a.q, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&p.mk, a.k, a.N, a.G, a.L, a.B, 64, kC, true);
    ok = ok && tma_map_heads(&p.mv, a.v, a.P, a.H, a.L, a.B, 32, kC, false);
    ok = ok && tma_map_heads(&p.my, a.y ? a.y : w, a.P, a.H, a.L, a.B, 32, 32, false);
    ok = ok && tma_map_heads(&p.mw, w ? w : a.y, a.P, a.H, a.L, a.B, 32, 32, false);
    if (!ok) return cudaErrorInvalidValue;
    p.tiles = pr.tiles;
    p.scal = pr.scal;
    p.tile_bytes = pr.tile_bytes;
    p.states = states;
    p.flags = pr.flags;
    p.carry = pr.carry;
    p.nc = pr.nc;
    p.pieces = pr.pieces;
    if (p.pieces.n > 1) {
        cudaError_t e = launch_form<1, false, FIND>(p, stream);
        if (e == cudaSuccess) e = launch_combine(p.pieces, a.init, a.B * a.H, a.P, a.N, stream);
        if (e != cudaSuccess) return e;
        return states ? launch_form<1, true, PIECES>(p, stream) : launch_form<1, false, PIECES>(p, stream);
    }
    const bool pairs = pair_heads(a);
    if (states) return pairs ? launch_form<2, true, WHOLE>(p, stream) : launch_form<1, true, WHOLE>(p, stream);
    return pairs ? launch_form<2, false, WHOLE>(p, stream) : launch_form<1, false, WHOLE>(p, stream);
}

Pieces plan_pieces(int64_t B, int64_t H, int64_t P, int64_t nc, bool backward) {
    Pieces q{1, (int)nc, nullptr, nullptr, nullptr};
    const int64_t pb = row_blocks(P), sms = sm_count(152) / imax<int64_t>(1, B * H);
    const int64_t most = imin<int64_t>(1 + (sms + 1) / (pb + 1), sms / pb);
    double best = (backward ? 5.9 : 2.45) * (double)nc;
    for (int64_t n = 2; n <= imin<int64_t>(most, nc); ++n) {
        const int64_t chunks = (nc + n - 1) / n;
        const double t = (backward ? 11.5 : 5.3) * (double)chunks + (backward ? 1.4 : 0.7) * (double)(n - 1) + (backward ? 30. : 20.);
        if (t < best && (n - 1) * chunks < nc) best = t, q.n = (int)n, q.chunks = (int)chunks;
    }
    return q;
}

namespace {

// The state carried over the pieces, S Phi + Psi in float32. A CTA has ROWS rows;
// thread (n, j) adds up the j-th quarter of the products of column n, and the
// quarters are then added in a fixed order. A value of Phi is replaced by the next
// piece's as soon as it has been used, so that a piece costs its products and two barriers.
// in[0] is a copy of the chains' first states (zero without them): the pieces then run at once without
// reading them, and the last piece may write its final state over them.
// 4 rows where these CTAs have an SM each, else 8, so that fewer read all of Phi: a whole call
// of B1 L8192 H4 takes 88 us with 4 and 97 with 8, the backward of B1 L2048 H24 184 and 180.
constexpr int kCarryPart = 32;
template <int ROWS> __global__ void __launch_bounds__(512, 2) combine_kernel(Pieces q, const float *first, int P, int N) {
    pdl_wait();
    __shared__ float4 s[128][ROWS / 4];  // [column][row]
    __shared__ float part[4][ROWS][128];
    const int n = threadIdx.x & 127, j = threadIdx.x >> 7, m0 = j * kCarryPart;
    const int64_t bh = blockIdx.x, p0 = (int64_t)blockIdx.y * ROWS + j;  // this thread adds up rows p0, p0 + 4
    // column n (past N the last one, whose sums are not kept) of Phi's rows m0, m0 + 1, ... (past N the last one, times 0)
    const int last = imin(n, N - 1), steps = imin(kCarryPart, imax(1, N - m0));
    const float *phi = q.phi + (bh * (q.n - 1) * N + imin(m0, N - 1)) * N + last;
    const float *psi = q.psi + (bh * (q.n - 1) * P + p0) * N + last;
    float *in = q.in + (bh * q.n * P + p0) * N + n;
    float f[kCarryPart], add[ROWS / 4];
    auto psi_at = [&](int k, int r) { return k < q.n - 1 && p0 + 4 * r < P ? psi[((int64_t)k * P + 4 * r) * N] : 0.f; };
    auto leave = [&](int k, int r, float v) {
        if (n < N && p0 + 4 * r < P) in[((int64_t)k * P + 4 * r) * N] = v;
        reinterpret_cast<float *>(&s[n][r])[j] = n < N ? v : 0.f;
    };
#pragma unroll
    for (int r = 0; r < ROWS / 4; ++r)
        if (n < N && p0 + 4 * r < P)
            in[(int64_t)4 * r * N] = first ? first[(bh * P + p0 + 4 * r) * N + n] : 0.f;
    const float *at = phi + (q.n > 2 ? (int64_t)N * N : 0);
#pragma unroll
    for (int i = 0; i < kCarryPart; ++i) {
        f[i] = *at;
        at += i + 1 < steps ? N : 0;
    }
#pragma unroll
    for (int r = 0; r < ROWS / 4; ++r) {
        leave(1, r, psi_at(0, r));
        add[r] = psi_at(1, r);
    }
    __syncthreads();
    for (int k = 1; k < q.n - 1; ++k) {
        float v[ROWS] = {};
        at = phi + (int64_t)imin(k + 1, q.n - 2) * N * N;
#pragma unroll
        for (int i = 0; i < kCarryPart; ++i) {
#pragma unroll
            for (int r = 0; r < ROWS; r += 4) {
                const float4 x = s[m0 + i][r / 4];
                v[r] = fmaf(x.x, f[i], v[r]), v[r + 1] = fmaf(x.y, f[i], v[r + 1]);
                v[r + 2] = fmaf(x.z, f[i], v[r + 2]), v[r + 3] = fmaf(x.w, f[i], v[r + 3]);
            }
            f[i] = *at;
            at += i + 1 < steps ? N : 0;
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) part[j][r][n] = v[r];
        __syncthreads();
#pragma unroll
        for (int r = 0; r < ROWS / 4; ++r) {
            const int w = 4 * r + j;
            leave(k + 1, r, ((part[0][w][n] + part[1][w][n]) + (part[2][w][n] + part[3][w][n])) + add[r]);
            add[r] = psi_at(k + 1, r);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_combine(const Pieces &q, const float *first, int64_t BH, int64_t P, int64_t N, cudaStream_t stream) {
    const int rows = BH * ((P + 3) / 4) <= sm_count(152) ? 4 : 8;
    return launch_programmatic(rows == 4 ? combine_kernel<4> : combine_kernel<8>, dim3((unsigned)BH, (unsigned)((P + rows - 1) / rows)),
                               dim3(512), 0, stream, q, first, (int)P, (int)N);
}

}  // namespace delta

namespace {
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
size_t chunks(int64_t L) { return (size_t)((L + delta::kC - 1) / delta::kC); }
}  // namespace

bool delta::tc_takes(int io, int64_t B, int64_t L, int64_t H, int64_t P, int64_t N, int64_t few) {
    if (L <= 16 && L * B * H * delta_row_blocks(P) <= few) return false;
    return io == IO_BF16 && P % 8 == 0 && N % 8 == 0 && N <= 128 && B * (int64_t)chunks(L) * H <= 0x7fffffffLL &&
           device_cc_major_cached() == 10;
}

// The recurrent kernel against these, N 128, P 64: 7 us and 13 for 16 tokens of 24 heads, 18 and 21 of
// 160; 29 and 37 for 4 tokens of 640 heads, but 54 and 50 with P 128; 11 and 14 for 24 tokens
// of 24 heads, but 16 and 14 of 80.
bool delta_tc_supported(int io, int64_t B, int64_t L, int64_t H, int64_t P, int64_t N) {
    return delta::tc_takes(io, B, L, H, P, N, 10240);
}

size_t delta_tc_workspace(int64_t B, int64_t L, int64_t H, int64_t P, int64_t N) {
    const size_t items = (size_t)(B * H) * chunks(L);
    return 256 + items * delta::kTilesFwd + up256(items * delta::kScal * 4) + up256((size_t)(B * H * delta::row_blocks(P)) * 8) +
           up256((size_t)(B * H * P * N) * 4) + delta::plan_pieces(B, H, P, (int64_t)chunks(L), false).bytes(B * H, P, N);
}

cudaError_t launch_delta_tc(const DeltaArgs &a, void *workspace, cudaStream_t stream) {
    delta::PrepArgs p;
    p.a = a;
    p.nc = (int64_t)chunks(a.L);
    p.tile_bytes = delta::kTilesFwd;
    const size_t items = (size_t)(a.B * a.H * p.nc);
    p.tiles = static_cast<uint8_t *>(workspace) + 256;
    uint8_t *o = p.tiles + items * delta::kTilesFwd;
    p.scal = reinterpret_cast<float *>(o);
    o += up256(items * delta::kScal * 4);
    p.flags = reinterpret_cast<int *>(o);
    o += up256((size_t)(a.B * a.H * delta::row_blocks(a.P)) * 8);
    p.carry = reinterpret_cast<float *>(o);
    p.pieces = delta::plan_pieces(a.B, a.H, a.P, p.nc, false);
    p.pieces.carve(o + up256((size_t)(a.B * a.H * a.P * a.N) * 4), a.B * a.H, a.P, a.N);
    cudaError_t e = delta::launch_prep(p, stream);
    return e != cudaSuccess ? e : delta::launch_chain(p, nullptr, nullptr, stream);
}

}  // namespace ssd
