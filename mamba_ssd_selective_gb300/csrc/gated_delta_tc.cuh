// What the tensor-core kernels of the gated delta rule share: the chunk's
// tiles and scalars in the workspace, packed float32 arithmetic, bounded waits.
//
// Within a chunk of 64 tokens, with c the inclusive sums of g, S0 the entering
// state, D_tj = exp(c_t - c_j) and s the output scale, the rule is a triangular
// solve for w (u_t = beta_t w_t is what is added along k_t):
//     A_tj = D_tj (k_t . k_j) beta_j, j < t            T = (I + A)^-1
//     R = V - exp(c) K S0^T                            w = T R
//     Y = s exp(c) Q S0^T + M w                        M_tj = s D_tj (q_t . k_j) beta_j, j <= t
//     S1 = exp(c_63) S0 + (exp(c_63 - c) beta w)^T K
// With beta on the columns of A nothing is divided by it, whatever its value.
// T and M T depend on the inputs alone: delta_prep_kernel forms them for every
// (b, head, chunk) at once, and the chains of chunks, forward and backward, read them.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"
#include "gated_delta_columns.h"
#include "launch.h"
#include "ssd_scan.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kC = 64;  // tokens per chunk
constexpr float kLog2e = 1.4426950408889634f;

// Workspace: for item (b, head, chunk) = (b H + h) nc + chunk the tiles T hi, M T
// hi, T lo and (backward) M T lo, 64 x 64 bf16 each in the 128-byte swizzle,
// and the scalars below, one float per token each, then exp(c_63).
constexpr uint32_t kTile = 8192, kTilesFwd = 3 * kTile, kTilesBwd = 4 * kTile;
enum {
    SC_EG,     // exp(c)
    SC_NEG,    // -exp(c)
    SC_BETA,
    SC_BTAIL,  // beta exp(c_63 - c)
    SC_CHAIN,  // the chains read the rows up to here, and exp(c_63) behind them
    SC_HI = SC_CHAIN,  // c in base-2 units, rounded to float32
    SC_ROW,    // 2^(c - hi)
    SC_INV,    // beta 2^(hi - c): D_tj beta_j = 2^(hi_t - hi_j) ROW_t INV_j
    SC_ROWS
};
constexpr int kScalEnd = SC_CHAIN * kC, kScalDecay = kScalEnd + 4;  // exp(c_63); the last three rows
constexpr uint32_t kScalBytes = kScalDecay * 4;                     // what the chains load
constexpr int kScal = kScalDecay + 3 * kC;

// Whether these kernels take a call: its sizes fit, and it isn't so short (tokens x blocks of 16 rows at most `few`,
// and at most 16 tokens) that the recurrent kernels are faster.
bool tc_takes(int io, int64_t B, int64_t L, int64_t H, int64_t P, int64_t N, int64_t few);

// Blocks of 128 state rows of a head.
__host__ __device__ inline int64_t row_blocks(int64_t P) { return (P + 127) / 128; }

// Few chains leave most of the GPU idle, and a chain's chunks cannot overlap. What a
// stretch of chunks does to a state is linear, S -> S Phi + Psi with Phi [N, N]
// and Psi [P, N], and the chain kernels find both: Psi is the state they leave
// when they start from zero, Phi the one that they leave on N rows when they start from
// the identity with v = 0. So a chain of nc chunks is cut into n pieces; Phi
// and Psi of all but the last are found at once (of the first only what it makes of the
// chain's first state), combine_kernel carries the state over the pieces, and a second
// run of all pieces at once forms the outputs. All of it in float32, Phi and Psi from
// the same hi + lo products as the states.
struct Pieces {
    int n, chunks;          // n = 1: the chain whole
    float *phi, *psi, *in;  // [B H][n - 1][N][N], [B H][n - 1][P][N], [B H][n][P][N] states entering the pieces
    size_t bytes(int64_t BH, int64_t P, int64_t N) const {
        return n == 1 ? 0 : sizeof(float) * (size_t)BH * (size_t)((n - 1) * N * (N + P) + n * P * N);
    }
    void carve(void *base, int64_t BH, int64_t P, int64_t N) {
        phi = static_cast<float *>(base);
        psi = phi + BH * (n - 1) * N * N;
        in = psi + BH * (n - 1) * P * N;
    }
};
// How the chains are run: whole (handed on between CTAs where they are cut), the
// pieces' Phi and Psi, or the pieces from their entering states.
enum { WHOLE, FIND, PIECES };
// The number of pieces, from times on GB300: whole, a chunk takes 2.45 us (5.9 with the
// backward's two chains); in pieces 5.3 (11.5), and 0.7 (1.4) for each piece that the
// state is carried over and 20 (30) for the launches more. Every CTA has an SM of its
// own. Whole against pieces, whole calls, N 128, P 64: B1 L4096 H24 187 and 132 us (backward
// 466 and 305), B1 L8192 H4 322 and 88 (767 and 189), B1 L2048 H24 100 and 85 (247 and 188);
// and where this rule leaves them whole: B1 L1024 H24 55 and 58, B1 L768 H4 44 and 46 (B1 L1024 H48 160 and 182).
// The costs are those of N 128, P 64 for every size. With P or N of 64 and 128 the cuts it makes paid as well: B1 L2048 H24
// whole and cut 88 and 66 (N 64), 98 and 82 (P 128), 90 and 73 (both), backward 211 and 154, 310 and 220, 262 and 194.
Pieces plan_pieces(int64_t B, int64_t H, int64_t P, int64_t nc, bool backward);
// The CTAs of a chain in the first run, and what CTA i of it does: `kind` a block of rows of Psi or, past them, Phi.
__host__ __device__ inline int find_units(int n, int pblocks) { return (n - 1) * (pblocks + 1) - 1; }
__device__ __forceinline__ void find_unit(int i, int pblocks, int &piece, int &kind) {
    i += i >= pblocks;  // the first piece has no Phi
    piece = i / (pblocks + 1), kind = i % (pblocks + 1);
}
// in[piece] from phi and psi; in[0] from the chains' first states [B H][P][N], which may be null (zero)
cudaError_t launch_combine(const Pieces &q, const float *first, int64_t BH, int64_t P, int64_t N, cudaStream_t stream);

struct PrepArgs {
    DeltaArgs a;
    int64_t nc;
    uint8_t *tiles;  // [B][H][nc][tile_bytes]
    float *scal;     // [B][H][nc][kScal]
    int *flags;      // [2][B H row_blocks(P)]: cleared here, set where the forward or the reverse chain hands a state on
    float *carry;    // [B][H][P][N]: that state
    Pieces pieces;
    uint32_t tile_bytes;
};
cudaError_t launch_prep(const PrepArgs &p, cudaStream_t stream);
// The chain over the chunks: y and the final state (each may be null), and for the backward the
// states entering each chunk [B][H][nc + 1][P][N] (the final one last) and w [B, L, H, P], in bf16.
cudaError_t launch_chain(const PrepArgs &p, __nv_bfloat16 *states, __nv_bfloat16 *w, cudaStream_t stream);

// Whether a CTA takes two heads of a group: where pairs alone fill the SMs (B8 L2048 H80 G40: 477 us in pairs, 599 one by
// one; the backward of B4 takes 92 us longer one by one); with fewer, one by one (B2 L2048 H80 would leave half of the SMs idle in pairs).
inline bool pair_heads(const DeltaArgs &a) {
    return a.P <= 64 && (a.H / a.G) % 2 == 0 && a.B * (a.H / 2) >= (int64_t)sm_count(152);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}
// A pair as bf16 pairs hi and lo, hi + lo within 2^-17 of each.
__device__ __forceinline__ void split2(uint64_t v, uint32_t &hi, uint32_t &lo) {
    float x, y;
    un2(v, x, y);
    hi = pack2(x, y);
    un2(fma2(f2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)), f2(-1.f, -1.f), v), x, y);
    lo = pack2(x, y);
}
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) { split2(f2(x, y), hi, lo); }

// Waits for the phase of `parity`; gives up after kWaitNs or once *fail is set.
// The part that really waits is out of line, so that the roles' loops stay small
// in the instruction cache, and looks at the clock once in 32 polls.
static __device__ __noinline__ bool wait_long(uint32_t addr, uint32_t parity, volatile int *fail) {
    const uint64_t t0 = tc::global_ns();
    for (;;) {
#pragma unroll 1
        for (int k = 0; k < 32; ++k)
            if (tc::mbar_try_wait(addr, parity)) return true;
        if (*fail) return false;
        if (tc::global_ns() - t0 > kWaitNs) {
            *fail = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *fail) {
    const uint32_t addr = tc::smem_u32(bar);
    return tc::mbar_try_wait(addr, parity) || wait_long(addr, parity, fail);
}

// The chains of chunks laid end to end, nc chunks each, cut into equal segments, one
// per CTA (to one chunk): B2 L2048 H80 took 179 us so and 245 with whole chains, B8 528 and 591. With at most one CTA per chain a segment is at least a chain
// long, so a chain spans two CTAs at most. A CTA first runs the head of the chain it
// ends in, then its whole chains, then the rest of the chain it begins in, which
// waits for the state that the CTA before has left in its first item: every
// head waits for nothing, so every wait ends, and is normally over before it begins.
struct Segments {
    int head, head_end, first, whole, rest, rest_start;  // chains (head and rest -1: none) and chunks
    __device__ void set(int64_t chains, int64_t nc) {
        const int64_t total = chains * nc, G = gridDim.x;
        const int64_t start = blockIdx.x * total / G, end = (blockIdx.x + 1) * total / G;
        const int64_t j0 = start / nc, j1 = (end - 1) / nc, cs = start % nc, ce = (end - 1) % nc + 1;
        head = rest = -1;
        head_end = rest_start = 0;
        if (ce < nc) head = (int)j1, head_end = (int)ce;
        const int64_t f0 = cs > 0 ? j0 + 1 : j0, f1 = ce < nc ? j1 - 1 : j1;
        first = (int)f0;
        whole = f1 >= f0 ? (int)(f1 - f0 + 1) : 0;
        if (cs > 0) rest = (int)j0, rest_start = (int)cs;
    }
    __device__ __forceinline__ int items() const { return (head >= 0) + whole + (rest >= 0); }
    // chain and chunks [c0, c1) of item k
    __device__ __forceinline__ void item(int k, int nc, int &chain, int &c0, int &c1) const {
        if (head >= 0) {
            if (k == 0) {
                chain = head, c0 = 0, c1 = head_end;
                return;
            }
            --k;
        }
        if (k < whole)
            chain = first + k, c0 = 0, c1 = nc;
        else
            chain = rest, c0 = rest_start, c1 = nc;
    }
};

// The flag of a chain whose state is handed on: set by one thread after the others' stores, waited for (bounded).
__device__ __forceinline__ void flag_set(int *f) { asm volatile("st.release.gpu.global.b32 [%0], 1;" ::"l"(f) : "memory"); }
static __device__ __noinline__ void flag_wait(const int *f, volatile int *fail) {
    const uint64_t t0 = tc::global_ns();
    for (;;) {
        int v;
        asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(f) : "memory");
        if (v || *fail) return;
        if (tc::global_ns() - t0 > kWaitNs) {
            *fail = 1;
            return;
        }
    }
}

// Launches a chain kernel: one CTA per chain, or one per SM where there are more
// chains; those wait on one another, so the launch is cooperative then.
template <typename Params>
cudaError_t launch_chains(void (*kern)(Params), const Params &p, int64_t chains, int64_t nc, int threads, size_t smem,
                          cudaStream_t stream) {
    const int64_t grid = imin<int64_t>(chains, sm_count(1));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (chains * nc % grid == 0 && chains % grid == 0) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
    } else {
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Byte offset of 16-byte piece `pc` of row `row` of a tile of 64 bf16 columns in the 128-byte swizzle.
__device__ __forceinline__ uint32_t piece(int row, int pc) { return (uint32_t)(row * 128 + ((pc ^ (row & 7)) << 4)); }

}  // namespace delta
}  // namespace ssd
