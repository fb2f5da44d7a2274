// Gated linear recurrence, per sequence and channel, with a weight lam per channel:
//     w_t = c softplus(lam) sigmoid(r_t)     a_t = exp(-w_t)     b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
//     h_t = a_t h_{t-1} + b_t                y_t = h_t
// its backward, and one token of it over a pool of states; activations in 8 bits.
//
// A run of tokens acts on the state as h -> A h + H, A the product of its a and H its result from zero, so runs are formed apart
// and joined in order. A lane has two channels; a warp holds 64 channels of a run in registers; the warps of a block lie one
// behind the other in time, 64 tokens in all, and so do the blocks of a cluster. A warp forms a, b and its (A, H); the warps of a
// block join theirs in shared memory, each block sends its own to the others of its cluster, and every warp goes over its run
// again from the state that enters it. The cluster then takes the next tokens of the sequence, the state kept by all of its
// threads, then another tile. Blocks' tokens are always joined one block after the other, so the result depends neither on the
// cluster's size nor on the batch nor on the padding. Tokens past a sequence's end act as a = 1, b = 0.
//
// What costs a step is latency more than anything: of the special functions, of the joining. So a block is small and an SM holds
// four of them, each at another place of its step (with 128 tokens a block and two an SM, B1 L65536 D1536 took 261 us where this took
// 242); nothing in a step waits for memory that was not asked for a step before; and the blocks meet on a barrier in shared memory
// that counts the bytes sent rather than on the cluster's, which would have the sender wait for everything it has written (B8 L2048
// D5120: 193 us so, 176 without). The whole forward: B8 L2048 D5120 in bf16 123 us, 5.4 TB/s; one block that walks a
// sequence alone, with plain loads, took 521.
#include <cooperative_groups.h>

#include <type_traits>

#include "gated_linear.cuh"
#include "launch.h"
#include "tc_host.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace linear {

constexpr int kTile = 64;                 // channels of a block, two a lane
constexpr int kFwdRun = kGroup;           // tokens of a warp in the forward: a group of the 8-bit values
constexpr int kFwdWarps = kState / kFwdRun;
constexpr int kBwdRun = 8;                // and in the backward, which keeps five numbers a token rather than two
constexpr int kBwdWarps = kState / kBwdRun;
constexpr int kMaxCluster = 16;
constexpr int kPackWarps = 8;
constexpr int kShort = kGroup, kShortThreads = 128;  // tokens of the kernels for short sequences, a run of the forward

// Blocks that an SM holds, by registers and shared memory.
template <typename T, bool PACK> __host__ __device__ constexpr int fwd_per_sm() { return sizeof(T) == 4 ? 2 : PACK ? 3 : 4; }
template <typename T> __host__ __device__ constexpr int bwd_per_sm() { return sizeof(T) == 4 ? 1 : 2; }

// ------------------------------------------------------- tiles in shared memory
// WIDE, for rows that begin at a multiple of 16 bytes: a thread has the TMA bring the block's tiles and a lane of each warp
// has it take the results away. Otherwise each warp fetches the rows of its own run: a pair of channels a lane where D is EVEN; else,
// and bytes always, by 4-byte copies of the aligned words around each row, of those at the tensor's end and the tile's only the bytes
// that belong to the tensor; a row then begins up to 3 bytes into its first word.
template <typename T, bool WIDE> struct Row {
    static constexpr int kPitch = kTile * (int)sizeof(T) + (WIDE || sizeof(T) == 4 ? 0 : 4);
};
__device__ __forceinline__ void copy4(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
template <int BYTES> __device__ __forceinline__ void copy_pair(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Rows 0..n-1 of `cols` elements from `base` on, which lie D apart, R at most. EVEN: of pairs of elements.
template <typename T, int PITCH, int R, bool EVEN>
__device__ __forceinline__ void fetch_rows(unsigned char *to, const T *base, int n, int cols, int64_t D, int lane) {
    const uint32_t dst = tc::smem_u32(to);
    if constexpr (EVEN && sizeof(T) > 1) {  // a pair a lane
        if (2 * lane >= cols) return;
        const T *from = base + 2 * lane;
#pragma unroll
        for (int t = 0; t < R; ++t, from += D)
            if (t < n) copy_pair<2 * sizeof(T)>(dst + t * PITCH + lane * 2 * (int)sizeof(T), from);
    } else {
        const int have = cols * (int)sizeof(T);
        const unsigned char *from = reinterpret_cast<const unsigned char *>(base);
#pragma unroll 4
        for (int t = 0; t < n; ++t, from += D * sizeof(T)) {
            const int off = (int)(reinterpret_cast<uintptr_t>(from) & 3);
            const unsigned char *word = from - off;
#pragma unroll
            for (int w = 0; w < (kTile * (int)sizeof(T) + 127 + (sizeof(T) == 4 ? 0 : 3)) / 128; ++w) {
                const int at = 4 * lane + 128 * w, left = off + have - at;
                if (left > 0) copy4(dst + t * PITCH + at, word + at, left < 4 ? left : 4);
            }
        }
    }
}
// Bytes that a row from `at` elements on begins into its first word.
template <typename T, bool WIDE, bool EVEN> __device__ __forceinline__ int shift(const void *base, int64_t at) {
    return WIDE || sizeof(T) == 4 || (EVEN && sizeof(T) == 2) ? 0 : (int)((reinterpret_cast<uintptr_t>(base) + (uintptr_t)at * sizeof(T)) & 3);
}
// The two channels of a lane in a row.
template <typename T, bool EVEN> __device__ __forceinline__ Raw<T, 2> row_pair(const unsigned char *row, int off, int lane, bool both) {
    Raw<T, 2> r;
    const T *p = reinterpret_cast<const T *>(row + off) + 2 * lane;
    if constexpr (EVEN) {
        r.word = *reinterpret_cast<const decltype(r.word) *>(p);
    } else {
        r.v[0] = p[0], r.v[1] = both ? p[1] : p[0];
    }
    return r;
}
template <typename T> __device__ __forceinline__ Raw<T, 2> rounded(uint64_t v) {
    Raw<T, 2> r;
    float v0, v1;
    un2(v, v0, v1);
    r.v[0] = from_f32<T>(v0), r.v[1] = from_f32<T>(v1);
    return r;
}
// The same two channels in global memory; `one` and `both`: whether they exist.
template <typename T, bool EVEN> __device__ __forceinline__ void store_pair(T *p, const Raw<T, 2> &r, bool one, bool both) {
    if constexpr (EVEN) {
        if (one) store<T, 2>(p, r);
    } else {
        if (one) p[0] = r.v[0];
        if (both) p[1] = r.v[1];
    }
}
// A lane's two channels of a warp's run, for the TMA to take away or to global memory at once.
template <typename T, bool WIDE, bool EVEN>
__device__ __forceinline__ void put_pair(unsigned char *row, T *p, const Raw<T, 2> &r, bool exists, bool one, bool both, int lane) {
    if constexpr (WIDE) {
        *reinterpret_cast<decltype(r.word) *>(row + 2 * sizeof(T) * lane) = r.word;
    } else {
        if (exists) store_pair<T, EVEN>(p, r, one, both);
    }
}

// ------------------------------------------------------------ runs, joined in order
// (A, H) of a lane's two channels: h -> A h + H.
struct alignas(16) Run2 {
    uint64_t a, h;
};
__device__ __forceinline__ uint64_t after(const Run2 &x, uint64_t h) { return fma2(x.a, h, x.h); }  // x, from h
__device__ __forceinline__ Run2 after(const Run2 &x, const Run2 &y) { return {mul2(x.a, y.a), fma2(y.a, x.h, y.h)}; }  // x, then y
__device__ __forceinline__ uint64_t unknown() { return f2(__uint_as_float(0x7fc00000u)); }
__device__ __forceinline__ Run2 nothing() { return {f2(1.f), f2(-0.f)}; }  // -0: what is added to zero of either sign and leaves it

// A step of a block: the tile and the tokens of a sequence that it is at. A thread works it out two steps ahead.
struct alignas(16) Step {
    int64_t base;          // of the block's first token and the tile's first channel in [B, L, D]
    int32_t b, t0;         // sequence; the block's first token (below 0: it has none)
    int32_t live, rows;    // of the block's kState tokens, those that count and those that exist
    int32_t c0, cols;      // the tile's first channel, its channels; 0: no more work
    int32_t begins, ends;  // whether the cluster begins, ends the sequence and tile
    int32_t brief;         // whether the sequence has kShort tokens or fewer
};
struct Walk {
    uint32_t item, items, tiles, clusters;
    int64_t first;            // token of the cluster
    int64_t start, stop, by;  // a sequence's steps: from token `start` by `by` until past `stop`
    int ours;                 // the block's first token from the cluster's
    __device__ __forceinline__ Step next(const LinearArgs &p) {
        Step s{};
        if (item >= items) return s;
        const uint32_t b = item / tiles;
        const int64_t t0 = first + ours;
        s.b = (int32_t)b, s.t0 = (int32_t)t0, s.c0 = (int32_t)(item - b * tiles) * kTile;
        s.cols = (int32_t)imin<int64_t>(kTile, p.D - s.c0);
        s.base = (b * p.L + t0) * p.D + s.c0;
        const int64_t n = seq_len(p.seqlens, b, p.L);
        s.brief = n <= kShort;
        if (t0 >= 0) {
            s.live = (int32_t)imin<int64_t>(kState, imax<int64_t>(0, n - t0));
            s.rows = (int32_t)imin<int64_t>(kState, imax<int64_t>(0, p.L - t0));
        }
        s.begins = first == start;
        first += by;
        s.ends = by > 0 ? first >= stop : first <= stop;
        if (s.ends) first = start, item += clusters;
        return s;
    }
};
// Of n tokens, those in the run of R from `place` on.
__device__ __forceinline__ int run_of(int R, int n, int place) { return max(0, min(R, n - place)); }

// The blocks of a cluster exchange a Run2 a lane: each sends its own to all of them, and the bytes count down the receiver's
// barrier. Two of each, taken in turn: a block sends for a step once all of its warps have read the one before.
struct Exchange {
    Run2 block[2][kMaxCluster][32];
    uint64_t bar[2];
};
// A thread whose wait has run out (`alive` false) goes on through its steps with the other threads of its block, but waits, arms
// barriers, has tiles brought and, from the next step on, sends no more: what it does not send has the other blocks' waits run out in
// turn, and no barrier counts a step's bytes for another's. A wait for the cluster's runs is twice as long as one for tiles, so that a
// block whose tiles do not come can still say so: its run is NaN, which goes on to all that comes after it, and its groups in 8 bits
// are marked as NaN too. See leave() for the end.
#ifdef SSD_DEBUG_BOUNDS
constexpr uint64_t kGiveUpNs = 100000000ull;
__device__ int g_withhold[3];  // has waits run out: kTiles, kRuns or 0, and the rank and step whose barrier counts bytes that nothing sends
__device__ __forceinline__ uint32_t withheld(int what, int rank, int step) {
    return g_withhold[0] == what && g_withhold[1] == rank && g_withhold[2] == step ? 16u : 0u;
}
#else
constexpr uint64_t kGiveUpNs = 1000000000ull;
__device__ __forceinline__ uint32_t withheld(int, int, int) { return 0; }
#endif
constexpr int kTiles = 1, kRuns = 2;
constexpr uint64_t kUnderWayNs = 100000ull;
__device__ unsigned long long g_gave_up;  // threads whose wait ran out on this device

// Barriers ready in all blocks of the cluster. `tiles`: that of the TMA's tiles.
__device__ __forceinline__ void exchange_init(Exchange &x, uint64_t *tiles, int blocks) {
    if (threadIdx.x == 0) {
        tc::mbar_init(&x.bar[0], 1);
        tc::mbar_init(&x.bar[1], 1);
        tc::mbar_init(tiles, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    if (blocks > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}
__device__ __forceinline__ void exchange_expect(Exchange &x, int step, int rank, int blocks) {
    tc::mbar_arrive_expect_tx(&x.bar[step & 1], blocks * 32 * (uint32_t)sizeof(Run2) + withheld(kRuns, rank, step));
}
// To the ranks first, first + every, ...
__device__ __forceinline__ void exchange_send(Exchange &x, int step, int rank, int blocks, int first, int every, int lane, const Run2 &own) {
    const uint32_t slot = tc::smem_u32(&x.block[step & 1][rank][lane]), bar = tc::smem_u32(&x.bar[step & 1]);
    uint32_t r0, r1, r2, r3;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r0), "=r"(r1) : "l"(own.a));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r2), "=r"(r3) : "l"(own.h));
    for (int j = first; j < blocks; j += every)
        asm volatile(
            "{\n\t.reg .b32 to, at;\n\t"
            "mapa.shared::cluster.u32 to, %0, %2;\n\t"
            "mapa.shared::cluster.u32 at, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [to], {%3, %4, %5, %6}, [at];\n\t}" ::"r"(slot),
            "r"(bar), "r"(j), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
            : "memory");
}
// False, now and from then on, where what a barrier counts has not come in that time.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, bool alive, uint64_t ns = kGiveUpNs) {
    if (!alive) return false;
    if (tc::mbar_wait(bar, parity, ns)) return true;
    atomicAdd(&g_gave_up, 1ull);
    return false;
}
// The carry over a cluster's blocks up to this one; `carry` goes on to the next step. What was not told is not guessed: NaN.
__device__ __forceinline__ uint64_t exchange_receive(Exchange &x, int step, int rank, int blocks, int lane, bool &alive, uint64_t &carry) {
    alive = wait_for(&x.bar[step & 1], (step >> 1) & 1, alive, 2 * kGiveUpNs);
    if (!alive) carry = unknown();
    uint64_t e = carry;
#pragma unroll 4
    for (int j = 0; j < blocks; ++j) {
        if (j == rank) e = carry;
        carry = after(x.block[step & 1][j][lane], carry);
    }
    return e;
}

// A block's end. Shared memory is given up once nothing more can come to it: a first thread whose waits all ended knows that all has come.
// One whose wait ran out sees to the tiles that it had brought, for as long again (`parity`: of the last that it has not seen come); the
// others' runs are on their way for microseconds once all blocks are here.
template <bool WIDE> __device__ __forceinline__ void leave(uint64_t *tiles, uint32_t parity, int blocks, bool alive) {
    if (WIDE && threadIdx.x == 0 && !alive) tc::mbar_wait(tiles, parity, kGiveUpNs);
    if (blocks > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    }
    if (threadIdx.x == 0 && !alive)
        for (const uint64_t since = tc::global_ns(); tc::global_ns() - since < kUnderWayNs;) {}
}

// ------------------------------------------------------------------ forward
// Bound by the latency of a step at the 16 warps that an SM's registers hold, which keep neither HBM (8 bytes a token and channel in
// bf16; B4 L2048 D5120 55 % of its peak) nor the issue slots (57 %) busy; B8 L2048 D5120 123 us, where the same tiles moved without
// arithmetic take 104. Instructions are time all the same: so two channels each where there is one for it. Runs of 16 tokens are what
// the registers of those warps hold (a and b of each: 64 of 128). With the 8 bits written too, B4 L2048 D5120: 112 us.
template <typename T, bool WIDE, bool PACK> struct alignas(128) FwdShared {
    static constexpr int kPitch = Row<T, WIDE>::kPitch;
    alignas(128) unsigned char in[3][kState][kPitch];  // x, r, i: brought anew once the block has its a and b
    alignas(128) unsigned char y[WIDE ? kState : 1][kTile * sizeof(T)];
    alignas(128) unsigned char q[PACK && WIDE ? 3 * kState : 1][kTile];  // run by run: x, r, i
    alignas(16) float lam[kTile], init[kTile];
    Run2 run[2][kFwdWarps][32];  // in turn: a warp may be at its next run while another reads these
    Exchange exchange;
    Step step[4];
    Walk walk;  // the planner's alone: out of the registers of all
    uint64_t tiles;
};
struct FwdMaps {
    CUtensorMap x, r, i;  // boxes of 64 x 64
    CUtensorMap y, q;     // of a warp's run; q of all three in 8 bits
};

// A run's x, r and i (z 0, 1, 2) in 8 bits, to `out`, the run's place in FwdShared::q. ALL: every token of it counts. Not `alive`: what
// is in the tile is not known, and kept as NaN.
template <typename T, bool WIDE, bool EVEN, bool ALL, typename F>
__device__ __forceinline__ void leave_in_8_bits(const LinearArgs &p, const F &pair, unsigned char (*out)[kTile], const Step &s, int place, int live, int rows,
                                                int lane, bool alive) {
    constexpr int R = kFwdRun;
    const int64_t D = p.D;
    const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
        Raw<T, 2> w[R];
#pragma unroll
        for (int t = 0; t < R; ++t) w[t] = pair(z, t);
        uint32_t top0 = 0, top1 = 0;
        if constexpr (sizeof(T) == 2) {
            uint32_t top = 0;  // bf16 without its sign orders like a whole number: two at once
#pragma unroll
            for (int t = 0; t < R; ++t)
                if (ALL || t < live) top = __vmaxu2(top, w[t].word & 0x7fff7fffu);
            top0 = top << 16, top1 = top & 0xffff0000u;
        } else {
#pragma unroll
            for (int t = 0; t < R; ++t)
                if (ALL || t < live) top0 = max(top0, abs_bits(w[t].v[0])), top1 = max(top1, abs_bits(w[t].v[1]));
        }
        if (!alive) top0 = top1 = 0x7fc00000u;
        Raw<uint8_t, 2> code;
        code.v[0] = (uint8_t)scale_code(top0), code.v[1] = (uint8_t)scale_code(top1);
        const int64_t groups = (p.L + kGroup - 1) / kGroup;
        store_pair<uint8_t, EVEN>(p.scales + ((z * p.B + s.b) * groups + (s.t0 + place) / kGroup) * D + s.c0 + 2 * lane, code, one, both);
        const uint64_t inv = f2(inverse_scale(code.v[0]), inverse_scale(code.v[1]));
        const uint32_t mask = (code.v[0] == 255 ? 0u : 0xffu) | (code.v[1] == 255 ? 0u : 0xff00u);
        int8_t *values = p.values + (z * p.B * p.L + place) * D + s.base + 2 * lane;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            float q0, q1;
            un2(fma2(pair_of(w[t]), inv, f2(kToWhole)), q0, q1);
            Raw<int8_t, 2> q;
            q.word = (uint16_t)(ALL || t < live ? __byte_perm(__float_as_uint(q0), __float_as_uint(q1), 0x0040) & mask : 0u);
            put_pair<int8_t, WIDE, EVEN>(out[WIDE ? z * R + t : 0], values + t * D, q, t < rows, one, both, lane);
        }
    }
}

template <typename T, bool WIDE, bool EVEN, bool PACK>
__global__ void __launch_bounds__(32 * kFwdWarps, fwd_per_sm<T, PACK>()) linear_fwd_kernel(LinearArgs p, const __grid_constant__ FwdMaps maps) {
    namespace cg = cooperative_groups;
    pdl_wait();
    constexpr int R = kFwdRun, PITCH = Row<T, WIDE>::kPitch;
    extern __shared__ __align__(128) unsigned char raw_smem[];
    FwdShared<T, WIDE, PACK> &sh = *reinterpret_cast<FwdShared<T, WIDE, PACK> *>(raw_smem);
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
    const int64_t D = p.D, L = p.L;
    const int place = warp * R;  // of this warp's run, from the block's first token
    const bool planner = threadIdx.x == 32 * (warps - 1);
    if (planner) {
        Walk walk{};
        walk.tiles = (uint32_t)((D + kTile - 1) / kTile), walk.items = (uint32_t)p.B * walk.tiles;  // below 2^31
        walk.item = blockIdx.x / (uint32_t)blocks, walk.clusters = gridDim.x / (uint32_t)blocks;
        walk.stop = L, walk.by = blocks * kState, walk.ours = rank * kState;
        sh.step[0] = walk.next(p), sh.step[1] = walk.next(p);
        sh.walk = walk;
    }
    exchange_init(sh.exchange, &sh.tiles, blocks);

    bool alive = true;
    // Has the next step's tiles brought, by one thread: the others of its warp, and the other warps, wait for the exchange.
    auto bring = [&](int step) {
        if constexpr (WIDE) {
            if (threadIdx.x != 0 || !alive) return;
            const Step s = sh.step[step & 3];
            if (s.cols > 0 && (s.begins || s.live > 0)) {
                const uint32_t some = s.cols * (uint32_t)sizeof(float);
                tc::mbar_arrive_expect_tx(&sh.tiles, (s.live > 0 ? 3 * kState * PITCH : 0) + (s.begins ? (p.init ? 2 : 1) * some : 0) + withheld(kTiles, rank, step));
                if (s.live > 0) {
                    tc::tma_load_3d(sh.in[0], &maps.x, &sh.tiles, s.c0, s.t0, s.b);
                    tc::tma_load_3d(sh.in[1], &maps.r, &sh.tiles, s.c0, s.t0, s.b);
                    tc::tma_load_3d(sh.in[2], &maps.i, &sh.tiles, s.c0, s.t0, s.b);
                }
                if (s.begins) {
                    tc::bulk_load(sh.lam, p.lam + s.c0, some, &sh.tiles);
                    if (p.init) tc::bulk_load(sh.init, p.init + s.b * D + s.c0, some, &sh.tiles);
                }
            }
        } else {
            const Step s = sh.step[step & 3];
            const int live = s.cols > 0 ? run_of(R, s.live, place) : 0;
            const int64_t at = s.base + place * D;
            fetch_rows<T, PITCH, R, EVEN>(sh.in[0][place], (const T *)p.x + at, live, s.cols, D, lane);
            fetch_rows<T, PITCH, R, EVEN>(sh.in[1][place], (const T *)p.r + at, live, s.cols, D, lane);
            fetch_rows<T, PITCH, R, EVEN>(sh.in[2][place], (const T *)p.i + at, live, s.cols, D, lane);
            copy_commit();
        }
    };
    bring(0);
    uint64_t carry = 0;
    Rate2 rate{};
    bool steep = false;
    uint32_t parity = 0;
    for (int step = 0;; ++step) {
        const Step s = sh.step[step & 3];
        if (s.cols == 0) break;
        const bool in_step = __all_sync(0xffffffffu, alive);  // with the cluster's other blocks: its run is sent, whatever comes of the tiles
        if (threadIdx.x == 0 && in_step) exchange_expect(sh.exchange, step, rank, blocks);
        const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
        const int64_t at = s.base + place * D + 2 * lane;
        const int live = run_of(R, s.live, place), rows = run_of(R, s.rows, place);  // tokens that count, that exist
        const int t0 = s.t0 + place;                                                  // of the run, where it exists
        if constexpr (WIDE) {
            if (s.begins || s.live > 0) alive = wait_for(&sh.tiles, parity, alive), parity ^= (uint32_t)alive;
        } else {
            copy_wait();
            __syncwarp();
        }
        if (s.begins) {
            const int64_t c = s.c0 + 2 * lane;
            float k0, k1;
            if constexpr (WIDE) {
                k0 = sh.lam[2 * lane], k1 = sh.lam[2 * lane + 1];
                carry = p.init ? f2(sh.init[2 * lane], sh.init[2 * lane + 1]) : 0;
            } else {
                k0 = one ? p.lam[c] : 0.f, k1 = both ? p.lam[c + 1] : 0.f;
                carry = p.init ? f2(one ? p.init[s.b * D + c] : 0.f, both ? p.init[s.b * D + c + 1] : 0.f) : 0;
            }
            k0 = p.c * softplus(k0), k1 = p.c * softplus(k1);
            rate = Rate2::of(k0, k1);
            steep = __any_sync(0xffffffffu, (one && !(k0 < kSteep)) || (both && !(k1 < kSteep)));
        }
        auto pair = [&](int z, int t) {
            const void *base = z == 0 ? p.x : z == 1 ? p.r : p.i;
            return row_pair<T, EVEN>(sh.in[z][place + t], shift<T, WIDE, EVEN>(base, at - 2 * lane + t * D), lane, both);
        };
        uint64_t a[R], h[R];
        Run2 own;
        uint64_t sum = 0;
        auto tokens = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            own = nothing();
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const Gates2 g = gates2<T, FAST, false>(pair_of(pair(1, t)), pair_of(pair(2, t)), rate, sum);
                a[t] = g.a;
                h[t] = mul2(g.f, pair_of(pair(0, t)));
                if (!FAST && t >= live) a[t] = f2(1.f), h[t] = nothing().h;
                own = after(own, {a[t], h[t]});
            }
        };
        bool fast = live == R && !steep && !s.brief;  // brief: the gates as linear_fwd_short_kernel has them
        if (fast) {
            tokens(std::true_type{});
            fast = !__any_sync(0xffffffffu, is_low(sum, one, both));
        }
        if (!fast) tokens(std::false_type{});
        if (!alive) own = {unknown(), unknown()};
        sh.run[step & 1][warp][lane] = own;
        if constexpr (WIDE) {  // the TMA has read what it was given of the step before
            if (lane == 0) tc::bulk_wait_read_all();
            __syncwarp();
        }
        if constexpr (PACK) {
            if (rows > 0) {
                auto *out = &sh.q[WIDE ? 3 * place : 0];
                if (live == R)
                    leave_in_8_bits<T, WIDE, EVEN, true>(p, pair, out, s, place, live, rows, lane, alive);
                else
                    leave_in_8_bits<T, WIDE, EVEN, false>(p, pair, out, s, place, live, rows, lane, alive);
                if constexpr (WIDE) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tc::tma_store_4d(&maps.q, out, s.c0, t0, s.b, 0);
                }
            }
        }
        __syncthreads();
        // the block's runs before this one, and all of them: every warp joins them, and sends to other blocks
        Run2 before = nothing(), all = nothing();
#pragma unroll
        for (int w = 0; w < kFwdWarps; ++w) {
            if (w == warp) before = all;
            if (w < warps) all = after(all, sh.run[step & 1][w][lane]);
        }
        if (in_step) exchange_send(sh.exchange, step, rank, blocks, warp, warps, lane, all);
        bring(step + 1);  // behind the sending, which the others wait for
        if (planner) sh.step[(step + 2) & 3] = sh.walk.next(p);
        uint64_t e = after(before, exchange_receive(sh.exchange, step, rank, blocks, lane, alive, carry));  // the state that enters this run
        if (warp == 0 && rows > 0 && p.states)
            store_pair<float, EVEN>(p.states + (s.b * ((L + kState - 1) / kState) + s.t0 / kState) * D + s.c0 + 2 * lane, rounded<float>(e), one, both);
        if (p.y && rows > 0) {
            auto results = [&](auto whole) {
#pragma unroll
                for (int t = 0; t < R; ++t) {
                    e = fma2(a[t], e, h[t]);
                    put_pair<T, WIDE, EVEN>(sh.y[WIDE ? place + t : 0], (T *)p.y + at + t * D, rounded<T>(decltype(whole)::value || t < live ? e : 0), t < rows,
                                      one, both, lane);
                }
            };
            if (live == R) results(std::true_type{}); else results(std::false_type{});
            if constexpr (WIDE) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::tma_store_3d(&maps.y, sh.y[place], s.c0, t0, s.b);
            }
        }
        if (WIDE && lane == 0) tc::bulk_commit();
        if (s.ends && rank == 0 && warp == 0 && p.final_state)
            store_pair<float, EVEN>(p.final_state + s.b * D + s.c0 + 2 * lane, rounded<float>(carry), one, both);
    }
    if constexpr (WIDE) {
        if (lane == 0) tc::bulk_wait_all();
    } else {
        copy_wait();
    }
    leave<WIDE>(&sh.tiles, parity, blocks, alive);
}

// A sequence of no tokens: its state goes through.
__global__ void __launch_bounds__(256) linear_keep_kernel(const float *init, float *final_state, int64_t n) {
    pdl_enter();
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j < n) final_state[j] = init ? init[j] : 0.f;
}

// ----------------------------------------------------------------- backward
// dh_t = dy_t + m_{t+1}, m_t = a_t dh_t (m behind the last token the gradient of the final state): the same kind of recurrence,
// backwards, a run acting as m -> A m + M. With f and g as in gates2 and grad_ratio, and psi_t = w_t dL/dw_t:
//     b = f x     dx = dh f     di = dh b (1 - iota)     psi = dh (g b - a w h_{t-1})     dr = psi (1 - rho)
//     dlam = sigmoid(lam) / softplus(lam) sum psi
// (psi rather than dL/dw, which has 1 / sqrt(1 - a^2): w over it goes to zero with w.) h_{t-1} is formed again from the state that
// enters each kState tokens, which are a block's; the warps and blocks lie one before the other in time.
// Bound by latency at 16 warps an SM, with 60 % of the issue slots and half of HBM's peak in use (14 bytes a token and channel in bf16, 11
// from 8 bits): B4 L2048 D5120 146 us, 4.0 TB/s, and 155 from 8 bits. Five numbers a token (a, b, f, e^-r and d) wait in registers for the
// exchange: so runs of 8 tokens. The 128 registers that two blocks an SM leave spill 4 to 52 bytes a thread, most where rows go by words.
template <typename T, bool WIDE, bool PACK> struct alignas(128) BwdShared {
    static constexpr int kPitch = PACK ? Row<int8_t, WIDE>::kPitch : Row<T, WIDE>::kPitch;
    alignas(128) unsigned char in[3][kState][kPitch];                     // x, r, i
    alignas(128) unsigned char dy[2][kState][Row<T, WIDE>::kPitch];       // read again at the end of a step
    alignas(128) unsigned char out[WIDE ? 3 * kState : 1][kTile * sizeof(T)];
    alignas(128) unsigned char scale[3][kState / kGroup][Row<uint8_t, WIDE>::kPitch];
    alignas(16) float lam[kTile], last[kTile], state[kTile];
    Run2 run[2][kBwdWarps][32];
    uint64_t h[2][kBwdWarps][32], sum[kBwdWarps][32];
    Exchange exchange;
    Step step[4];
    Walk walk;  // the planner's alone: out of the registers of all
    uint64_t tiles;
};
struct BwdMaps {
    CUtensorMap x, r, i, dy;  // boxes of 64 x 64
    CUtensorMap q, scale;     // x, r and i in 8 bits at once, and 4 groups of their scales
    CUtensorMap dx, dr, di;   // of a warp's run
};

// The two channels of a lane in 8 bits, as numbers: byte v as 2^23 + 128 + v, less that, exactly; times the scale.
__device__ __forceinline__ uint64_t from_8(uint32_t two, uint64_t scale) {
    const uint32_t v = two ^ 0x8080u;
    const uint64_t n = f2(__uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7441)));
    return mul2(add2(n, f2(-8388736.f)), scale);
}

template <typename T, bool WIDE, bool EVEN, bool PACK>
__global__ void __launch_bounds__(32 * kBwdWarps, bwd_per_sm<T>()) linear_bwd_kernel(LinearBwdArgs p, const __grid_constant__ BwdMaps maps) {
    namespace cg = cooperative_groups;
    pdl_wait();
    constexpr int R = kBwdRun, PITCH = BwdShared<T, WIDE, PACK>::kPitch, DY = Row<T, WIDE>::kPitch, SC = Row<uint8_t, WIDE>::kPitch;
    extern __shared__ __align__(128) unsigned char raw_smem[];
    BwdShared<T, WIDE, PACK> &sh = *reinterpret_cast<BwdShared<T, WIDE, PACK> *>(raw_smem);
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
    const int64_t D = p.f.D, L = p.f.L, chunks = (L + kState - 1) / kState, groups = (L + kGroup - 1) / kGroup;
    const int64_t plane = p.f.B * L * D, scales = p.f.B * groups * D;
    // Rank 0 and warp 0 have the latest tokens. A step begins a cluster's chunks before the one it came from, at the start of a
    // sequence before its first token.
    const int place = (warps - 1 - warp) * R;  // of this warp's run, from the block's first token
    const bool planner = threadIdx.x == 32 * (warps - 1);
    if (planner) {
        Walk walk{};
        walk.tiles = (uint32_t)((D + kTile - 1) / kTile), walk.items = (uint32_t)p.f.B * walk.tiles;  // below 2^31
        walk.item = blockIdx.x / (uint32_t)blocks, walk.clusters = gridDim.x / (uint32_t)blocks;
        walk.by = -(int64_t)blocks * kState, walk.stop = walk.by, walk.ours = (blocks - 1 - rank) * kState;
        walk.first = walk.start = (chunks - blocks) * kState;
        sh.step[0] = walk.next(p.f), sh.step[1] = walk.next(p.f);
        sh.walk = walk;
    }
    exchange_init(sh.exchange, &sh.tiles, blocks);

    bool alive = true;
    auto bring = [&](int step) {  // as in the forward
        if constexpr (WIDE) {
            if (threadIdx.x != 0 || !alive) return;
            const Step s = sh.step[step & 3];
            if (s.cols > 0 && (s.begins || s.live > 0)) {
                const uint32_t some = s.cols * (uint32_t)sizeof(float);
                tc::mbar_arrive_expect_tx(&sh.tiles, (s.live > 0 ? 3 * kState * PITCH + kState * DY + some + (PACK ? 3 * (kState / kGroup) * SC : 0) : 0) +
                                                         (s.begins ? (p.dfinal ? 2 : 1) * some : 0) + withheld(kTiles, rank, step));
                if (s.live > 0) {
                    if constexpr (PACK) {
                        tc::tma_load_4d(sh.in, &maps.q, &sh.tiles, s.c0, s.t0, s.b, 0);
                        tc::tma_load_4d(sh.scale, &maps.scale, &sh.tiles, s.c0, s.t0 / kGroup, s.b, 0);
                    } else {
                        tc::tma_load_3d(sh.in[0], &maps.x, &sh.tiles, s.c0, s.t0, s.b);
                        tc::tma_load_3d(sh.in[1], &maps.r, &sh.tiles, s.c0, s.t0, s.b);
                        tc::tma_load_3d(sh.in[2], &maps.i, &sh.tiles, s.c0, s.t0, s.b);
                    }
                    tc::tma_load_3d(sh.dy[step & 1], &maps.dy, &sh.tiles, s.c0, s.t0, s.b);
                    tc::bulk_load(sh.state, p.f.states + (s.b * chunks + s.t0 / kState) * D + s.c0, some, &sh.tiles);
                }
                if (s.begins) {
                    tc::bulk_load(sh.lam, p.f.lam + s.c0, some, &sh.tiles);
                    if (p.dfinal) tc::bulk_load(sh.last, p.dfinal + s.b * D + s.c0, some, &sh.tiles);
                }
            }
        } else {
            const Step s = sh.step[step & 3];
            const int live = s.cols > 0 ? run_of(R, s.live, place) : 0;
            const int64_t at = s.base + place * D;
            if (live > 0) {
                if constexpr (PACK) {
                    for (int z = 0; z < 3; ++z) {
                        fetch_rows<int8_t, PITCH, R, EVEN>(sh.in[z][place], p.f.values + z * plane + at, live, s.cols, D, lane);
                        if (place % kGroup == 0)  // one of a group's two runs brings its scale
                            fetch_rows<uint8_t, SC, 1, EVEN>(sh.scale[z][place / kGroup], p.f.scales + z * scales + (s.b * groups + (s.t0 + place) / kGroup) * D + s.c0, 1,
                                                    s.cols, D, lane);
                    }
                } else {
                    fetch_rows<T, PITCH, R, EVEN>(sh.in[0][place], (const T *)p.f.x + at, live, s.cols, D, lane);
                    fetch_rows<T, PITCH, R, EVEN>(sh.in[1][place], (const T *)p.f.r + at, live, s.cols, D, lane);
                    fetch_rows<T, PITCH, R, EVEN>(sh.in[2][place], (const T *)p.f.i + at, live, s.cols, D, lane);
                }
                fetch_rows<T, DY, R, EVEN>(sh.dy[step & 1][place], (const T *)p.dy + at, live, s.cols, D, lane);
            }
            copy_commit();
        }
    };
    bring(0);
    uint64_t carry = 0, sum = 0;
    Rate2 rate{};
    bool steep = false;
    uint32_t parity = 0;
    for (int step = 0;; ++step) {
        const Step s = sh.step[step & 3];
        if (s.cols == 0) break;
        const bool in_step = __all_sync(0xffffffffu, alive);  // with the cluster's other blocks: its run is sent, whatever comes of the tiles
        if (threadIdx.x == 0 && in_step) exchange_expect(sh.exchange, step, rank, blocks);
        const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
        const int64_t at = s.base + place * D + 2 * lane;
        const int live = run_of(R, s.live, place), rows = run_of(R, s.rows, place);  // tokens that count, that exist
        const int t0 = s.t0 + place;                                                  // of the run, where it exists
        if constexpr (WIDE) {
            if (s.begins || s.live > 0) alive = wait_for(&sh.tiles, parity, alive), parity ^= (uint32_t)alive;
        } else {
            copy_wait();
            if (PACK) __syncthreads(); else __syncwarp();  // scales are shared by two warps
        }
        const int64_t c = s.c0 + 2 * lane;
        if (s.begins) {
            float k0, k1;
            if constexpr (WIDE) {
                k0 = sh.lam[2 * lane], k1 = sh.lam[2 * lane + 1];
                carry = p.dfinal ? f2(sh.last[2 * lane], sh.last[2 * lane + 1]) : 0;
            } else {
                k0 = one ? p.f.lam[c] : 0.f, k1 = both ? p.f.lam[c + 1] : 0.f;
                carry = p.dfinal ? f2(one ? p.dfinal[s.b * D + c] : 0.f, both ? p.dfinal[s.b * D + c + 1] : 0.f) : 0;
            }
            sum = 0;
            k0 = p.f.c * softplus(k0), k1 = p.f.c * softplus(k1);
            rate = Rate2::of(k0, k1);
            steep = __any_sync(0xffffffffu, (one && !(k0 < kSteep)) || (both && !(k1 < kSteep)));
        }
        uint64_t h = 0;  // the state that enters the block's tokens
        if (s.live > 0) {
            if constexpr (WIDE) {
                h = f2(sh.state[2 * lane], sh.state[2 * lane + 1]);
            } else {
                const float *state = p.f.states + (s.b * chunks + s.t0 / kState) * D + c;
                h = f2(one ? state[0] : 0.f, both ? state[1] : 0.f);
            }
        }
        uint64_t scale[3];
        if constexpr (PACK) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                const Raw<uint8_t, 2> code = row_pair<uint8_t, EVEN>(
                    sh.scale[z][place / kGroup], shift<uint8_t, WIDE, EVEN>(p.f.scales, z * scales + (s.b * groups + t0 / kGroup) * D + s.c0), lane, both);
                scale[z] = f2(scale_of(code.v[0]), scale_of(code.v[1]));
            }
        }
        auto value = [&](int z, int t) {
            if constexpr (PACK) {
                const Raw<int8_t, 2> q =
                    row_pair<int8_t, EVEN>(sh.in[z][place + t], shift<int8_t, WIDE, EVEN>(p.f.values, z * plane + at - 2 * lane + t * D), lane, both);
                return from_8(q.word, scale[z]);
            } else {
                const void *base = z == 0 ? p.f.x : z == 1 ? p.f.r : p.f.i;
                return pair_of(row_pair<T, EVEN>(sh.in[z][place + t], shift<T, WIDE, EVEN>(base, at - 2 * lane + t * D), lane, both));
            }
        };
        auto dy_of = [&](int t) {
            return pair_of(row_pair<T, EVEN>(sh.dy[step & 1][place + t], shift<T, WIDE, EVEN>(p.dy, at - 2 * lane + t * D), lane, both));
        };
        uint64_t a[R], b[R], f[R], er[R], d[R];  // er: e^-r, from which rho and 1 - rho are formed again
        Run2 own;    // of m, backwards
        uint64_t H;  // and of h, forwards; its A is the same
        uint64_t args = 0;
        auto tokens = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            H = 0;
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const Gates2 g = gates2<T, FAST, true>(value(1, t), value(2, t), rate, args);
                a[t] = g.a, f[t] = g.f, er[t] = g.er;
                b[t] = mul2(g.f, value(0, t));
                d[t] = mul2(b[t], g.not_iota);
                if (!FAST && t >= live) a[t] = f2(1.f), b[t] = 0;
                H = fma2(a[t], H, b[t]);
            }
            own = nothing();
#pragma unroll
            for (int t = R - 1; t >= 0; --t) {
                own.a = mul2(own.a, a[t]);
                own.h = mul2(a[t], add2(FAST || t < live ? dy_of(t) : 0, own.h));
            }
        };
        bool fast = live == R && !steep;
        if (fast) {
            tokens(std::true_type{});
            fast = !__any_sync(0xffffffffu, is_low(args, one, both));
        }
        if (!fast) tokens(std::false_type{});
        if (!alive) own = {unknown(), unknown()}, H = unknown();
        sh.run[step & 1][warp][lane] = own;
        sh.h[step & 1][warp][lane] = H;
        if constexpr (WIDE) {  // the TMA has read what it was given of the step before
            if (lane == 0) tc::bulk_wait_read_all();
        }
        __syncthreads();
        Run2 before = nothing(), all = nothing();
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            if (w == warp) before = all;
            all = after(all, sh.run[step & 1][w][lane]);
        }
        if (in_step) exchange_send(sh.exchange, step, rank, blocks, warp, warps, lane, all);
        bring(step + 1);  // behind the sending, which the others wait for
        if (planner) sh.step[(step + 2) & 3] = sh.walk.next(p.f);
        // h over the earlier runs (the later warps') to this one; then b becomes what multiplies dh in psi, and er 1 - rho
#pragma unroll 1
        for (int w = warps - 1; w > warp; --w) h = fma2(sh.run[step & 1][w][lane].a, h, sh.h[step & 1][w][lane]);
#pragma unroll
        for (int t = 0; t < R; ++t) {
            float u0, u1;
            un2(add2(er[t], f2(1.f)), u0, u1);
            const uint64_t rho = f2(rcp_approx(u0), rcp_approx(u1)), w2 = mul2(rho, rate.twice), g = grad_ratio(w2, a[t], steep);
            const uint64_t factor = fma2(mul2(mul2(a[t], w2), f2(-0.5f)), h, mul2(g, b[t]));
            h = fma2(a[t], h, b[t]);
            b[t] = factor;
            er[t] = mul2(er[t], rho);
        }
        uint64_t m = after(before, exchange_receive(sh.exchange, step, rank, blocks, lane, alive, carry));  // from the later runs
        if (rows > 0) {
            auto results = [&](auto whole) {
                constexpr bool ALL = decltype(whole)::value;
#pragma unroll
                for (int t = R - 1; t >= 0; --t) {
                    const uint64_t dh = add2(m, ALL || t < live ? dy_of(t) : 0), psi = mul2(dh, b[t]);
                    const uint64_t v[3] = {mul2(dh, f[t]), mul2(psi, er[t]), mul2(dh, d[t])};
                    if (ALL || t < live) sum = add2(sum, psi);
                    m = mul2(a[t], dh);
#pragma unroll
                    for (int z = 0; z < 3; ++z)
                        put_pair<T, WIDE, EVEN>(sh.out[WIDE ? z * kState + place + t : 0], (T *)(z == 0 ? p.dx : z == 1 ? p.dr : p.di) + at + t * D,
                                          rounded<T>(ALL || t < live ? v[z] : 0), t < rows, one, both, lane);
                }
            };
            if (live == R) results(std::true_type{}); else results(std::false_type{});
            if constexpr (WIDE) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_3d(&maps.dx, sh.out[place], s.c0, t0, s.b);
                    tc::tma_store_3d(&maps.dr, sh.out[kState + place], s.c0, t0, s.b);
                    tc::tma_store_3d(&maps.di, sh.out[2 * kState + place], s.c0, t0, s.b);
                    tc::bulk_commit();
                }
            }
        }
        if (s.ends) {
            sh.sum[warp][lane] = sum;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < warps; ++w) sum = add2(sum, sh.sum[w][lane]);
                store_pair<float, EVEN>(p.part + ((int64_t)s.b * blocks + rank) * D + c, rounded<float>(sum), one, both);
                if (rank == 0 && p.dinit) store_pair<float, EVEN>(p.dinit + s.b * D + c, rounded<float>(carry), one, both);
            }
        }
    }
    if constexpr (WIDE) {
        if (lane == 0) tc::bulk_wait_all();
    } else {
        copy_wait();
    }
    leave<WIDE>(&sh.tiles, parity, blocks, alive);
}

// --------------------------------------------------------- short sequences
// Up to kShort tokens, a run of the kernels above: a thread goes over V channels of a whole sequence alone, its tokens in registers;
// there is nothing to join, and the number of sequences is what fills the device (forward B64 L16 D2560 10.4 us, 14.7 as above; B256 L1
// D5120 18 and 86; backward 20 and 31, 53 and 225; a single sequence of 16 tokens 4.7 and 4.0, its backward 8.6 and 6.6: the rule goes
// by the padded length alone, so that neither results nor times of a sequence hang on how many there are). 64 sequences of 17 tokens
// take 21 and 39 us. The forward gives bitwise what the kernel above gives a sequence of as many tokens in a batch padded to more:
// the gates of its slow form, which `Step::brief` has it take there too, and the final state from the run's (A, H).

template <typename T, int V> __device__ __forceinline__ uint64_t two_of(const Raw<T, V> &w) { return f2(to_f32(w.v[0]), to_f32(w.v[V - 1])); }
template <int V> __device__ __forceinline__ uint64_t two_at(const float *p, int64_t at) { return p ? f2(p[at], p[at + V - 1]) : 0; }
template <typename T, int V> __device__ __forceinline__ void put_two(T *p, uint64_t v) {
    float v0, v1;
    un2(v, v0, v1);
    Raw<T, V> r;
    r.v[V - 1] = from_f32<T>(v1), r.v[0] = from_f32<T>(v0);
    store<T, V>(p, r);
}

template <typename T, int V> __global__ void __launch_bounds__(kShortThreads) linear_fwd_short_kernel(LinearArgs p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) * V, b = blockIdx.y, D = p.D;
    if (c0 >= D) return;
    const int rows = (int)p.L, live = (int)seq_len(p.seqlens, b, p.L);
    const int64_t at = b * p.L * D + c0;
    Raw<T, V> w[3][kShort];
#pragma unroll
    for (int t = 0; t < kShort; ++t)
        if (t < live) {
            w[0][t] = load<T, V>((const T *)p.x + at + t * D);
            w[1][t] = load<T, V>((const T *)p.r + at + t * D);
            w[2][t] = load<T, V>((const T *)p.i + at + t * D);
        }
    const Rate2 k = Rate2::of(p.c * softplus(p.lam[c0]), p.c * softplus(p.lam[c0 + V - 1]));
    const uint64_t init = two_at<V>(p.init, b * D + c0);
    uint64_t h = init, unused = 0;
    Run2 own = nothing();  // the final state is the run's from the first one, as linear_fwd_kernel has it
    if (p.states) put_two<float, V>(p.states + b * D + c0, init);
#pragma unroll
    for (int t = 0; t < kShort; ++t) {
        if (t >= rows) break;
        if (t < live) {
            const Gates2 g = gates2<T, false, false>(two_of<T, V>(w[1][t]), two_of<T, V>(w[2][t]), k, unused);
            const uint64_t one = mul2(g.f, two_of<T, V>(w[0][t]));
            h = fma2(g.a, h, one);
            own = after(own, {g.a, one});
        }
        if (p.y) put_two<T, V>((T *)p.y + at + t * D, t < live ? h : 0);
    }
    if (p.final_state) put_two<float, V>(p.final_state + b * D + c0, after(own, init));
    if (!p.values) return;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
        uint32_t top0 = 0, top1 = 0;
#pragma unroll
        for (int t = 0; t < kShort; ++t)
            if (t < live) top0 = max(top0, abs_bits(to_f32(w[z][t].v[0]))), top1 = max(top1, abs_bits(to_f32(w[z][t].v[V - 1])));
        const uint32_t code0 = scale_code(top0), code1 = scale_code(top1);
        Raw<uint8_t, V> code;
        code.v[V - 1] = (uint8_t)code1, code.v[0] = (uint8_t)code0;
        store<uint8_t, V>(p.scales + (z * p.B + b) * D + c0, code);
        const uint64_t inv = f2(inverse_scale(code0), inverse_scale(code1));
#pragma unroll
        for (int t = 0; t < kShort; ++t) {
            if (t >= rows) break;
            float q0, q1;
            un2(fma2(two_of<T, V>(w[z][t]), inv, f2(kToWhole)), q0, q1);
            Raw<int8_t, V> q;
            q.v[V - 1] = t < live && code1 != 255 ? (int8_t)(__float_as_uint(q1) & 0xff) : (int8_t)0;
            q.v[0] = t < live && code0 != 255 ? (int8_t)(__float_as_uint(q0) & 0xff) : (int8_t)0;
            store<int8_t, V>(p.values + z * p.B * p.L * D + at + t * D, q);
        }
    }
}

template <typename T, int V, bool PACK> __global__ void __launch_bounds__(kShortThreads) linear_bwd_short_kernel(LinearBwdArgs p) {
    pdl_enter();
    using W = std::conditional_t<PACK, int8_t, T>;
    const int64_t c0 = ((int64_t)blockIdx.x * kShortThreads + threadIdx.x) * V, b = blockIdx.y, D = p.f.D, L = p.f.L;
    if (c0 >= D) return;
    const int rows = (int)L, live = (int)seq_len(p.f.seqlens, b, L);
    const int64_t at = b * L * D + c0, plane = p.f.B * L * D;
    const W *from[3];
    if constexpr (PACK) {
        from[0] = p.f.values, from[1] = p.f.values + plane, from[2] = p.f.values + 2 * plane;
    } else {
        from[0] = (const T *)p.f.x, from[1] = (const T *)p.f.r, from[2] = (const T *)p.f.i;
    }
    Raw<W, V> w[3][kShort];
    Raw<T, V> dy[kShort];
#pragma unroll
    for (int t = 0; t < kShort; ++t)
        if (t < live) {
#pragma unroll
            for (int z = 0; z < 3; ++z) w[z][t] = load<W, V>(from[z] + at + t * D);
            dy[t] = load<T, V>((const T *)p.dy + at + t * D);
        }
    uint64_t scale[3] = {0, 0, 0};
    if constexpr (PACK) {
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            const Raw<uint8_t, V> code = load<uint8_t, V>(p.f.scales + (z * p.f.B + b) * D + c0);
            scale[z] = f2(scale_of(code.v[0]), scale_of(code.v[V - 1]));
        }
    }
    auto value = [&](int z, int t) {
        if constexpr (PACK) return mul2(f2((float)w[z][t].v[0], (float)w[z][t].v[V - 1]), scale[z]);
        else return two_of<T, V>(w[z][t]);
    };
    const Rate2 k = Rate2::of(p.f.c * softplus(p.f.lam[c0]), p.f.c * softplus(p.f.lam[c0 + V - 1]));
    uint64_t before[kShort], h = two_at<V>(p.f.states, b * D + c0), m = two_at<V>(p.dfinal, b * D + c0), sum = 0, unused = 0;
#pragma unroll
    for (int t = 0; t < kShort; ++t) {
        if (t >= live) break;
        const Gates2 g = gates2<T, false, false>(value(1, t), value(2, t), k, unused);
        before[t] = h;
        h = fma2(g.a, h, mul2(g.f, value(0, t)));
    }
#pragma unroll
    for (int t = kShort - 1; t >= 0; --t) {
        if (t >= rows) continue;
        uint64_t dx = 0, dr = 0, di = 0;
        if (t < live) {
            const Gates2 g = gates2<T, false, true>(value(1, t), value(2, t), k, unused);
            const uint64_t bt = mul2(g.f, value(0, t)), dh = add2(m, two_of<T, V>(dy[t]));
            const uint64_t factor = fma2(mul2(mul2(g.a, g.t), f2(-0.5f)), before[t], mul2(grad_ratio(g.t, g.a, true), bt)), psi = mul2(dh, factor);
            dx = mul2(dh, g.f);
            di = mul2(dh, mul2(bt, g.not_iota));
            dr = mul2(psi, mul2(g.er, g.rho));
            sum = add2(sum, psi);
            m = mul2(g.a, dh);
        }
        put_two<T, V>((T *)p.dx + at + t * D, dx);
        put_two<T, V>((T *)p.dr + at + t * D, dr);
        put_two<T, V>((T *)p.di + at + t * D, di);
    }
    put_two<float, V>(p.part + b * D + c0, sum);
    if (p.dinit) put_two<float, V>(p.dinit + b * D + c0, m);
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
// A thread takes V channels of ROWS rows of the batch, the weights' softplus formed once for them, and all of their loads under way
// before the first is used. In a graph, from L2, 256 rows of 5120 channels in bf16 take 5.0 us, one row of 1536 1.6; a call from Python is
// the host's 13.
template <typename T, int V, int ROWS> __global__ void __launch_bounds__(256) linear_step_kernel(LinearStepArgs p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * V, b0 = (int64_t)blockIdx.y * ROWS;
    if (c0 >= p.D) return;
    Raw<T, V> x[ROWS], r[ROWS], i[ROWS];
    float state[ROWS][V];
    int64_t slot[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) slot[j] = b0 + j >= p.B ? -2 : p.slots ? (int64_t)p.slots[b0 + j] : b0 + j;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        if (slot[j] >= p.nslots) slot[j] = -1;
        if (slot[j] < 0) continue;
        const int64_t at = (b0 + j) * p.D + c0;
        x[j] = load<T, V>((const T *)p.x + at), r[j] = load<T, V>((const T *)p.r + at), i[j] = load<T, V>((const T *)p.i + at);
#pragma unroll
        for (int v = 0; v < V; ++v) state[j][v] = p.state[slot[j] * p.D + c0 + v];
    }
    const Rate2 k = Rate2::of(p.c * softplus(p.lam[c0]), p.c * softplus(p.lam[c0 + V - 1]));
    auto two = [](const Raw<T, V> &w) { return f2(to_f32(w.v[0]), to_f32(w.v[V - 1])); };
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        float h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.f;
        if (slot[j] >= 0) {
            uint64_t unused = 0;
            const Gates2 g = gates2<T, false, false>(two(r[j]), two(i[j]), k, unused);
            float h0, h1;
            un2(fma2(g.a, f2(state[j][0], state[j][V - 1]), mul2(g.f, two(x[j]))), h0, h1);
            h[V - 1] = h1, h[0] = h0;
#pragma unroll
            for (int v = 0; v < V; ++v) p.new_state[slot[j] * p.D + c0 + v] = h[v];
        }
        if (b0 + j < p.B) store_f32<T, V>((T *)p.y + (b0 + j) * p.D + c0, h);  // zero for an idle row, whose state is not touched
    }
}

// ------------------------------------------------------------------- 8 bits
// A warp takes 32 V channels of one group of tokens, a lane 16 bytes of each row where rows are multiples of that. Bound by HBM: at
// B8 L2048 D2560 in bf16 22 us each way, 5.8 TB/s, in float32 36 and 35, 6.0 TB/s (bf16 41 us with one channel an instruction, whose
// registers left an SM one block).
template <typename T, int V> __global__ void __launch_bounds__(32 * kPackWarps, 2) pack8_kernel(Pack8Args p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + (threadIdx.x & 31)) * V, b = blockIdx.z, D = p.D;
    const int64_t groups = (p.L + kGroup - 1) / kGroup, g = (int64_t)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
    if (c0 >= D || g >= groups) return;
    const int64_t t0 = g * kGroup, at = (b * p.L + t0) * D + c0;
    const int rows = (int)imin<int64_t>(kGroup, p.L - t0);
    const int live = (int)imax<int64_t>(0, imin<int64_t>(rows, seq_len(p.seqlens, b, p.L) - t0));
    Raw<T, V> x[kGroup];
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
        if (t < live) x[t] = load<T, V>((const T *)p.x + at + t * D);
    Raw<uint8_t, V> code;
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {  // two channels at once, as in the forward
        uint64_t inv[V / 2];
        uint32_t mask[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < kGroup; ++t) top = __vmaxu2(top, x[t].u[k] & 0x7fff7fffu);
            const uint32_t c0 = scale_code(top << 16), c1 = scale_code(top & 0xffff0000u);
            code.v[2 * k] = (uint8_t)c0, code.v[2 * k + 1] = (uint8_t)c1;
            inv[k] = f2(inverse_scale(c0), inverse_scale(c1));
            mask[k] = (c0 == 255 ? 0u : 0xffu) | (c1 == 255 ? 0u : 0xff00u);
        }
        store<uint8_t, V>(p.scales + (b * groups + g) * D + c0, code);
#pragma unroll
        for (int t = 0; t < kGroup; ++t) {
            Raw<int8_t, V> q;
            uint32_t two[V / 2];
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                float q0, q1;
                un2(fma2(f2(__uint_as_float(x[t].u[k] << 16), __uint_as_float(x[t].u[k] & 0xffff0000u)), inv[k], f2(kToWhole)), q0, q1);
                two[k] = __byte_perm(__float_as_uint(q0), __float_as_uint(q1), 0x0040) & mask[k];
            }
            if constexpr (V == 2) {
                q.word = (uint16_t)two[0];
            } else {
#pragma unroll
                for (int k = 0; k < V / 4; ++k) q.u[k] = __byte_perm(two[2 * k], two[2 * k + 1], 0x5410);
            }
            if (t < rows) store<int8_t, V>(p.values + at + t * D, q);
        }
    } else {
        float inv[V];
        uint32_t finite[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < kGroup; ++t) top = max(top, abs_bits(to_f32(x[t].v[v])));
            code.v[v] = (uint8_t)scale_code(top);
            inv[v] = inverse_scale(code.v[v]);
            finite[v] = code.v[v] == 255 ? 0u : 0xffu;
        }
        store<uint8_t, V>(p.scales + (b * groups + g) * D + c0, code);
#pragma unroll
        for (int t = 0; t < kGroup; ++t) {
            Raw<int8_t, V> q;
#pragma unroll
            for (int v = 0; v < V; ++v) q.v[v] = (int8_t)(__float_as_uint(fmaf(to_f32(x[t].v[v]), inv[v], kToWhole)) & finite[v]);
            if (t < rows) store<int8_t, V>(p.values + at + t * D, q);
        }
    }
}

template <typename T, int V> __global__ void __launch_bounds__(32 * kPackWarps) unpack8_kernel(Pack8Args p) {
    pdl_enter();
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + (threadIdx.x & 31)) * V, b = blockIdx.z, D = p.D;
    const int64_t groups = (p.L + kGroup - 1) / kGroup, g = (int64_t)blockIdx.x * kPackWarps + (threadIdx.x >> 5);
    if (c0 >= D || g >= groups) return;
    const int64_t t0 = g * kGroup, at = (b * p.L + t0) * D + c0;
    const int rows = (int)imin<int64_t>(kGroup, p.L - t0);
    const Raw<uint8_t, V> code = load<uint8_t, V>(p.scales + (b * groups + g) * D + c0);
    Raw<int8_t, V> q[kGroup];
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
        if (t < rows) q[t] = load<int8_t, V>(p.values + at + t * D);
    float scale[V];
#pragma unroll
    for (int v = 0; v < V; ++v) scale[v] = scale_of(code.v[v]);
#pragma unroll
    for (int t = 0; t < kGroup; ++t) {
        float f[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            // byte v as 2^23 + 128 + v, less that: the conversion instruction takes four times as long
            const uint32_t n = __byte_perm(q[t].u[v / 4] ^ 0x80808080u, 0x4b000000u, 0x7440 + v % 4);
            f[v] = (__uint_as_float(n) - 8388736.f) * scale[v];
        }
        if (t < rows) store_f32<T, V>((T *)p.out + at + t * D, f);
    }
}

// --------------------------------------------------------------------- host

// f(integral_constant V): two channels a thread where rows are a multiple of two.
template <typename F> cudaError_t for_width(int64_t D, F &&f) {
    if (D % 2 == 0) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}
constexpr size_t kSmemPerSM = 233472, kSmemPerBlock = 232448;  // a block's also takes 1 KB of the SM's
constexpr int kMaxPerSM = 4;

// Clusters of KERN that the current device holds at once, by the blocks on an SM and those of a cluster; asked of the driver once per
// device below 64 and else on every call.
template <auto KERN> class ClusterTable {
  public:
    ClusterTable(int threads, int per_sm, size_t smem) : threads_(threads), per_sm_(per_sm), smem_(smem) {}
    // shared memory a block asks for so that an SM takes n
    size_t smem(int n) const { return n >= per_sm_ ? smem_ : imin(kSmemPerBlock, kSmemPerSM / n - 1024) / 128 * 128; }
    cudaError_t open() {
        static DeviceOnce configured;
        cudaError_t e = cudaSuccess;
        if (configured.pending(&dev_, &e)) {
            e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemPerBlock);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(KERN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) configured.done(dev_);
        }
        return e;
    }
    cudaError_t at_once(int n, int blocks, int *count) {
        static std::atomic<int> known[64][kMaxPerSM + 1][kMaxCluster + 1];  // and one
        std::atomic<int> *slot = dev_ >= 0 && dev_ < 64 ? &known[dev_][n][blocks] : nullptr;
        if (slot && (*count = slot->load(std::memory_order_acquire) - 1) >= 0) return cudaSuccess;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)blocks), cfg.blockDim = dim3((unsigned)threads_), cfg.dynamicSmemBytes = smem(n);
        cfg.attrs = attr, cfg.numAttrs = 1;
        cudaError_t e = cudaOccupancyMaxActiveClusters(count, KERN, &cfg);
        if (e == cudaSuccess && slot) slot->store(*count + 1, std::memory_order_release);
        return e;
    }

  private:
    int dev_ = 0, threads_, per_sm_;
    size_t smem_;
};

// Launches KERN over `items` sequences and tiles of L tokens, a run of `run` tokens a warp; an SM holds `per_sm` blocks.
// The blocks of a cluster and those on an SM are those whose waves times steps cost least. A block more in the cluster makes a step
// 4 % dearer (the forward at B8 L2048 D5120 takes 2.7 us a step with 2, 3.05 with 4, 3.4 with 8, 3.7 with 12; the backward at B4 3.7,
// 3.95, 4.8 and 5.0), one more on the SM a tenth (the same forward 2.4 us with 2, 2.8 with 3, 3.05 with 4). Fewer blocks on an SM than
// it holds, by asking for more shared memory than they need, is right where there are few clusters: a cluster's blocks are
// otherwise put on as few SMs as hold them (B1 L65536 D1536: 235 us in clusters of 16 with 4 on an SM, 213 in clusters of 15 with 3).
// A grid that fills the device is not launched as a programmatic dependent: placed while the kernel before it drains, clusters
// find holes that no other cluster fits, and the last of them wait for the first (forward 142 us rather than 124, backward 215 rather
// than 174). One that leaves half of the places free is (B1 L512 D1536: 5.2 us rather than 6.4).
template <auto KERN, typename Args, typename Maps>
cudaError_t launch_clusters(const Args &a, const Maps &maps, int64_t items, int64_t L, int run, int per_sm, size_t smem, cudaStream_t stream,
                            int *blocks_taken) {
    const int warps = (int)imin<int64_t>(kState / run, (L + run - 1) / run);  // no more than have a token
    const int64_t need = (L + kState - 1) / kState;
    ClusterTable<KERN> table(32 * (kState / run), per_sm, smem);
    cudaError_t e = table.open();
    int best = 0, on_sm = 0, held = 0;
    double cost = 0;
    for (int n = per_sm; n >= 1; --n)
        for (int blocks = 1; blocks <= kMaxCluster && blocks <= need; ++blocks) {
            int count = 0;
            if (e == cudaSuccess) e = table.at_once(n, blocks, &count);
            if (e != cudaSuccess) return e;
            if (count < 1) continue;
            const double c = (double)((items + count - 1) / count) * (double)((need + blocks - 1) / blocks) * (1.0 + 0.04 * blocks) * (0.6 + 0.1 * n);
            if (best == 0 || c < cost) best = blocks, on_sm = n, held = count, cost = c;
        }
    if (best == 0) return cudaErrorInvalidConfiguration;
    if (blocks_taken) *blocks_taken = best;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)best, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(imin<int64_t>(items, held) * best)), cfg.blockDim = dim3((unsigned)(32 * warps));
    cfg.dynamicSmemBytes = table.smem(on_sm), cfg.stream = stream, cfg.attrs = attr;
    cfg.numAttrs = cfg.gridDim.x * 2 <= (unsigned)(sm_count(1) * per_sm) ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, KERN, a, maps);
}

template <int V> dim3 short_grid(const LinearArgs &a) {
    return dim3((unsigned)((a.D / V + kShortThreads - 1) / kShortThreads), (unsigned)a.B);
}

template <typename T, bool WIDE, bool EVEN, bool PACK> cudaError_t forward_p(const LinearArgs &a, const FwdMaps &maps, cudaStream_t stream) {
    return launch_clusters<linear_fwd_kernel<T, WIDE, EVEN, PACK>>(a, maps, a.B * ((a.D + kTile - 1) / kTile), a.L, kFwdRun, fwd_per_sm<T, PACK>(),
                                                             sizeof(FwdShared<T, WIDE, PACK>), stream, nullptr);
}
template <typename T> cudaError_t forward_t(const LinearArgs &a, cudaStream_t stream) {
    if (a.L == 0) {
        if (!a.final_state || a.final_state == a.init) return cudaSuccess;
        return launch_programmatic(linear_keep_kernel, dim3((unsigned)((a.B * a.D + 255) / 256)), dim3(256), 0, stream, a.init,
                                   a.final_state, a.B * a.D);
    }
    if (a.L <= kShort)
        return for_width(a.D, [&](auto vw) {
            constexpr int V = decltype(vw)::value;
            return launch_programmatic(linear_fwd_short_kernel<T, V>, short_grid<V>(a), dim3(kShortThreads), 0, stream, a);
        });
    FwdMaps m{};
    const int size = (int)sizeof(T);
    bool wide = a.D * size % 16 == 0 && tma_map_rows(&m.x, a.x, size, a.D, a.L, a.B, kTile, kState) &&
                tma_map_rows(&m.r, a.r, size, a.D, a.L, a.B, kTile, kState) && tma_map_rows(&m.i, a.i, size, a.D, a.L, a.B, kTile, kState) &&
                (!a.y || tma_map_rows(&m.y, a.y, size, a.D, a.L, a.B, kTile, kFwdRun));
    if (a.values) {
        wide = wide && a.D % 16 == 0 && tma_map_planes(&m.q, a.values, a.D, a.L, a.B, 3, kTile, kFwdRun);
        if (wide) return forward_p<T, true, true, true>(a, m, stream);
        return a.D % 2 == 0 ? forward_p<T, false, true, true>(a, m, stream) : forward_p<T, false, false, true>(a, m, stream);
    }
    if (wide) return forward_p<T, true, true, false>(a, m, stream);
    return a.D % 2 == 0 ? forward_p<T, false, true, false>(a, m, stream) : forward_p<T, false, false, false>(a, m, stream);
}

template <typename T, bool WIDE, bool EVEN, bool PACK> cudaError_t backward_p(const LinearBwdArgs &a, const BwdMaps &maps, cudaStream_t stream, int *blocks) {
    return launch_clusters<linear_bwd_kernel<T, WIDE, EVEN, PACK>>(a, maps, a.f.B * ((a.f.D + kTile - 1) / kTile), a.f.L, kBwdRun,
                                                             bwd_per_sm<T>(), sizeof(BwdShared<T, WIDE, PACK>), stream, blocks);
}
template <typename T> cudaError_t backward_t(const LinearBwdArgs &a, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    int blocks = 0;  // none has added to the sum for dlam
    const int64_t B = a.f.B, L = a.f.L, D = a.f.D;
    if (B > 0 && L > 0 && L <= kShort) {
        blocks = 1;
        e = for_width(D, [&](auto vw) {
            constexpr int V = decltype(vw)::value;
            return a.f.values ? launch_programmatic(linear_bwd_short_kernel<T, V, true>, short_grid<V>(a.f), dim3(kShortThreads), 0, stream, a)
                              : launch_programmatic(linear_bwd_short_kernel<T, V, false>, short_grid<V>(a.f), dim3(kShortThreads), 0, stream, a);
        });
    } else if (B > 0 && L > 0) {
        BwdMaps m{};
        const int size = (int)sizeof(T);
        bool wide = D * size % 16 == 0 && tma_map_rows(&m.dy, a.dy, size, D, L, B, kTile, kState) &&
                    tma_map_rows(&m.dx, a.dx, size, D, L, B, kTile, kBwdRun) && tma_map_rows(&m.dr, a.dr, size, D, L, B, kTile, kBwdRun) &&
                    tma_map_rows(&m.di, a.di, size, D, L, B, kTile, kBwdRun);
        if (a.f.values) {
            wide = wide && D % 16 == 0 && tma_map_planes(&m.q, a.f.values, D, L, B, 3, kTile, kState) &&
                   tma_map_planes(&m.scale, a.f.scales, D, (L + kGroup - 1) / kGroup, B, 3, kTile, kState / kGroup);
            e = wide         ? backward_p<T, true, true, true>(a, m, stream, &blocks)
                : D % 2 == 0 ? backward_p<T, false, true, true>(a, m, stream, &blocks)
                             : backward_p<T, false, false, true>(a, m, stream, &blocks);
        } else {
            wide = wide && tma_map_rows(&m.x, a.f.x, size, D, L, B, kTile, kState) && tma_map_rows(&m.r, a.f.r, size, D, L, B, kTile, kState) &&
                   tma_map_rows(&m.i, a.f.i, size, D, L, B, kTile, kState);
            e = wide         ? backward_p<T, true, true, false>(a, m, stream, &blocks)
                : D % 2 == 0 ? backward_p<T, false, true, false>(a, m, stream, &blocks)
                             : backward_p<T, false, false, false>(a, m, stream, &blocks);
        }
    } else if (B > 0 && a.dinit && a.dinit != a.dfinal) {
        e = launch_programmatic(linear_keep_kernel, dim3((unsigned)((B * D + 255) / 256)), dim3(256), 0, stream, a.dfinal, a.dinit, B * D);
    }
    if (e != cudaSuccess) return e;
    return launch_programmatic(linear_dlam_kernel, dim3((unsigned)((D + 31) / 32)), dim3(32, 8), 0, stream, (const float *)a.part, a.f.lam,
                               a.dlam, B * blocks, D);
}

}  // namespace linear

int64_t linear_bwd_parts(int64_t B) { return B * linear::kMaxCluster; }

cudaError_t launch_linear(int io, const LinearArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::forward_t<__nv_bfloat16>(a, stream) : linear::forward_t<float>(a, stream);
}

cudaError_t launch_linear_bwd(int io, const LinearBwdArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::backward_t<__nv_bfloat16>(a, stream) : linear::backward_t<float>(a, stream);
}

namespace linear {
template <typename T, int V, int ROWS> cudaError_t step_v(const LinearStepArgs &a, cudaStream_t stream) {
    const int64_t vecs = a.D / V;
    const int threads = (int)imin<int64_t>(256, (vecs + 31) / 32 * 32);
    const dim3 grid((unsigned)((vecs + threads - 1) / threads), (unsigned)((a.B + ROWS - 1) / ROWS));
    return launch_programmatic(linear_step_kernel<T, V, ROWS>, grid, dim3(threads), 0, stream, a);
}
// Four rows a thread where that leaves two threads or more for every lane of the device.
template <typename T> cudaError_t step_t(const LinearStepArgs &a, cudaStream_t stream) {
    return for_width(a.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        return a.B / 4 * (a.D / V) >= 256ll * sm_count(1) ? step_v<T, V, 4>(a, stream) : step_v<T, V, 1>(a, stream);
    });
}
}  // namespace linear

cudaError_t launch_linear_step(int io, const LinearStepArgs &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::step_t<__nv_bfloat16>(a, stream) : linear::step_t<float>(a, stream);
}

cudaError_t linear_withhold(int what, int rank, int step) {
#ifdef SSD_DEBUG_BOUNDS
    const int w[3] = {what, rank, step};
    return cudaMemcpyToSymbol(linear::g_withhold, w, sizeof(w));
#else
    return cudaErrorNotSupported;
#endif
}

cudaError_t linear_gave_up(unsigned long long *count, cudaStream_t stream) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(count, linear::g_gave_up, sizeof(*count), 0, cudaMemcpyDeviceToHost, stream);
    return e == cudaSuccess ? cudaStreamSynchronize(stream) : e;
}

namespace linear {
template <typename T, int V> cudaError_t pack8_v(const Pack8Args &a, cudaStream_t stream) {
    const int64_t groups = (a.L + kGroup - 1) / kGroup;
    const dim3 grid((unsigned)((groups + kPackWarps - 1) / kPackWarps), (unsigned)((a.D + 32 * V - 1) / (32 * V)), (unsigned)a.B), block(32 * kPackWarps);
    return a.out ? launch_programmatic(unpack8_kernel<T, V>, grid, block, 0, stream, a) : launch_programmatic(pack8_kernel<T, V>, grid, block, 0, stream, a);
}
template <typename T> cudaError_t pack8_t(const Pack8Args &a, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    return a.D % V == 0 ? pack8_v<T, V>(a, stream) : a.D % 2 == 0 ? pack8_v<T, 2>(a, stream) : pack8_v<T, 1>(a, stream);
}
}  // namespace linear

cudaError_t launch_pack8(int io, const Pack8Args &a, cudaStream_t stream) {
    return io == IO_BF16 ? linear::pack8_t<__nv_bfloat16>(a, stream) : linear::pack8_t<float>(a, stream);
}

}  // namespace ssd
