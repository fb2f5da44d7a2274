// Gated linear recurrence, per sequence and channel, with a weight lam per channel:
//     w_t = c softplus(lam) sigmoid(r_t)     a_t = exp(-w_t)     b_t = sqrt(1 - a_t^2) sigmoid(i_t) x_t
//     h_t = a_t h_{t-1} + b_t                y_t = h_t
// its backward, and one token of it over a pool of states.
//
// A run of tokens acts on the state as h -> A h + H, A the product of its a and H its result from zero, so runs are formed
// apart and joined in order. A lane has two channels; a warp holds 64 channels of a run in registers, the warps of a block lie
// one behind the other in time, and so do the blocks of a cluster. A warp forms a, b and its (A, H), the warps of a block
// join theirs in shared memory, each block sends its own to the others of its cluster, and every warp goes over its run again
// from the state that enters it. The cluster then takes the next tokens of the sequence, the state kept by all of its threads.
// Blocks of kBlock tokens are always joined one after the other, so the result depends neither on the cluster's size nor on
// the batch. Tokens past a sequence's end act as a = 1, b = 0 and are not read.
#include <cooperative_groups.h>

#include "gated_linear.cuh"
#include "launch.h"
#include "ssd_scan.h"
#include "tc_ptx.cuh"

namespace ssd {
namespace linear {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTile = 64;                 // channels of a block, two a lane
constexpr int kFwdRun = kGroup;           // tokens of a warp in the forward: a group of the 8-bit values
constexpr int kBwdRun = kState / kWarps;  // and in the backward, whose block takes the tokens between two saved states
constexpr int kMaxCluster = 8;            // blocks; 4 for rows that are fetched by words, so that two blocks fit an SM

// ------------------------------------------------------- copies to shared memory
// A warp fetches the rows of its own runs, two steps ahead, and only it reads them: no barrier but its own. WIDE: 16 bytes a
// lane, for rows that begin at a multiple of 16 bytes. Otherwise 4 bytes: the aligned words around each row, of those at the
// tensor's end and the tile's only the bytes that belong to the tensor; a row then begins up to 3 bytes into its first word.
template <int BYTES> __device__ __forceinline__ void copy(uint32_t to, const void *from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, bool WIDE> struct Row {  // in shared memory
    static constexpr int kPitch = kTile * (int)sizeof(T) + (WIDE || sizeof(T) == 4 ? 0 : 4);
};

// Rows 0..n-1 of a tile, R at most, of `cols` channels from `base` on, which lie D apart. ACROSS: the bytes from one row to the
// next in shared memory; V: the channels of a piece, where WIDE.
template <typename T, bool WIDE, int R, int ACROSS, int V = 16 / (int)sizeof(T)>
__device__ __forceinline__ void fetch_rows(unsigned char *to, const T *base, int n, int cols, int64_t D, int lane) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (WIDE) {
        constexpr int PER = kTile / V, ROWS = 32 / PER;  // lanes a row, rows at once
        static_assert(R % ROWS == 0, "");
        const int piece = lane % PER, first = lane / PER;
        const int c = piece * V;
        if (c < cols) {
            const T *from = base + first * D + c;
            const int64_t next = ROWS * D;
#pragma unroll
            for (int j = 0; j < R / ROWS; ++j, from += next)
                if (j * ROWS + first < n) copy<V * (int)sizeof(T)>(dst + (j * ROWS + first) * ACROSS + piece * V * (int)sizeof(T), from);
        }
    } else {
        const int have = cols * (int)sizeof(T);  // bytes of the tile's row
        const unsigned char *from = reinterpret_cast<const unsigned char *>(base);
#pragma unroll 4
        for (int t = 0; t < n; ++t, from += D * sizeof(T)) {
            const int off = (int)(reinterpret_cast<uintptr_t>(from) & 3);
            const unsigned char *word = from - off;
#pragma unroll
            for (int w = 0; w < (kTile * (int)sizeof(T) + 127 + (sizeof(T) == 4 ? 0 : 3)) / 128; ++w) {
                const int at = 4 * lane + 128 * w, left = off + have - at;
                if (left > 0) copy4(dst + t * ACROSS + at, word + at, left < 4 ? left : 4);
            }
        }
    }
}
// The two channels of a lane in a row fetched so; `off` the bytes that the row begins into its first word.
template <typename T, bool WIDE> __device__ __forceinline__ Raw<T, 2> row_pair(const unsigned char *row, int off, int lane, bool both) {
    Raw<T, 2> r;
    const T *p = reinterpret_cast<const T *>(row + off) + 2 * lane;
    if constexpr (WIDE) {
        r.word = *reinterpret_cast<const decltype(r.word) *>(p);
    } else {
        r.v[0] = p[0], r.v[1] = both ? p[1] : p[0];
    }
    return r;
}
// The same two channels in global memory; `both` and `one`: whether they exist.
template <typename T, bool WIDE> __device__ __forceinline__ void store_pair(T *p, const Raw<T, 2> &r, bool one, bool both) {
    if constexpr (WIDE) {
        if (one) store<T, 2>(p, r);
    } else {
        if (one) p[0] = r.v[0];
        if (both) p[1] = r.v[1];
    }
}
template <typename T, bool WIDE> __device__ __forceinline__ void store_pair(T *p, float a, float b, bool one, bool both) {
    Raw<T, 2> r;
    r.v[0] = from_f32<T>(a), r.v[1] = from_f32<T>(b);
    store_pair<T, WIDE>(p, r, one, both);
}

// The same rows from shared memory, where each lane has put its two channels: 16 bytes of T a lane (or as many values of a
// smaller type U).
template <typename T, typename U, int R, int ACROSS>
__device__ __forceinline__ void leave_rows(const unsigned char *from, U *base, int n, int cols, int64_t D, int lane) {
    constexpr int V = 16 / (int)sizeof(T), PER = kTile / V, ROWS = 32 / PER;
    const int piece = lane % PER, first = lane / PER;
    if (piece * V >= cols) return;
    U *to = base + first * D + piece * V;
    const int64_t next = ROWS * D;
#pragma unroll
    for (int j = 0; j < R / ROWS; ++j, to += next)
        if (j * ROWS + first < n) {
            Raw<U, V> r;
            r.word = *reinterpret_cast<const decltype(r.word) *>(from + (j * ROWS + first) * ACROSS + piece * V * sizeof(U));
            store<U, V>(to, r);
        }
}

// ------------------------------------------------------------ runs, joined in order
// (A, H) of a lane's two channels: h -> A h + H.
struct alignas(16) Run2 {
    uint64_t a, h;
};
__device__ __forceinline__ uint64_t after(const Run2 &x, uint64_t h) { return fma2(x.a, h, x.h); }  // x, from h
__device__ __forceinline__ Run2 after(const Run2 &x, const Run2 &y) { return {mul2(x.a, y.a), fma2(y.a, x.h, y.h)}; }  // x, then y

// A step of a cluster: the tile of a sequence that it is at. The first thread works it out three steps ahead, while it would wait.
struct Step {
    int64_t base;      // of the step's first token and the tile's first channel in [B, L, D]
    int64_t b;
    int32_t first;     // token
    int32_t len;       // tokens of the sequence
    int32_t cols;      // channels of the tile; 0: no more work
    int32_t c0;
};
struct Walk {
    uint32_t item, items, tiles, clusters;
    int64_t first;
    // the step here; then goes on
    __device__ __forceinline__ Step forward(const LinearArgs &p, int span) {
        Step s{};
        if (item >= items) return s;
        const uint32_t b = item / tiles;
        s.b = b, s.c0 = (int32_t)(item - b * tiles) * kTile, s.first = (int32_t)first;
        s.cols = (int32_t)imin<int64_t>(kTile, p.D - s.c0);
        s.len = (int32_t)seq_len(p.seqlens, b, p.L);
        s.base = (b * p.L + first) * p.D + s.c0;
        first += span;
        if (first >= p.L) first = 0, item += clusters;
        return s;
    }
    // the same from a sequence's end, where steps begin at `last`
    __device__ __forceinline__ Step backward(const LinearArgs &p, int span, int64_t last) {
        Step s{};
        if (item >= items) return s;
        const uint32_t b = item / tiles;
        s.b = b, s.c0 = (int32_t)(item - b * tiles) * kTile, s.first = (int32_t)first;
        s.cols = (int32_t)imin<int64_t>(kTile, p.D - s.c0);
        s.len = (int32_t)seq_len(p.seqlens, b, p.L);
        s.base = (b * p.L + first) * p.D + s.c0;
        if (first <= 0) {
            first = last, item += clusters;
        } else {
            first -= span;
        }
        return s;
    }
};
// Tokens of a run of R from t0 on that are below `end`.
__device__ __forceinline__ int run_of(int R, int64_t end, int64_t t0) { return (int)imax<int64_t>(0, imin<int64_t>(R, end - t0)); }

// The blocks of a cluster exchange a Run2 a lane: each sends its own to all of them, and the bytes count down the receiver's
// barrier. (A cluster barrier would have the sender wait for everything that it has written to memory before.) Two of each,
// taken in turn: a block sends for a step once all of its warps have read the one before.
template <int MAX> struct Exchange {
    static constexpr int kMax = MAX;
    Run2 block[2][MAX][32];
    uint64_t bar[2];
};
constexpr uint64_t kGiveUpNs = 1000000000ull;
__device__ int g_gave_up;  // SSD_ERR_TIMEOUT once a wait was given up on this device

template <int MAX> __device__ __forceinline__ void exchange_init(Exchange<MAX> &x, int blocks) {
    if (threadIdx.x == 0) {
        tc::mbar_init(&x.bar[0], 1);
        tc::mbar_init(&x.bar[1], 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    if (blocks > 1) {  // the others are there, with their barriers
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}
// To the ranks first, first + every, ...
template <int MAX> __device__ __forceinline__ void exchange_send(Exchange<MAX> &x, int step, int rank, int blocks, int first, int every, int lane, const Run2 &own) {
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
// False, now and from then on, where the others' runs have not come in kGiveUpNs.
template <int MAX> __device__ __forceinline__ bool exchange_wait(Exchange<MAX> &x, int step, bool alive) {
    if (!alive) return false;
    if (tc::mbar_wait(&x.bar[step & 1], (step >> 1) & 1, kGiveUpNs)) return true;
    atomicCAS(&g_gave_up, SSD_OK, SSD_ERR_TIMEOUT);
    return false;
}

// ------------------------------------------------------------------ forward
// Bound by HBM (8 bytes a token and channel in bf16) with the issue slots and the special function unit close behind it: so two
// channels an instruction where there is one for it, and results leave through shared memory, 16 bytes a lane (the rows that were
// fetched make room for them).
template <typename T, bool WIDE> struct FwdShared {
    static constexpr int kAcross = Row<T, WIDE>::kPitch;
    unsigned char row[2][kWarps][3][kFwdRun][kAcross];
    Run2 run[2][kWarps][32];  // in turn: a warp may be at its next run while another reads these
    Exchange<WIDE ? kMaxCluster : 4> exchange;
    Step step[4];
};

// A run's values in 8 bits: rows of z (0: x, 1: r, 2: i) from `w`, which holds what `row` held of them.
template <typename T, bool WIDE, int R, int ACROSS>
__device__ __forceinline__ void leave_in_8_bits(const LinearArgs &p, int z, const Raw<T, 2> (&w)[R], unsigned char *row, const Step &s, int64_t t0,
                                                int live, int rows, int lane) {
    const int64_t D = p.D;
    int8_t *values = p.values + (z * p.B * p.L + t0 - s.first) * D + s.base;
    const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
    uint32_t top0 = 0, top1 = 0;
    if constexpr (sizeof(T) == 2) {
        uint32_t top = 0;  // bf16 without its sign orders like a whole number: two at once
#pragma unroll
        for (int t = 0; t < R; ++t)
            if (t < live) top = __vmaxu2(top, w[t].word & 0x7fff7fffu);
        top0 = top << 16, top1 = top & 0xffff0000u;
    } else {
#pragma unroll
        for (int t = 0; t < R; ++t)
            if (t < live) top0 = max(top0, abs_bits(w[t].v[0])), top1 = max(top1, abs_bits(w[t].v[1]));
    }
    Raw<uint8_t, 2> code;
    code.v[0] = (uint8_t)scale_code(top0), code.v[1] = (uint8_t)scale_code(top1);
    store_pair<uint8_t, WIDE>(p.scales + ((z * p.B + s.b) * ((p.L + kGroup - 1) / kGroup) + t0 / kGroup) * D + s.c0 + 2 * lane, code, one, both);
    const uint64_t inv = f2(inverse_scale(code.v[0]), inverse_scale(code.v[1]));
    const uint32_t mask = (code.v[0] == 255 ? 0u : 0xffu) | (code.v[1] == 255 ? 0u : 0xff00u);
    __syncwarp();  // every lane has read the row
#pragma unroll
    for (int t = 0; t < R; ++t) {
        float q0, q1;
        un2(fma2(pair_of(w[t]), inv, f2(kToWhole)), q0, q1);
        Raw<int8_t, 2> q;
        q.word = (uint16_t)(t < live ? __byte_perm(__float_as_uint(q0), __float_as_uint(q1), 0x0040) & mask : 0u);
        if constexpr (WIDE) {
            *reinterpret_cast<uint16_t *>(row + t * ACROSS + 2 * lane) = q.word;
        } else {
            if (t < rows) store_pair<int8_t, WIDE>(values + t * D + 2 * lane, q, one, both);
        }
    }
    if constexpr (WIDE) {
        __syncwarp();
        leave_rows<T, int8_t, R, ACROSS>(row, values, rows, s.cols, D, lane);
        __syncwarp();
    }
}

template <typename T, bool WIDE, bool PACK>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) linear_fwd_kernel(LinearArgs p) {
    namespace cg = cooperative_groups;
    pdl_enter();
    constexpr int R = kFwdRun, ACROSS = FwdShared<T, WIDE>::kAcross;
    extern __shared__ __align__(16) unsigned char raw_smem[];
    FwdShared<T, WIDE> &sh = *reinterpret_cast<FwdShared<T, WIDE> *>(raw_smem);
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
    const int64_t D = p.D, L = p.L;
    const int span = warps * R * blocks, mine = (rank * warps + warp) * R;  // a step's tokens; of them, where this warp's run is
    Walk walk{blockIdx.x / (uint32_t)blocks, 0, (uint32_t)((D + kTile - 1) / kTile), gridDim.x / (uint32_t)blocks, 0};
    walk.items = (uint32_t)p.B * walk.tiles;  // below 2^31
    if (threadIdx.x == 0)
        for (int j = 0; j < 3; ++j) sh.step[j] = walk.forward(p, span);
    exchange_init(sh.exchange, blocks);

    auto fetch = [&](int step) {
        const Step s = sh.step[step & 3];
        if (s.cols > 0) {
            const int live = run_of(R, s.len, (int64_t)s.first + mine);
            const int64_t at = s.base + mine * D;
            auto &to = sh.row[step & 1][warp];
            fetch_rows<T, WIDE, R, ACROSS>(to[0][0], (const T *)p.x + at, live, s.cols, D, lane);
            fetch_rows<T, WIDE, R, ACROSS>(to[1][0], (const T *)p.r + at, live, s.cols, D, lane);
            fetch_rows<T, WIDE, R, ACROSS>(to[2][0], (const T *)p.i + at, live, s.cols, D, lane);
        }
        copy_commit();
    };
    fetch(0);
    fetch(1);
    uint64_t carry = 0;
    Rate2 rate{};
    bool steep = false, alive = true;
    for (int step = 0;; ++step) {
        const Step s = sh.step[step & 3];
        if (s.cols == 0) break;
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&sh.exchange.bar[step & 1], blocks * 32 * (uint32_t)sizeof(Run2));
        const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
        const int64_t t0 = (int64_t)s.first + mine, at = s.base + mine * D + 2 * lane;
        const int live = run_of(R, s.len, t0), rows = run_of(R, L, t0);  // tokens that count, that exist
        auto &in = sh.row[step & 1][warp];
        if (s.first == 0) {
            const int64_t c = s.c0 + 2 * lane;
            float k0 = one ? p.lam[c] : 0.f, k1 = both ? p.lam[c + 1] : 0.f;
            carry = p.init ? f2(one ? p.init[s.b * D + c] : 0.f, both ? p.init[s.b * D + c + 1] : 0.f) : 0;
            k0 = p.c * softplus(k0), k1 = p.c * softplus(k1);
            rate = Rate2::of(k0, k1);
            steep = __any_sync(0xffffffffu, (one && !(k0 < kSteep)) || (both && !(k1 < kSteep)));
        }
        copy_wait<1>();
        __syncwarp();
        auto pair = [&](int z, int t) {
            const void *base = z == 0 ? p.x : z == 1 ? p.r : p.i;
            const int off = WIDE || sizeof(T) == 4
                                ? 0
                                : (int)((reinterpret_cast<uintptr_t>(base) + (uintptr_t)(at - 2 * lane + t * D) * sizeof(T)) & 3);
            return row_pair<T, WIDE>(in[z][t], off, lane, both);
        };
        uint64_t a[R], h[R];
        Run2 own;
        Raw<T, 2> low;
        auto tokens = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            own.a = f2(1.f), own.h = f2(0.f);
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const Raw<T, 2> r = pair(1, t), i = pair(2, t);
                if (FAST) {
                    if (t == 0) low = r; else lower(low, r);
                    lower(low, i);
                }
                const Gates2 g = gates2<T, FAST, false>(pair_of(r), pair_of(i), rate);
                a[t] = g.a;
                h[t] = mul2(g.f, pair_of(pair(0, t)));
                if (!FAST && t >= live) a[t] = f2(1.f), h[t] = f2(0.f);
                own = after(own, {a[t], h[t]});
            }
        };
        bool fast = live == R && !steep;
        if (fast) {
            tokens(std::true_type{});
            fast = !__any_sync(0xffffffffu, one && is_low(low));
        }
        if (!fast) tokens(std::false_type{});
        sh.run[step & 1][warp][lane] = own;
        __syncthreads();
        // The block's runs before this one, and all of them: every warp joins them, and sends to another block.
        Run2 before{f2(1.f), f2(0.f)}, all = before;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            if (w == warp) before = all;
            all = after(all, sh.run[step & 1][w][lane]);
        }
        exchange_send(sh.exchange, step, rank, blocks, warp, warps, lane, all);
        if (threadIdx.x == 0) sh.step[(step + 3) & 3] = walk.forward(p, span);
        alive = exchange_wait(sh.exchange, step, alive);
        if (!alive) carry = f2(__uint_as_float(0x7fc00000u));  // what was not told is not guessed
        uint64_t e = carry;                                     // the state that enters this run
#pragma unroll 4
        for (int j = 0; j < blocks; ++j) {
            if (j == rank) e = carry;
            carry = after(sh.exchange.block[step & 1][j][lane], carry);
        }
        e = after(before, e);
        if (rows > 0 && p.states && t0 % kState == 0) {
            float e0, e1;
            un2(e, e0, e1);
            store_pair<float, WIDE>(p.states + (s.b * ((L + kState - 1) / kState) + t0 / kState) * D + s.c0 + 2 * lane, e0, e1, one, both);
        }
        Raw<T, 2> words[R];
        if constexpr (PACK) {
#pragma unroll
            for (int t = 0; t < R; ++t) words[t] = pair(0, t);
        }
        __syncwarp();
        if (p.y) {
            auto results = [&](auto whole) {
#pragma unroll
                for (int t = 0; t < R; ++t) {
                    float y0, y1;
                    e = fma2(a[t], e, h[t]);
                    un2(e, y0, y1);
                    if (!decltype(whole)::value && t >= live) y0 = y1 = 0.f;
                    Raw<T, 2> y;
                    y.v[0] = from_f32<T>(y0), y.v[1] = from_f32<T>(y1);
                    if constexpr (WIDE) {
                        *reinterpret_cast<decltype(y.word) *>(in[0][t] + 2 * sizeof(T) * lane) = y.word;
                    } else {
                        if (t < rows) store_pair<T, WIDE>((T *)p.y + at + t * D, y, one, both);
                    }
                }
            };
            if (live == R) results(std::true_type{}); else results(std::false_type{});
            if constexpr (WIDE) {
                __syncwarp();
                leave_rows<T, T, R, ACROSS>(in[0][0], (T *)p.y + at - 2 * lane, rows, s.cols, D, lane);
                __syncwarp();
            }
        }
        if constexpr (PACK) {
            if (rows > 0) {
                leave_in_8_bits<T, WIDE, R, ACROSS>(p, 0, words, in[0][0], s, t0, live, rows, lane);
#pragma unroll
                for (int z = 1; z < 3; ++z) {
#pragma unroll
                    for (int t = 0; t < R; ++t) words[t] = pair(z, t);
                    leave_in_8_bits<T, WIDE, R, ACROSS>(p, z, words, in[z][0], s, t0, live, rows, lane);
                }
            }
        }
        __syncwarp();
        fetch(step + 2);
        if (s.first + (int64_t)span >= L && rank == 0 && warp == 0 && p.final_state) {
            float e0, e1;
            un2(carry, e0, e1);
            store_pair<float, WIDE>(p.final_state + s.b * D + s.c0 + 2 * lane, e0, e1, one, both);
        }
    }
    copy_wait<0>();
}

// A sequence of no tokens: its state goes through.
__global__ void __launch_bounds__(256) linear_keep_kernel(const float *init, float *final_state, int64_t n) {
    pdl_enter();
    const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (j < n) final_state[j] = init ? init[j] : 0.f;
}

// ----------------------------------------------------------------- backward
// dh_t = dy_t + m_{t+1}, m_t = a_t dh_t (m behind the last token the gradient of the final state): the same kind of recurrence,
// backwards, a run acting as m -> A m + M. With f and g as in gates2 and psi_t = w_t dL/dw_t:
//     b = f x     dx = dh f     di = dh b (1 - iota)     psi = dh (g b - a w h_{t-1})     dr = psi (1 - rho)
//     dlam = sigmoid(lam) / softplus(lam) sum psi
// (psi rather than dL/dw, which has 1 / sqrt(1 - a^2): w over it goes to zero with w.) h_{t-1} is formed again from the state that
// enters each kState tokens, which are a block's; the warps and blocks lie one before the other in time.
// Bound as the forward is (14 bytes a token and channel in bf16, 11 from 8 bits).
template <typename T, bool WIDE, bool PACK> struct BwdShared {
    static constexpr int kAcross = Row<T, WIDE>::kPitch;  // 8-bit rows too: the gradients' rows take their place
    unsigned char row[2][kWarps][4][kBwdRun][kAcross];    // x, r, i and dy; then dx, dr and di
    float state[4][kTile];
    unsigned char scale[2][kWarps][3][kTile + 4];
    Run2 run[2][kWarps][32];
    uint64_t h[2][kWarps][32], sum[kWarps][32];
    Exchange<WIDE ? kMaxCluster : 4> exchange;
    Step step[4];
};

// The two channels of a lane in 8 bits, as numbers: byte v as 2^23 + 128 + v, less that, exactly; times the scale.
__device__ __forceinline__ uint64_t from_8(uint32_t two, uint64_t scale) {
    const uint32_t v = two ^ 0x8080u;
    const uint64_t n = f2(__uint_as_float(__byte_perm(v, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(v, 0x4b000000u, 0x7441)));
    return mul2(add2(n, f2(-8388736.f)), scale);
}

// Whether a run's gates are all above kLowGate.
template <typename T, bool PACK> struct Low {
    Raw<T, 2> least;
    __device__ __forceinline__ void see(const Raw<T, 2> &r, const Raw<T, 2> &i, bool first) {
        if (first) least = r; else lower(least, r);
        lower(least, i);
    }
    __device__ __forceinline__ bool any() const { return is_low(least); }
};
template <typename T> struct Low<T, true> {
    Raw<float, 2> least;
    __device__ __forceinline__ void see(uint64_t r, uint64_t i, bool first) {
        Raw<float, 2> a, b;
        un2(r, a.v[0], a.v[1]);
        un2(i, b.v[0], b.v[1]);
        if (first) least = a; else lower(least, a);
        lower(least, b);
    }
    __device__ __forceinline__ bool any() const { return is_low(least); }
};

template <typename T, bool WIDE, bool PACK>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) linear_bwd_kernel(LinearBwdArgs p) {
    namespace cg = cooperative_groups;
    pdl_enter();
    constexpr int R = kBwdRun, ACROSS = BwdShared<T, WIDE, PACK>::kAcross;
    extern __shared__ __align__(16) unsigned char raw_smem[];
    BwdShared<T, WIDE, PACK> &sh = *reinterpret_cast<BwdShared<T, WIDE, PACK> *>(raw_smem);
    const cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)cluster.block_rank(), blocks = (int)cluster.num_blocks();
    const int64_t D = p.f.D, L = p.f.L, chunks = (L + kState - 1) / kState, groups = (L + kGroup - 1) / kGroup;
    const int64_t plane = p.f.B * L * D, scales = p.f.B * groups * D;
    // This warp's run, from the step's first token: rank 0 and warp 0 have the latest. A step begins a cluster's chunks before the
    // one it came from, at the start of a sequence before its first token.
    const int mine = (blocks - 1 - rank) * kState + (warps - 1 - warp) * R;
    Walk walk{blockIdx.x / (uint32_t)blocks, 0, (uint32_t)((D + kTile - 1) / kTile), gridDim.x / (uint32_t)blocks, 0};
    walk.items = (uint32_t)p.f.B * walk.tiles;  // below 2^31
    walk.first = (chunks - blocks) * kState;
    if (threadIdx.x == 0)
        for (int j = 0; j < 3; ++j) sh.step[j] = walk.backward(p.f, blocks * kState, (chunks - blocks) * kState);
    exchange_init(sh.exchange, blocks);

    auto fetch = [&](int step) {
        const Step s = sh.step[step & 3];
        const int64_t t0 = (int64_t)s.first + mine;
        if (s.cols > 0 && t0 >= 0) {
            const int live = run_of(R, s.len, t0);
            const int64_t at = s.base + mine * D;
            auto &to = sh.row[step & 1][warp];
            if constexpr (PACK) {
                if (live > 0) {
                    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
                    for (int z = 0; z < 3; ++z) {
                        fetch_rows<int8_t, WIDE, R, ACROSS, V>(to[z][0], p.f.values + z * plane + at, live, s.cols, D, lane);
                        const uint8_t *scale = p.f.scales + z * scales + (s.b * groups + t0 / kGroup) * D + s.c0;
                        unsigned char *row = sh.scale[step & 1][warp][z];
                        if constexpr (WIDE) {
                            if (lane * 4 < s.cols) copy<4>(tc::smem_u32(row + lane * 4), scale + lane * 4);
                        } else {
                            fetch_rows<uint8_t, false, 1, kTile + 4>(row, scale, 1, s.cols, D, lane);
                        }
                    }
                }
            } else {
                fetch_rows<T, WIDE, R, ACROSS>(to[0][0], (const T *)p.f.x + at, live, s.cols, D, lane);
                fetch_rows<T, WIDE, R, ACROSS>(to[1][0], (const T *)p.f.r + at, live, s.cols, D, lane);
                fetch_rows<T, WIDE, R, ACROSS>(to[2][0], (const T *)p.f.i + at, live, s.cols, D, lane);
            }
            fetch_rows<T, WIDE, R, ACROSS>(to[3][0], (const T *)p.dy + at, live, s.cols, D, lane);
            if (warp == 0) {  // the state that enters the block's tokens: read behind the block's barrier
                const float *state = p.f.states + (s.b * chunks + t0 / kState) * D + s.c0;
#pragma unroll
                for (int c = lane; c < kTile; c += 32)
                    if (c < s.cols) copy<4>(tc::smem_u32(&sh.state[step & 3][c]), state + c);
            }
        }
        copy_commit();
    };
    fetch(0);
    fetch(1);
    uint64_t carry = 0, sum = 0;
    Rate2 rate{};
    bool steep = false, alive = true;
    for (int step = 0;; ++step) {
        const Step s = sh.step[step & 3];
        if (s.cols == 0) break;
        if (threadIdx.x == 0) tc::mbar_arrive_expect_tx(&sh.exchange.bar[step & 1], blocks * 32 * (uint32_t)sizeof(Run2));
        const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
        const int64_t t0 = (int64_t)s.first + mine, at = s.base + mine * D + 2 * lane;
        const int live = t0 < 0 ? 0 : run_of(R, s.len, t0), rows = t0 < 0 ? 0 : run_of(R, L, t0);
        auto &in = sh.row[step & 1][warp];
        if (s.first == (chunks - blocks) * kState) {
            const int64_t c = s.c0 + 2 * lane;
            float k0 = one ? p.f.lam[c] : 0.f, k1 = both ? p.f.lam[c + 1] : 0.f;
            carry = p.dfinal ? f2(one ? p.dfinal[s.b * D + c] : 0.f, both ? p.dfinal[s.b * D + c + 1] : 0.f) : 0;
            sum = 0;
            k0 = p.f.c * softplus(k0), k1 = p.f.c * softplus(k1);
            rate = Rate2::of(k0, k1);
            steep = __any_sync(0xffffffffu, (one && !(k0 < kSteep)) || (both && !(k1 < kSteep)));
        }
        copy_wait<1>();
        __syncwarp();
        auto shift = [&](const void *base, int64_t from, int size) {  // bytes that a row begins into its first word
            return WIDE || size == 4 ? 0 : (int)((reinterpret_cast<uintptr_t>(base) + (uintptr_t)from * size) & 3);
        };
        auto pair = [&](int z, int t) {
            const void *base = z == 0 ? p.f.x : z == 1 ? p.f.r : z == 2 ? p.f.i : p.dy;
            return row_pair<T, WIDE>(in[z][t], shift(base, at - 2 * lane + t * D, sizeof(T)), lane, both);
        };
        uint64_t scale[3];
        if constexpr (PACK) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                const Raw<uint8_t, 2> code =
                    row_pair<uint8_t, WIDE>(sh.scale[step & 1][warp][z], shift(p.f.scales, z * scales + (s.b * groups + t0 / kGroup) * D + s.c0, 1), lane, both);
                scale[z] = f2(scale_of(code.v[0]), scale_of(code.v[1]));
            }
        }
        auto value = [&](int z, int t) {
            if constexpr (PACK) {
                const Raw<int8_t, 2> q = row_pair<int8_t, WIDE>(in[z][t], shift(p.f.values, z * plane + at - 2 * lane + t * D, 1), lane, both);
                return from_8(q.word, scale[z]);
            } else {
                return pair_of(pair(z, t));
            }
        };
        uint64_t a[R], b[R], f[R], rho[R], d[R];
        Run2 own;   // of m, backwards
        uint64_t H;  // and of h, forwards; its A is the same
        Low<T, PACK> low;
        auto tokens = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            const uint64_t minus = f2(-1.f), unit = f2(1.f);
            H = 0;
#pragma unroll
            for (int t = 0; t < R; ++t) {
                uint64_t r, i;
                if constexpr (PACK) {
                    r = value(1, t), i = value(2, t);
                    if (FAST) low.see(r, i, t == 0);
                } else {
                    const Raw<T, 2> rw = pair(1, t), iw = pair(2, t);
                    if (FAST) low.see(rw, iw, t == 0);
                    r = pair_of(rw), i = pair_of(iw);
                }
                const Gates2 g = gates2<T, FAST, true>(r, i, rate);
                a[t] = g.a, f[t] = g.f, rho[t] = g.rho;
                b[t] = mul2(g.f, value(0, t));
                d[t] = g.iota;
                if (!FAST && t >= live) a[t] = unit, b[t] = 0;
                H = fma2(a[t], H, b[t]);
            }
            own.a = unit, own.h = 0;
#pragma unroll
            for (int t = R - 1; t >= 0; --t) {
                const uint64_t dy = FAST || t < live ? pair_of(pair(3, t)) : 0;
                own.a = mul2(own.a, a[t]);
                own.h = mul2(a[t], add2(dy, own.h));
            }
        };
        bool fast = live == R && !steep;
        if (fast) {
            tokens(std::true_type{});
            fast = !__any_sync(0xffffffffu, one && low.any());
        }
        if (!fast) tokens(std::false_type{});
        sh.run[step & 1][warp][lane] = own;
        sh.h[step & 1][warp][lane] = H;
        __syncthreads();
        Run2 before{f2(1.f), 0}, all = before;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) {
            if (w == warp) before = all;
            all = after(all, sh.run[step & 1][w][lane]);
        }
        exchange_send(sh.exchange, step, rank, blocks, warp, warps, lane, all);
        if (threadIdx.x == 0) sh.step[(step + 3) & 3] = walk.backward(p.f, blocks * kState, (chunks - blocks) * kState);
        // h, from the block's state over the earlier runs (the later warps') to this one; with it what multiplies dh in psi
        uint64_t h = f2(sh.state[step & 3][2 * lane], sh.state[step & 3][2 * lane + 1]);
        for (int w = warps - 1; w > warp; --w) h = fma2(sh.run[step & 1][w][lane].a, h, sh.h[step & 1][w][lane]);
        {
            const uint64_t minus = f2(-1.f), unit = f2(1.f);
#pragma unroll
            for (int t = 0; t < R; ++t) {
                const uint64_t w2 = mul2(rho[t], rate.twice), g = grad_ratio(w2, a[t], steep);
                const uint64_t c = fma2(mul2(mul2(a[t], w2), f2(-0.5f)), h, mul2(g, b[t]));  // g b - a w h
                h = fma2(a[t], h, b[t]);
                d[t] = mul2(b[t], fma2(d[t], minus, unit));
                b[t] = c;
                rho[t] = fma2(rho[t], minus, unit);
            }
        }
        alive = exchange_wait(sh.exchange, step, alive);
        if (!alive) carry = f2(__uint_as_float(0x7fc00000u));  // what was not told is not guessed
        uint64_t m = carry;                                     // that comes to this run from the later ones
#pragma unroll 4
        for (int j = 0; j < blocks; ++j) {
            if (j == rank) m = carry;
            carry = after(sh.exchange.block[step & 1][j][lane], carry);
        }
        m = after(before, m);
        auto results = [&](auto whole) {
#pragma unroll
            for (int t = R - 1; t >= 0; --t) {
                constexpr bool ALL = decltype(whole)::value;
                const uint64_t dh = add2(m, ALL || t < live ? pair_of(pair(3, t)) : 0), psi = mul2(dh, b[t]);
                const uint64_t out[3] = {mul2(dh, f[t]), mul2(psi, rho[t]), mul2(dh, d[t])};
                if (ALL || t < live) sum = add2(sum, psi);
                m = mul2(a[t], dh);
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    float v0, v1;
                    un2(out[z], v0, v1);
                    if (!ALL && t >= live) v0 = v1 = 0.f;
                    Raw<T, 2> v;
                    v.v[0] = from_f32<T>(v0), v.v[1] = from_f32<T>(v1);
                    if constexpr (WIDE) {
                        *reinterpret_cast<decltype(v.word) *>(in[z][t] + 2 * sizeof(T) * lane) = v.word;
                    } else {
                        if (t < rows) store_pair<T, WIDE>((T *)(z == 0 ? p.dx : z == 1 ? p.dr : p.di) + at + t * D, v, one, both);
                    }
                }
            }
        };
        __syncwarp();  // the rows of x, r and i have been read
        if (live == R) results(std::true_type{}); else results(std::false_type{});
        __syncwarp();
        if constexpr (WIDE) {
            leave_rows<T, T, R, ACROSS>(in[0][0], (T *)p.dx + at - 2 * lane, rows, s.cols, D, lane);
            leave_rows<T, T, R, ACROSS>(in[1][0], (T *)p.dr + at - 2 * lane, rows, s.cols, D, lane);
            leave_rows<T, T, R, ACROSS>(in[2][0], (T *)p.di + at - 2 * lane, rows, s.cols, D, lane);
            __syncwarp();
        }
        fetch(step + 2);
        if (s.first <= 0) {  // the sequence is done
            sh.sum[warp][lane] = sum;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < warps; ++w) sum = add2(sum, sh.sum[w][lane]);
                float s0, s1;
                un2(sum, s0, s1);
                store_pair<float, WIDE>(p.part + (s.b * blocks + rank) * D + s.c0 + 2 * lane, s0, s1, one, both);
                if (rank == 0 && p.dinit) {
                    un2(carry, s0, s1);
                    store_pair<float, WIDE>(p.dinit + s.b * D + s.c0 + 2 * lane, s0, s1, one, both);
                }
            }
        }
    }
    copy_wait<0>();
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
    const float *lam = p.lam + c0, *state = p.state + slot * p.D + c0;
    auto two = [&](const Raw<T, V> &w) { return f2(to_f32(w.v[0]), to_f32(w.v[V - 1])); };
    const Rate2 k = Rate2::of(p.c * softplus(lam[0]), p.c * softplus(lam[V - 1]));
    const Gates2 g = gates2<T, false, false>(two(r), two(i), k);
    float h0, h1;
    un2(fma2(g.a, f2(state[0], state[V - 1]), mul2(g.f, two(x))), h0, h1);
    h[V - 1] = h1, h[0] = h0;
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

// Clusters of `blocks` blocks of KERN that the device holds at once; asked of the driver once per device and size.
template <auto KERN> cudaError_t clusters_at_once(int blocks, int threads, size_t smem, int *count) {
    static std::atomic<int> known[64][kMaxCluster + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> *slot = dev < 64 ? &known[dev][blocks] : nullptr;
    if (slot && (*count = slot->load(std::memory_order_acquire)) > 0) return cudaSuccess;
    e = allow_shared<KERN>(smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(KERN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)blocks), cfg.blockDim = dim3((unsigned)threads), cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr, cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(count, KERN, &cfg);
    if (e == cudaSuccess && slot) slot->store(*count, std::memory_order_release);
    return e;
}

// Launches KERN over `items` sequences and tiles of `L` tokens in blocks of `tokens`. The cluster's size: the one whose waves
// times steps are fewest, a step of a cluster counted a tenth dearer than one of a single block for the meeting.
template <auto KERN, typename Args> cudaError_t launch_clusters(const Args &a, int64_t items, int64_t L, int most, int warps, int run, size_t smem, cudaStream_t stream,
                                                         int *blocks_taken = nullptr) {
    const int64_t tokens = (int64_t)warps * run, need = (L + tokens - 1) / tokens;
    int best = 1, held = 1;
    double cost = 0;
    for (int blocks = 1; blocks <= most && blocks <= need; ++blocks) {
        int count = 0;
        cudaError_t e = clusters_at_once<KERN>(blocks, kThreads, smem, &count);
        if (e != cudaSuccess) return e;
        if (count < 1) continue;
        const double c = (double)((items + count - 1) / count) * (double)((need + blocks - 1) / blocks) * (blocks > 1 ? 1.1 : 1.0);
        if (blocks == 1 || c < cost) best = blocks, held = count, cost = c;
    }
    if (blocks_taken) *blocks_taken = best;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)best, attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(imin<int64_t>(items, held) * best)), cfg.blockDim = dim3((unsigned)(32 * warps));
    cfg.dynamicSmemBytes = smem, cfg.stream = stream, cfg.attrs = attr, cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, KERN, a);
}

// Whether every row of `t`-byte elements begins at a multiple of 16 bytes.
bool wide_rows(int64_t D, size_t t) { return D * (int64_t)t % 16 == 0; }

template <typename T, bool WIDE> cudaError_t forward_w(const LinearArgs &a, cudaStream_t stream) {
    const int64_t items = a.B * ((a.D + kTile - 1) / kTile);
    const int warps = warps_for(a.L, kFwdRun);
    const size_t smem = sizeof(FwdShared<T, WIDE>);
    return a.values ? launch_clusters<linear_fwd_kernel<T, WIDE, true>>(a, items, a.L, WIDE ? kMaxCluster : 4, warps, kFwdRun, smem, stream)
                    : launch_clusters<linear_fwd_kernel<T, WIDE, false>>(a, items, a.L, WIDE ? kMaxCluster : 4, warps, kFwdRun, smem, stream);
}
template <typename T> cudaError_t forward_t(const LinearArgs &a, cudaStream_t stream) {
    if (a.L == 0) {
        if (!a.final_state || a.final_state == a.init) return cudaSuccess;
        return launch_programmatic(linear_keep_kernel, dim3((unsigned)((a.B * a.D + 255) / 256)), dim3(256), 0, stream, a.init,
                                   a.final_state, a.B * a.D);
    }
    return wide_rows(a.D, sizeof(T)) ? forward_w<T, true>(a, stream) : forward_w<T, false>(a, stream);
}

template <typename T, bool WIDE, bool PACK> cudaError_t backward_p(const LinearBwdArgs &a, cudaStream_t stream, int *blocks) {
    const int64_t items = a.f.B * ((a.f.D + kTile - 1) / kTile);
    return launch_clusters<linear_bwd_kernel<T, WIDE, PACK>>(a, items, a.f.L, WIDE ? kMaxCluster : 4, warps_for(a.f.L, kBwdRun), kBwdRun, sizeof(BwdShared<T, WIDE, PACK>),
                                                             stream, blocks);
}
template <typename T> cudaError_t backward_t(const LinearBwdArgs &a, cudaStream_t stream) {
    cudaError_t e = cudaSuccess;
    int blocks = 0;  // none has added to the sum for dlam
    if (a.f.B > 0 && a.f.L > 0) {
        const bool wide = wide_rows(a.f.D, sizeof(T));
        e = a.f.values ? (wide ? backward_p<T, true, true>(a, stream, &blocks) : backward_p<T, false, true>(a, stream, &blocks))
                       : (wide ? backward_p<T, true, false>(a, stream, &blocks) : backward_p<T, false, false>(a, stream, &blocks));
    } else if (a.f.B > 0 && a.dinit && a.dinit != a.dfinal) {
        e = launch_programmatic(linear_keep_kernel, dim3((unsigned)((a.f.B * a.f.D + 255) / 256)), dim3(256), 0, stream, a.dfinal, a.dinit,
                                a.f.B * a.f.D);
    }
    if (e != cudaSuccess) return e;
    return launch_programmatic(linear_dlam_kernel, dim3((unsigned)((a.f.D + 31) / 32)), dim3(32, 8), 0, stream, (const float *)a.part, a.f.lam,
                               a.dlam, a.f.B * blocks, a.f.D);
}

}  // namespace linear

int64_t linear_bwd_parts(int64_t B) { return B * linear::kMaxCluster; }

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
