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
constexpr int kMaxCluster = 8;

// ------------------------------------------------------- copies to shared memory
// A warp fetches the rows of its own runs, two steps ahead, and only it reads them: no barrier but its own. WIDE: 16 bytes a
// lane, for rows that begin at a multiple of 16 bytes. Otherwise 4 bytes: the aligned words around each row, of those at the
// tensor's end and the tile's only the bytes that belong to the tensor; a row then begins up to 3 bytes into its first word.
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
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
// next in shared memory.
template <typename T, bool WIDE, int R, int ACROSS>
__device__ __forceinline__ void fetch_rows(unsigned char *to, const T *base, int n, int cols, int64_t D, int lane) {
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (WIDE) {
        constexpr int PER = kTile * (int)sizeof(T) / 16, ROWS = 32 / PER > R ? R : 32 / PER;  // lanes a row, rows at once
        const int piece = lane % PER, first = lane / PER;
        const int c = piece * (16 / (int)sizeof(T));
        if (c < cols && first < ROWS) {
            const T *from = base + first * D + c;
            const int64_t next = ROWS * D;
#pragma unroll
            for (int j = 0; j < R / ROWS; ++j, from += next)
                if (j * ROWS + first < n) copy16(dst + (j * ROWS + first) * ACROSS + piece * 16, from);
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

// A step of a cluster: the tile of a sequence that it is at, as its first thread works out two steps ahead.
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
};
// Tokens of a run of R from t0 on that are below `end`.
__device__ __forceinline__ int run_of(int R, int64_t end, int64_t t0) { return (int)imax<int64_t>(0, imin<int64_t>(R, end - t0)); }

// The blocks of a cluster exchange a Run2 a lane: each sends its own to all of them, and the bytes count down the receiver's
// barrier. (A cluster barrier would have the sender wait for everything that it has written to memory before.) Two of each,
// taken in turn: a block sends for a step once all of its warps have read the one before.
struct Exchange {
    Run2 block[2][kMaxCluster][32];
    uint64_t bar[2];
};
constexpr uint64_t kGiveUpNs = 1000000000ull;
__device__ int g_gave_up;  // SSD_ERR_TIMEOUT once a wait was given up on this device

__device__ __forceinline__ void exchange_init(Exchange &x, int blocks) {
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
__device__ __forceinline__ void exchange_send(Exchange &x, int step, int rank, int blocks, int lane, const Run2 &own) {
    const uint32_t slot = tc::smem_u32(&x.block[step & 1][rank][lane]), bar = tc::smem_u32(&x.bar[step & 1]);
    uint32_t r0, r1, r2, r3;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r0), "=r"(r1) : "l"(own.a));
    asm("mov.b64 {%0, %1}, %2;" : "=r"(r2), "=r"(r3) : "l"(own.h));
    for (int j = 0; j < blocks; ++j)
        asm volatile(
            "{\n\t.reg .b32 to, at;\n\t"
            "mapa.shared::cluster.u32 to, %0, %2;\n\t"
            "mapa.shared::cluster.u32 at, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [to], {%3, %4, %5, %6}, [at];\n\t}" ::"r"(slot),
            "r"(bar), "r"(j), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
            : "memory");
}
// False, now and from then on, where the others' runs have not come in kGiveUpNs.
__device__ __forceinline__ bool exchange_wait(Exchange &x, int step, bool alive) {
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
    Run2 run[kWarps][32];
    Exchange exchange;
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
    if (threadIdx.x == 0) sh.step[0] = walk.forward(p, span), sh.step[1] = walk.forward(p, span);
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
    uint64_t carry = 0, rate2 = 0, rate_log2 = 0;
    bool steep = false, alive = true;
    for (int step = 0;; ++step) {
        const Step s = sh.step[step & 3];
        if (s.cols == 0) break;
        if (threadIdx.x == 0) {
            sh.step[(step + 2) & 3] = walk.forward(p, span);
            tc::mbar_arrive_expect_tx(&sh.exchange.bar[step & 1], blocks * 32 * (uint32_t)sizeof(Run2));
        }
        const bool one = 2 * lane < s.cols, both = 2 * lane + 1 < s.cols;
        const int64_t t0 = (int64_t)s.first + mine, at = s.base + mine * D + 2 * lane;
        const int live = run_of(R, s.len, t0), rows = run_of(R, L, t0);  // tokens that count, that exist
        auto &in = sh.row[step & 1][warp];
        if (s.first == 0) {
            const int64_t c = s.c0 + 2 * lane;
            float k0 = one ? p.lam[c] : 0.f, k1 = both ? p.lam[c + 1] : 0.f;
            carry = p.init ? f2(one ? p.init[s.b * D + c] : 0.f, both ? p.init[s.b * D + c + 1] : 0.f) : 0;
            k0 = p.c * softplus(k0), k1 = p.c * softplus(k1);
            rate2 = f2(2.f * k0, 2.f * k1), rate_log2 = f2(kLog2e * k0, kLog2e * k1);
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
                const Gates2 g = gates2<T, FAST>(pair_of(r), pair_of(i), rate2, rate_log2);
                a[t] = g.a;
                h[t] = mul2(mul2(mul2(g.beta2, g.rbeta), g.iota), pair_of(pair(0, t)));
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
        sh.run[warp][lane] = own;
        __syncthreads();
        Run2 before{f2(1.f), f2(0.f)};  // the block's runs before this one
        for (int w = 0; w < warp; ++w) before = after(before, sh.run[w][lane]);
        if (warp == warps - 1) exchange_send(sh.exchange, step, rank, blocks, lane, after(before, own));
        alive = exchange_wait(sh.exchange, step, alive);
        if (!alive) carry = f2(__uint_as_float(0x7fc00000u));  // what was not told is not guessed
        uint64_t e = carry;                                     // the state that enters this run
        for (int j = 0; j < rank; ++j) e = after(sh.exchange.block[step & 1][j][lane], e);
        carry = e;
        for (int j = rank; j < blocks; ++j) carry = after(sh.exchange.block[step & 1][j][lane], carry);
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
// dh_t = dy_t + m_{t+1}, m_t = a_t dh_t (m behind the last token the gradient of the final state): the same kind of
// recurrence, backwards, a run acting as m -> A m + M. With psi_t = w_t dL/dw_t:
//     dx = dh beta iota     di = dh b (1 - iota)     psi = dh (a^2 b w / beta^2 - a w h_{t-1})     dr = psi (1 - rho)
//     dlam = sigmoid(lam) / softplus(lam) sum psi
// (psi rather than dL/dw, which has 1 / beta: w / beta goes to zero with w.) h_{t-1} is formed again from the state that
// enters each kState tokens. A block goes over its sequence from the end, kState tokens at a time.
__device__ __forceinline__ float one_minus_a2(float w, float a) {
    const float t = 2.f * w;
    float p = fmaf(t, 0.0067828623577952385f, -0.0410132110118866f);
    p = fmaf(t, p, 0.16655193269252777f);
    p = fmaf(t, p, -0.49999287724494934f);
    p = fmaf(t, p, 0.9999999403953552f);
    return t < 0.5f ? t * p : fmaf(-a, a, 1.f);
}
template <typename T, int V, bool PACK> __global__ void __launch_bounds__(kThreads) linear_bwd_kernel(LinearBwdArgs p) {
    pdl_enter();
    constexpr int R = kBwdRun;
    __shared__ float run[3][kWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t c0 = ((int64_t)blockIdx.y * 32 + lane) * V, b = blockIdx.z, D = p.f.D, L = p.f.L;
    const bool on = c0 < D;
    const int64_t len = seq_len(p.f.seqlens, b, L), n = p.f.B * L * D, groups = (L + kGroup - 1) / kGroup;
    float k[V], carry[V], sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        k[v] = on ? p.f.c * softplus(p.f.lam[c0 + v]) : 0.f;
        carry[v] = on && p.dfinal ? p.dfinal[b * D + c0 + v] : 0.f;
        sum[v] = 0.f;
    }
    for (int64_t chunk = (L + kState - 1) / kState - 1; chunk >= 0; --chunk) {
        const int64_t t0 = chunk * kState + warp * R, at = (b * L + t0) * D + c0;
        const int live = on ? (int)imax<int64_t>(0, imin<int64_t>(R, len - t0)) : 0;
        const int rows = on ? (int)imax<int64_t>(0, imin<int64_t>(R, L - t0)) : 0;
        float a[R][V], bb[R][V], rho[R][V], iota[R][V], dy[R][V], A[V], H[V], M[V];
        float scale[3][V];
        if constexpr (PACK) {
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                Raw<uint8_t, V> code;
                if (live > 0) code = load<uint8_t, V>(p.f.scales + ((z * p.f.B + b) * groups + t0 / kGroup) * D + c0);
#pragma unroll
                for (int v = 0; v < V; ++v) scale[z][v] = scale_of(code.v[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            float x[V], r[V], i[V];
            Raw<T, V> d;
            if (t < live) d = load<T, V>((const T *)p.dy + at + t * D);
            if constexpr (PACK) {
                Raw<int8_t, V> q[3];
#pragma unroll
                for (int z = 0; z < 3; ++z)
                    if (t < live) q[z] = load<int8_t, V>(p.f.values + z * n + at + t * D);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    x[v] = (float)q[0].v[v] * scale[0][v];
                    r[v] = (float)q[1].v[v] * scale[1][v];
                    i[v] = (float)q[2].v[v] * scale[2][v];
                }
            } else {
                Raw<T, V> q[3];
                if (t < live) {
                    q[0] = load<T, V>((const T *)p.f.x + at + t * D);
                    q[1] = load<T, V>((const T *)p.f.r + at + t * D);
                    q[2] = load<T, V>((const T *)p.f.i + at + t * D);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) x[v] = to_f32(q[0].v[v]), r[v] = to_f32(q[1].v[v]), i[v] = to_f32(q[2].v[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gates g = gates<T>(r[v], i[v], k[v]);
                a[t][v] = t < live ? g.a : 1.f;
                bb[t][v] = t < live ? g.beta2 * g.rbeta * g.iota * x[v] : 0.f;
                rho[t][v] = g.rho, iota[t][v] = g.iota, dy[t][v] = to_f32(d.v[v]);
                A[v] *= a[t][v];
                H[v] = fmaf(a[t][v], H[v], bb[t][v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            M[v] = 0.f;
#pragma unroll
            for (int t = R - 1; t >= 0; --t) M[v] = a[t][v] * (dy[t][v] + M[v]);
        }
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) {
            run[0][warp][lane * V + v] = A[v];
            run[1][warp][lane * V + v] = H[v];
            run[2][warp][lane * V + v] = M[v];
        }
        __syncthreads();
        float h[V], m[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = on ? p.f.states[(b * ((L + kState - 1) / kState) + chunk) * D + c0 + v] : 0.f;
            for (int w = 0; w < warp; ++w) h[v] = fmaf(run[0][w][lane * V + v], h[v], run[1][w][lane * V + v]);
            m[v] = carry[v];
            for (int w = warps - 1; w >= 0; --w) {
                if (w == warp) m[v] = carry[v];
                carry[v] = fmaf(run[0][w][lane * V + v], carry[v], run[2][w][lane * V + v]);
            }
        }
        float before[R][V];
#pragma unroll
        for (int t = 0; t < R; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[t][v] = h[v];
                h[v] = fmaf(a[t][v], h[v], bb[t][v]);
            }
#pragma unroll
        for (int t = R - 1; t >= 0; --t) {
            float dx[V], dr[V], di[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float av = a[t][v], w = k[v] * rho[t][v], beta2 = one_minus_a2(w, av);
                const float rb = rsqrt_approx(fmaxf(beta2, 1e-37f));
                const float dh = dy[t][v] + m[v];
                const float psi = dh * av * w * (av * bb[t][v] * rb * rb - before[t][v]);
                dx[v] = dh * beta2 * rb * iota[t][v];
                di[v] = dh * bb[t][v] * (1.f - iota[t][v]);
                dr[v] = psi * (1.f - rho[t][v]);
                if (t < live) {
                    sum[v] += psi;
                } else {
                    dx[v] = dr[v] = di[v] = 0.f;
                }
                m[v] = av * dh;
            }
            if (t < rows) {
                store_f32<T, V>((T *)p.dx + at + t * D, dx);
                store_f32<T, V>((T *)p.dr + at + t * D, dr);
                store_f32<T, V>((T *)p.di + at + t * D, di);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) run[0][warp][lane * V + v] = sum[v];
    __syncthreads();
    if (!on || warp != 0) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += run[0][w][lane * V + v];
        p.part[b * D + c0 + v] = s;
        if (p.dinit) p.dinit[b * D + c0 + v] = carry[v];
    }
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
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const Gates g = gates<T>(to_f32(r.v[v]), to_f32(i.v[v]), p.c * softplus(p.lam[c0 + v]));
        h[v] = fmaf(g.a, p.state[slot * p.D + c0 + v], g.beta2 * g.rbeta * g.iota * to_f32(x.v[v]));
    }
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
template <auto KERN, typename Args> cudaError_t launch_clusters(const Args &a, int64_t items, int64_t L, int warps, int run, size_t smem, cudaStream_t stream) {
    const int64_t tokens = (int64_t)warps * run, need = (L + tokens - 1) / tokens;
    int best = 1, held = 1;
    double cost = 0;
    for (int blocks = 1; blocks <= kMaxCluster && blocks <= need; ++blocks) {
        int count = 0;
        cudaError_t e = clusters_at_once<KERN>(blocks, kThreads, smem, &count);
        if (e != cudaSuccess) return e;
        if (count < 1) continue;
        const double c = (double)((items + count - 1) / count) * (double)((need + blocks - 1) / blocks) * (blocks > 1 ? 1.1 : 1.0);
        if (blocks == 1 || c < cost) best = blocks, held = count, cost = c;
    }
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
    return a.values ? launch_clusters<linear_fwd_kernel<T, WIDE, true>>(a, items, a.L, warps, kFwdRun, smem, stream)
                    : launch_clusters<linear_fwd_kernel<T, WIDE, false>>(a, items, a.L, warps, kFwdRun, smem, stream);
}
template <typename T> cudaError_t forward_t(const LinearArgs &a, cudaStream_t stream) {
    if (a.L == 0) {
        if (!a.final_state || a.final_state == a.init) return cudaSuccess;
        return launch_programmatic(linear_keep_kernel, dim3((unsigned)((a.B * a.D + 255) / 256)), dim3(256), 0, stream, a.init,
                                   a.final_state, a.B * a.D);
    }
    return wide_rows(a.D, sizeof(T)) ? forward_w<T, true>(a, stream) : forward_w<T, false>(a, stream);
}

template <typename T> cudaError_t backward_t(const LinearBwdArgs &a, cudaStream_t stream) {
    return for_width(a.f.D, [&](auto vw) {
        constexpr int V = decltype(vw)::value;
        cudaError_t e = cudaSuccess;
        if (a.f.B > 0) {
            const dim3 grid(1, tiles(a.f.D, V), (unsigned)a.f.B), block(32 * warps_for(a.f.L, kBwdRun));
            e = a.f.values ? launch_programmatic(linear_bwd_kernel<T, V, true>, grid, block, 0, stream, a)
                           : launch_programmatic(linear_bwd_kernel<T, V, false>, grid, block, 0, stream, a);
        }
        if (e != cudaSuccess) return e;
        return launch_programmatic(linear_dlam_kernel, dim3((unsigned)((a.f.D + 31) / 32)), dim3(32, 8), 0, stream,
                                   (const float *)a.part, a.f.lam, a.dlam, a.f.B, a.f.D);
    });
}

}  // namespace linear

int64_t linear_bwd_parts(int64_t B) { return B; }

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
