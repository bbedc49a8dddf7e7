// The gated linear recurrence, channel by channel:
//
//     h_t = a_t h_{t-1} + b_t x_t
//
// with a given and b = 1, or a = 1 / (1 + exp(-g)) and b = 1 - a, and its
// gradients
//
//     G_t = dh_t + a_{t+1} G_{t+1},  dx = b G,  da = G (h_{t-1} - [sigmoid] x),
//     dg = da a b,  dh0 = a_1 G_1
//
// Bound by memory: 6 bytes a value forward (sigmoid, bf16), 10 backward (8 sequences
// of 4096 tokens and 2048 channels: 63 us, 94 % of the copy bandwidth, and 114 us,
// 87 %).  What a piece of tokens does to the state is h -> P h + H, and pieces
// compose: a CTA owns 64 channels of a stream of tokens and takes tiles of 8 R of
// them, each of its 8 warps a run of R consecutive tokens, a lane two channels.  A
// warp finds P and H of its run, the runs' are joined through shared memory, and a
// second walk over the values, still in registers, gives the outputs: the inputs
// are read once.  Gradients go the other way with the same P: what leaves a run
// towards earlier tokens is u -> P u + V; the states h_{t-1} that they need start
// from those that the forward pass kept every 64 tokens, a tile of the gradients.
//
// Few streams of few channels: a cluster of 2 to 8 CTAs takes consecutive tiles
// of one stream, and every CTA sends its tile's P and H to the others' shared
// memory, so that a long sequence is still read once (65536 tokens 160 us, 99 %).
// With fewer than 1.5 CTAs an SM a cluster is doubled (clusters of 4 and one CTA an SM:
// 176 us).
//
// A stream is one sequence, or several: packed ones (a table gives each token's
// sequence) or dense ones of up to 64 tokens, whole ones in a tile and without clusters.
// There a run knows which of its tokens
// start or end a sequence or belong to none; a start takes h0 in the place of the
// state that arrives, by selection, never by a factor of 0 (a NaN would pass).
#include <cudaTypedefs.h>

#include "gdn_pair.cuh"
#include "gdn_sm100.cuh"

namespace gdn {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

using namespace sm100;

constexpr int kChannels = 64;  // of a CTA
constexpr int kWarps = 8;      // runs of a tile
constexpr int kScanThreads = kWarps * 32;
constexpr long long kWaitLimit = 2000000000LL;  // about 1 s of SM clocks
constexpr long long kDrainLimit = kWaitLimit / 16;

// a and b of a gate.  b = 1 - a is formed without the difference: a near 1
// would leave nothing of it.
template <bool SIG> __device__ __forceinline__ void gate_ab(float g, float &a, float &b) {
    if constexpr (!SIG) {
        a = g;
        b = 1.f;
    } else {
        const float e = expf(-fabsf(g)), r = 1.f / (1.f + e), s = e * r;
        a = g < 0.f ? s : r;
        b = g < 0.f ? r : s;
    }
}
// The same of two bf16 gates, by the fast exp and quotient; they are held at -87:
// exp(87) stays a number and so does b.
__device__ __forceinline__ void gate_ab2(uint32_t w, Pair &a, Pair &b) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0xc2aec2aeu));
    const float2 g = split(mul2(unpack(w), both(-1.4426950408889634f)));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(g.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(g.y));
    const Pair ep = pair(e.x, e.y), minus_d = fma2(ep, both(-1.f), both(-1.f));
    const float2 d = split(minus_d);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(-d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(-d.y));
    // one step of Newton's: products of thousands of a's gather a quotient's bias (1e-6
    // of an end state for 1e-7)
    const Pair q = pair(r.x, r.y);
    a = fma2(fma2(minus_d, q, both(1.f)), q, q);
    b = mul2(ep, a);
}

template <typename T, bool SIG> struct GateType { using type = T; };
template <typename T> struct GateType<T, false> { using type = float; };

// a and b of a lane's gates in shared memory (without a sigmoid b is not used).
template <typename T, bool SIG>
__device__ __forceinline__ void gates2(const typename GateType<T, SIG>::type *p, Pair &a, Pair &b) {
    if constexpr (!SIG) {
        a = load2(p);
        b = a;
    } else if constexpr (sizeof(T) == 2) {
        gate_ab2(*reinterpret_cast<const uint32_t *>(p), a, b);
    } else {
        const float2 g = *reinterpret_cast<const float2 *>(p);
        float2 x, y;
        gate_ab<SIG>(g.x, x.x, y.x);
        gate_ab<SIG>(g.y, x.y, y.y);
        a = pair(x.x, x.y);
        b = pair(y.x, y.y);
    }
}

// Tokens of a warp's run and tiles in flight, by the bytes of a token's channel.
// (Registers hold two or three float32 a token and channel.)
template <typename T, bool SIG, bool BACK> struct Shape {
    using G = typename GateType<T, SIG>::type;
    static constexpr int kRun = !BACK && sizeof(T) == 2 ? 16 : 8;
    static constexpr int kTokens = kRun * kWarps;  // of a tile
    static constexpr int kXBytes = kTokens * kChannels * (int)sizeof(T);
    static constexpr int kGBytes = kTokens * kChannels * (int)sizeof(G);
    static constexpr int kStage = kXBytes * (BACK ? 2 : 1) + kGBytes;
    // two CTAs an SM: a third tile of 48 KB would leave one (float32 gradients 143 -> 115 us)
    static constexpr int kStages = BACK && kStage <= 32768 ? 3 : 2;
    // most CTAs of a cluster: the totals of more would leave one CTA an SM
    static constexpr int kCluster = BACK && kStages * kStage > 81920 ? 4 : 8;
};

struct ScanRun {
    const float *h0, *dh_T;
    float *states;
    void *h, *dx, *dgate;
    float *h_T, *dh0;
    const int *map;    // packed: the sequence of each token, or -1
    int D, groups, cluster;
    int total;         // tokens
    int stream;        // tokens of a stream
    int step;          // tokens of a tile that are its own
    int rows;          // tokens of a box
    int T, blocks;     // dense sequences: tokens, and kept states
    int *status;
};
// Self-test (kernels of their own): the clocks of a wait, and the tile of each stream that is
// not copied.
struct LostRun : ScanRun {
    long long limit;
    int lost;
};
__device__ __forceinline__ long long wait_limit(const ScanRun &) { return kWaitLimit; }
__device__ __forceinline__ long long wait_limit(const LostRun &p) { return p.limit; }
__device__ __forceinline__ bool is_lost(const ScanRun &, int) { return false; }
__device__ __forceinline__ bool is_lost(const LostRun &p, int tile) { return tile == p.lost; }

struct Piece {         // what a run or a tile does to a lane's channels: c -> p c + h
    Pair p, h;
};
template <int N> struct Totals {  // of a tile, sent through a cluster
    Piece piece[2][N][32];
    int reset[2][N];
};
template <typename S, bool BACK, bool CLUSTER> struct ScanShared {
    Piece run[2][kWarps][32];
    Pair state[BACK ? 2 : 1][BACK ? kWarps : 1][32];  // backward: the forward pass's h
    int reset[2][kWarps];  // bit 0: a start among the run's tokens, bit 1: an end
    Totals<S::kCluster> totals[CLUSTER ? 1 : 0];
    uint64_t full[8], sent[2];
    int abort;
};

__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, uint64_t *bar, int c,
                                         int t) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(t)
        : "memory");
}
__device__ __forceinline__ uint32_t peer(const void *p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void send4(uint32_t dst, uint32_t bar, const Piece &v) {
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(dst),
        "l"(v.p.v), "l"(v.h.v), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void send1(uint32_t dst, uint32_t bar, int v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(dst),
                 "r"(v), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// A wait with a limit; the first that runs out ends all others of the CTA.  Its threads
// walk on through their tiles, with what they have, so that all meet at every barrier.  A
// thread whose wait has run out announces and sends no more (a barrier whose phase is open
// may not be arrived at again), and nothing is fetched; without its totals the other CTAs of
// a cluster run out in turn.
template <bool CLUSTER, typename RUN>
__device__ __forceinline__ bool wait_full(uint64_t *bar, uint32_t parity, int *abort, const RUN &p) {
    auto ready = [&] { return CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (ready()) return true;
    const long long t0 = clock64();
    volatile int *const flag = abort;
    while (!ready()) {
        if (*flag) return false;
        if (clock64() - t0 > wait_limit(p)) {
            *flag = 1;
            if (p.status) atomicOr(p.status, kStatusTimeout);
            return false;
        }
    }
    return true;
}
// After one that ran out: copies in flight, and totals that other CTAs have sent, land before
// the CTA ends.
__device__ __forceinline__ void drain(uint64_t *bar, int n) {
    for (int i = 0; i < n; ++i) {
        mbar_wait(&bar[i], 0, kDrainLimit);
        mbar_wait(&bar[i], 1, kDrainLimit);
    }
}

// The state after a piece.
__device__ __forceinline__ void over(Pair &c, const Piece &k, bool reset) {
    c = either(reset, k.h, fma2(k.p, c, k.h));
}
// Two pieces as one.
__device__ __forceinline__ void join(Piece &t, const Piece &k, bool reset) {
    over(t.h, k, reset);
    t.p = mul2(t.p, k.p);
}

// f with the warp's number as a constant: the walks over the other runs' pieces
// are straight lines then (as loops they were a third of the gradients' instructions).
template <int N> struct Number { static constexpr int value = N; };
template <typename F> __device__ __forceinline__ void as_constant(int warp, F &&f) {
    switch (warp) {
        case 0: f(Number<0>()); break;
        case 1: f(Number<1>()); break;
        case 2: f(Number<2>()); break;
        case 3: f(Number<3>()); break;
        case 4: f(Number<4>()); break;
        case 5: f(Number<5>()); break;
        case 6: f(Number<6>()); break;
        default: f(Number<7>()); break;
    }
}

// Which of a run's tokens are in a sequence, start one, end one; lane l holds
// the sequence of token l - 1 of the run.
struct RunMask {
    unsigned act, start, end;
    int seq;
};
// The sequence of this lane's token, ahead of the tile that needs it.  tile0: the
// tile's first token in the stream (unsigned: one ahead of a stream's end may lie past
// 2^31, one before its start below 0), r0: the run's in the tile.
template <bool MASKED, int R>
__device__ __forceinline__ int run_entry(const ScanRun &p, int base, int len, unsigned tile0, int r0) {
    if constexpr (!MASKED) return 0;
    const int lane = threadIdx.x & 31, k = r0 + lane - 1;
    const unsigned t = tile0 + (unsigned)k;
    if (lane >= R + 2 || t >= (unsigned)len) return -1;
    if (p.map) return p.map[t];
    // whole sequences in a tile: a neighbour is one of the tile's own tokens
    return k >= 0 && k < p.step ? (base + (int)t) / p.T : -1;
}
template <bool MASKED, int R>
__device__ __forceinline__ RunMask run_mask(int seq, int len, int t0) {
    RunMask m;
    constexpr unsigned all = (1u << R) - 1u;
    m.seq = seq;
    if constexpr (!MASKED) {
        const int n = min(max(len - t0, 0), R);
        m.act = n >= R ? all : (1u << n) - 1u;
        m.start = m.end = 0;
    } else {
        const int lane = threadIdx.x & 31;
        const int before = __shfl_up_sync(0xffffffffu, seq, 1), after = __shfl_down_sync(0xffffffffu, seq, 1);
        const bool mine = seq >= 0 && lane >= 1 && lane <= R;
        m.act = (__ballot_sync(0xffffffffu, mine) >> 1) & all;
        m.start = (__ballot_sync(0xffffffffu, mine && seq != before) >> 1) & all;
        m.end = (__ballot_sync(0xffffffffu, mine && seq != after) >> 1) & all;
    }
    return m;
}
__device__ __forceinline__ int run_seq(const RunMask &m, int i) {
    return __shfl_sync(0xffffffffu, m.seq, i + 1);
}

// A tile's totals to the CTAs of the cluster: every warp has them and sends them to
// one.
template <int N>
__device__ __forceinline__ void send_totals(Totals<N> &to, uint64_t *sent, int buf, int rank, int cluster,
                                            const Piece &t, int reset) {
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    if (r >= cluster) return;
    const uint32_t bar = peer(&sent[buf], r);
    send4(peer(&to.piece[buf][rank][lane], r), bar, t);
    if (lane == 0) send1(peer(&to.reset[buf][rank], r), bar, reset);
}
__device__ __forceinline__ void expect_totals(uint64_t *sent, int buf, int cluster) {
    mbar_arrive_expect_tx(&sent[buf], cluster * (32 * sizeof(Piece) + sizeof(int)));
}
// The tiles' totals applied to c, this CTA's state of the stream before them: c
// becomes what it is after them; returns what it is before this CTA's tile.
template <bool MASKED, int N>
__device__ __forceinline__ Pair apply_totals(const Totals<N> &to, int buf, int rank, int cluster, Pair &c) {
    const int lane = threadIdx.x & 31;
    Pair mine = c;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        if (r < cluster) {
            mine = either(r == rank, c, mine);
            over(c, to.piece[buf][r][lane], MASKED && to.reset[buf][r]);
        }
    }
    return mine;
}

// ------------------------------------------------------------------ forward

template <typename T, bool SIG, bool MASKED, bool CLUSTER, typename RUN>
__global__ void __launch_bounds__(kScanThreads, 2)
    scan_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                const RUN p) {
    using S = Shape<T, SIG, false>;
    using G = typename S::G;
    constexpr int R = S::kRun, ST = S::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ScanShared<S, false, CLUSTER> sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cluster = CLUSTER ? p.cluster : 1;
    const int rank = CLUSTER ? (int)(blockIdx.x % cluster) : 0;
    const int item = CLUSTER ? (int)(blockIdx.x / cluster) : (int)blockIdx.x;
    const int stream = item / p.groups, group = item - stream * p.groups;
    const int base = stream * p.stream, len = min(p.stream, p.total - base);
    const int tiles = (len + p.step - 1) / p.step, slabs = (tiles + cluster - 1) / cluster;
    const int c0 = group * kChannels, c = c0 + 2 * lane;
    const bool live = c < p.D;
    const uint32_t bytes = p.rows * kChannels * (sizeof(T) + sizeof(G));
    auto fetch = [&](int n) {  // by one thread
        const int j = n * cluster + rank, s = n % ST;
        if (j >= tiles) return;
        mbar_arrive_expect_tx(&sh.full[s], bytes);
        if (is_lost(p, j)) return;
        load_box(smem + s * S::kStage, &mx, &sh.full[s], c0, base + j * p.step);
        load_box(smem + s * S::kStage + S::kXBytes, &mg, &sh.full[s], c0, base + j * p.step);
    };
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int s = 0; s < ST; ++s) mbar_init(&sh.full[s], 1);
        mbar_init(&sh.sent[0], 1);
        mbar_init(&sh.sent[1], 1);
        fence_mbar_init();
        for (int n = 0; n < ST; ++n) fetch(n);
    }
    const Pair zero = both(0.f), one = both(1.f);
    Pair carry = zero;
    if (!MASKED && p.h0 && live) carry = load2(p.h0 + (long long)stream * p.D + c);
    if constexpr (CLUSTER) cluster_sync();
    else __syncthreads();
    T *const out = static_cast<T *>(p.h);
    if constexpr (MASKED) pdl_wait();  // for the table
    int entry = run_entry<MASKED, R>(p, base, len, rank * p.step, warp * R);
    bool gone = false;  // a wait for totals has run out
    for (int n = 0; n < slabs; ++n) {
        const int j = n * cluster + rank, buf = n & 1, s = n % ST;
        const int tile0 = j * p.step, t0 = tile0 + warp * R;
        const RunMask m = run_mask<MASKED, R>(entry, len, t0);
        entry = run_entry<MASKED, R>(p, base, len, (unsigned)tile0 + (unsigned)(cluster * p.step), warp * R);
        if (CLUSTER && threadIdx.x == 0 && !gone) expect_totals(sh.sent, buf, cluster);
        const T *const xs = reinterpret_cast<const T *>(smem + s * S::kStage) + warp * R * kChannels + 2 * lane;
        const G *const gs = reinterpret_cast<const G *>(smem + s * S::kStage + S::kXBytes) +
                            warp * R * kChannels + 2 * lane;
        Pair a[R], u[R];
        Piece k = {one, zero};
        constexpr unsigned all = (1u << R) - 1u;
        const bool plain = m.act == all && (!MASKED || m.start == 0);
        if (MASKED && !plain) {
#pragma unroll
            for (int i = 0; i < R; ++i) {  // the starts' states, all loads in flight
                u[i] = zero;
                if (m.start >> i & 1) {
                    const long long at = (long long)run_seq(m, i) * p.D + c;
                    if (p.h0 && live) u[i] = load2(p.h0 + at);
                    // kept states of short dense sequences: their starts
                    if (!p.map && p.states && live) store2(p.states + at, u[i]);
                }
            }
        }
        if (j < tiles) wait_full<false>(&sh.full[s], (n / ST) & 1, &sh.abort, p);
        if (plain) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Pair b;
                gates2<T, SIG>(gs + i * kChannels, a[i], b);
                u[i] = load2(xs + i * kChannels);
                if constexpr (SIG) u[i] = mul2(b, u[i]);
                k.p = mul2(k.p, a[i]);
                k.h = fma2(a[i], k.h, u[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in = m.act >> i & 1, start = MASKED && (m.start >> i & 1);
                Pair b, x = load2(xs + i * kChannels);
                gates2<T, SIG>(gs + i * kChannels, a[i], b);
                if constexpr (SIG) x = mul2(b, x);
                if (start) x = fma2(a[i], u[i], x);
                u[i] = either(in, x, zero);
                a[i] = either(in, a[i], one);
                k.p = mul2(k.p, a[i]);
                k.h = either(start, u[i], fma2(a[i], k.h, u[i]));
            }
        }
        sh.run[buf][warp][lane] = k;
        if (MASKED && lane == 0) sh.reset[buf][warp] = m.start != 0;
        __syncthreads();
        // the stage is in registers
        if (threadIdx.x == 0 && !sh.abort) fetch(n + ST);
        Pair h = carry;
        auto reset = [&](int w) { return MASKED ? sh.reset[buf][w] : 0; };
        if constexpr (CLUSTER) {
            Piece before = {one, zero}, t;
            int cut = 0, all_cut;
            as_constant(warp, [&](auto number) {
                constexpr int W = decltype(number)::value;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    join(before, sh.run[buf][w][lane], reset(w));
                    cut |= reset(w);
                }
                t = before;
                all_cut = cut;
#pragma unroll
                for (int w = W; w < kWarps; ++w) {
                    join(t, sh.run[buf][w][lane], reset(w));
                    all_cut |= reset(w);
                }
            });
            auto &to = sh.totals[0];
            if (!gone) send_totals(to, sh.sent, buf, rank, cluster, t, all_cut);
            if (!wait_full<true>(&sh.sent[buf], (n >> 1) & 1, &sh.abort, p)) gone = true;
            h = apply_totals<MASKED>(to, buf, rank, cluster, carry);
            over(h, before, cut);
        } else {
            as_constant(warp, [&](auto number) {
                constexpr int W = decltype(number)::value;
#pragma unroll
                for (int w = 0; w < W; ++w) over(h, sh.run[buf][w][lane], reset(w));
                carry = h;
#pragma unroll
                for (int w = W; w < kWarps; ++w) over(carry, sh.run[buf][w][lane], reset(w));
            });
        }
        // the state before every 64th token
        const bool mapped = !MASKED || p.map;
        if (p.states && mapped && t0 % kScanBlock == 0 && t0 < len && live)
            store2(p.states + ((MASKED ? 0 : (long long)stream * p.blocks) + t0 / kScanBlock) * p.D + c, h);
        T *o = out + ((long long)(base + t0) * p.D + c);
        if (plain && (!MASKED || m.end == 0)) {
            if (out && live) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    h = fma2(a[i], h, u[i]);
                    store2(o + (long long)i * p.D, h);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in = m.act >> i & 1, start = MASKED && (m.start >> i & 1);
                h = either(start, u[i], fma2(a[i], h, u[i]));
                if (out && live && in) store2(o + (long long)i * p.D, h);
                if (MASKED && p.h_T && (m.end >> i & 1)) {
                    const long long at = (long long)run_seq(m, i) * p.D + c;
                    if (live) store2(p.h_T + at, h);
                }
            }
        }
    }
    if (!MASKED && p.h_T && rank == 0 && warp == 0 && live)
        store2(p.h_T + (long long)stream * p.D + c, carry);
    if (sh.abort && threadIdx.x == 0) {
        drain(sh.full, ST);
        if constexpr (CLUSTER) drain(sh.sent, 2);
    }
    if constexpr (CLUSTER) cluster_sync();  // no CTA sends to one that has ended
}

// ------------------------------------------------------------------ backward

// Tiles last to first: rank 0 of a cluster has the latest.
template <typename T, bool SIG, bool MASKED, bool CLUSTER, typename RUN>
__global__ void __launch_bounds__(kScanThreads, 2)
    scan_backward_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                         const __grid_constant__ CUtensorMap md, const RUN p) {
    using S = Shape<T, SIG, true>;
    using G = typename S::G;
    constexpr int R = S::kRun, ST = S::kStages;
    static_assert(S::kTokens == kScanBlock, "a tile starts from a kept state");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ScanShared<S, true, CLUSTER> sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cluster = CLUSTER ? p.cluster : 1;
    const int rank = CLUSTER ? (int)(blockIdx.x % cluster) : 0;
    const int item = CLUSTER ? (int)(blockIdx.x / cluster) : (int)blockIdx.x;
    const int stream = item / p.groups, group = item - stream * p.groups;
    const int base = stream * p.stream, len = min(p.stream, p.total - base);
    const int tiles = (len + p.step - 1) / p.step, slabs = (tiles + cluster - 1) / cluster;
    const int c0 = group * kChannels, c = c0 + 2 * lane;
    const bool live = c < p.D;
    const uint32_t bytes = p.rows * kChannels * (2 * sizeof(T) + sizeof(G));
    auto fetch = [&](int n) {  // by one thread
        const int j = tiles - 1 - (n * cluster + rank), s = n % ST;
        if (j < 0) return;
        uint8_t *const at = smem + s * S::kStage;
        mbar_arrive_expect_tx(&sh.full[s], bytes);
        if (is_lost(p, j)) return;
        load_box(at, &mx, &sh.full[s], c0, base + j * p.step);
        load_box(at + S::kXBytes, &mg, &sh.full[s], c0, base + j * p.step);
        load_box(at + S::kXBytes + S::kGBytes, &md, &sh.full[s], c0, base + j * p.step);
    };
    if (threadIdx.x == 0) {
        sh.abort = 0;
        for (int s = 0; s < ST; ++s) mbar_init(&sh.full[s], 1);
        mbar_init(&sh.sent[0], 1);
        mbar_init(&sh.sent[1], 1);
        fence_mbar_init();
        for (int n = 0; n < ST; ++n) fetch(n);
    }
    const Pair zero = both(0.f), one = both(1.f), minus = both(-1.f);
    Pair carry = zero;  // a G of the token after
    if (!MASKED && p.dh_T && live) carry = load2(p.dh_T + (long long)stream * p.D + c);
    if constexpr (CLUSTER) cluster_sync();
    else __syncthreads();
    // The state that the forward pass kept before a tile.  Always a load, and what it
    // gives taken as it is (where there is no tile, no such channel or a start it goes
    // nowhere): a choice would wait for the load where it stands, a tile ahead of its
    // use (8 x 4096 tokens: 136 us for 110).
    const float *const kept0 = p.states + (MASKED ? 0 : (long long)stream * p.blocks) * p.D + (live ? c : 0);
    auto kept = [&](int j) { return load2(kept0 + (long long)max(j, 0) * p.D); };
    if constexpr (MASKED) pdl_wait();  // for the table
    Pair next = kept(tiles - 1 - rank);
    int entry = run_entry<MASKED, R>(p, base, len, (tiles - 1 - rank) * p.step, warp * R);
    bool gone = false;  // a wait for totals has run out
    for (int n = 0; n < slabs; ++n) {
        const int j = tiles - 1 - (n * cluster + rank), buf = n & 1, s = n % ST;
        const int tile0 = j * p.step, t0 = tile0 + warp * R;
        RunMask m = {0, 0, 0, -1};
        if (j >= 0) m = run_mask<MASKED, R>(entry, len, t0);
        entry = run_entry<MASKED, R>(p, base, len, (unsigned)tile0 - (unsigned)(cluster * p.step), warp * R);
        Pair h = next;
        next = kept(j - cluster);
        if (CLUSTER && threadIdx.x == 0 && !gone) expect_totals(sh.sent, buf, cluster);
        const uint8_t *const stage = smem + s * S::kStage;
        const int at0 = warp * R * kChannels + 2 * lane;
        const T *const xs = reinterpret_cast<const T *>(stage) + at0;
        const G *const gs = reinterpret_cast<const G *>(stage + S::kXBytes) + at0;
        const T *const ds = reinterpret_cast<const T *>(stage + S::kXBytes + S::kGBytes) + at0;
        if (j >= 0) wait_full<false>(&sh.full[s], (n / ST) & 1, &sh.abort, p);
        Pair a[R] = {}, b[R] = {}, u[R] = {};  // u = b x
        Pair H = zero;
        Piece k = {one, zero};
        constexpr unsigned all = (1u << R) - 1u;
        const bool plain = m.act == all && (!MASKED || (m.start | m.end) == 0);
        // h0 of a start, dh_T of an end
        auto start_state = [&](int i) {
            const long long at = (long long)run_seq(m, i) * p.D + c;
            return p.h0 && live ? load2(p.h0 + at) : zero;
        };
        auto end_grad = [&](int i) {
            const long long at = (long long)run_seq(m, i) * p.D + c;
            return p.dh_T && live ? load2(p.dh_T + at) : zero;
        };
        if (plain) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                gates2<T, SIG>(gs + i * kChannels, a[i], b[i]);
                u[i] = load2(xs + i * kChannels);
                if constexpr (SIG) u[i] = mul2(b[i], u[i]);
                k.p = mul2(k.p, a[i]);
                H = fma2(a[i], H, u[i]);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) k.h = fma2(a[i], k.h, mul2(a[i], load2(ds + i * kChannels)));
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const bool in = m.act >> i & 1;
                gates2<T, SIG>(gs + i * kChannels, a[i], b[i]);
                a[i] = either(in, a[i], one);
                u[i] = load2(xs + i * kChannels);
                if constexpr (SIG) u[i] = mul2(b[i], u[i]);
                u[i] = either(in, u[i], zero);
                if (MASKED && (m.start >> i & 1)) H = start_state(i);
                k.p = mul2(k.p, a[i]);
                H = fma2(a[i], H, u[i]);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const bool in = m.act >> i & 1;
                if (MASKED && (m.end >> i & 1)) k.h = end_grad(i);
                k.h = fma2(a[i], k.h, mul2(a[i], either(in, load2(ds + i * kChannels), zero)));
            }
        }
        sh.run[buf][warp][lane] = k;
        sh.state[buf][warp][lane] = H;
        if (MASKED && lane == 0) sh.reset[buf][warp] = (m.start != 0) | (m.end != 0) << 1;
        __syncthreads();
        // every warp is through with the tile before
        if (threadIdx.x == 0 && n > 0 && !sh.abort) fetch(n - 1 + ST);
        Pair v = carry;  // a G of the run's next token
        auto reset = [&](int w, int bit) { return MASKED ? sh.reset[buf][w] & bit : 0; };
        if constexpr (CLUSTER) {
            Piece after = {one, zero}, t;
            int cut = 0, all_cut;
            as_constant(warp, [&](auto number) {
                constexpr int W = decltype(number)::value;
#pragma unroll
                for (int w = kWarps - 1; w > W; --w) {
                    join(after, sh.run[buf][w][lane], reset(w, 2));
                    cut |= reset(w, 2);
                }
                t = after;
                all_cut = cut;
#pragma unroll
                for (int w = W; w >= 0; --w) {
                    join(t, sh.run[buf][w][lane], reset(w, 2));
                    all_cut |= reset(w, 2);
                }
#pragma unroll
                for (int w = 0; w < W; ++w)
                    over(h, {sh.run[buf][w][lane].p, sh.state[buf][w][lane]}, reset(w, 1));
            });
            auto &to = sh.totals[0];
            if (!gone) send_totals(to, sh.sent, buf, rank, cluster, t, all_cut);
            if (!wait_full<true>(&sh.sent[buf], (n >> 1) & 1, &sh.abort, p)) gone = true;
            v = apply_totals<MASKED>(to, buf, rank, cluster, carry);
            over(v, after, cut);
        } else {
            as_constant(warp, [&](auto number) {
                constexpr int W = decltype(number)::value;
#pragma unroll
                for (int w = 0; w < W; ++w)
                    over(h, {sh.run[buf][w][lane].p, sh.state[buf][w][lane]}, reset(w, 1));
#pragma unroll
                for (int w = kWarps - 1; w > W; --w) over(v, sh.run[buf][w][lane], reset(w, 2));
                carry = v;
#pragma unroll
                for (int w = W; w >= 0; --w) over(carry, sh.run[buf][w][lane], reset(w, 2));
            });
        }
        if (m.act) {
            T *const dx = static_cast<T *>(p.dx) + ((long long)(base + t0) * p.D + c);
            G *const dg = static_cast<G *>(p.dgate) + ((long long)(base + t0) * p.D + c);
            Pair past[R] = {};
            // the gradients of token i: v becomes a G, dgate = a G (b h_{t-1} - b x)
            auto token = [&](int i, Pair d, bool out) {
                const Pair g = add2(d, v);
                v = mul2(a[i], g);
                if (!out) return;
                if constexpr (SIG) {
                    store2(dx + (long long)i * p.D, mul2(b[i], g));
                    store2(dg + (long long)i * p.D, mul2(v, fma2(u[i], minus, mul2(b[i], past[i]))));
                } else {
                    store2(dx + (long long)i * p.D, g);
                    store2(dg + (long long)i * p.D, mul2(g, past[i]));
                }
            };
            if (plain) {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    past[i] = h;
                    h = fma2(a[i], h, u[i]);
                }
#pragma unroll
                for (int i = R - 1; i >= 0; --i) token(i, load2(ds + i * kChannels), live);
            } else {
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (MASKED && (m.start >> i & 1)) h = start_state(i);
                    past[i] = h;
                    h = fma2(a[i], h, u[i]);
                }
#pragma unroll
                for (int i = R - 1; i >= 0; --i) {
                    const bool in = m.act >> i & 1;
                    if (MASKED && (m.end >> i & 1)) v = end_grad(i);
                    token(i, either(in, load2(ds + i * kChannels), zero), in && live);
                    if (MASKED && p.dh0 && (m.start >> i & 1)) {
                        const long long at = (long long)run_seq(m, i) * p.D + c;
                        if (live) store2(p.dh0 + at, v);
                    }
                }
            }
        }
    }
    if (!MASKED && p.dh0 && rank == 0 && warp == 0 && live)
        store2(p.dh0 + (long long)stream * p.D + c, carry);
    if (sh.abort && threadIdx.x == 0) {
        drain(sh.full, ST);
        if constexpr (CLUSTER) drain(sh.sent, 2);
    }
    if constexpr (CLUSTER) cluster_sync();  // no CTA sends to one that has ended
}

// ------------------------------------------------------------------ packed tokens

// The sequence of each token, or -1, 1024 tokens a CTA; and the end states of
// sequences without tokens (end = start or 0), shared out among the CTAs.  A
// sequence whose offsets fall, pass T or start before the end of an earlier one
// (of those that neither fall nor pass T) has none and sets the bounds bit.
constexpr int kMapThreads = 1024;
__global__ void __launch_bounds__(kMapThreads)
    scan_map_kernel(const int *offsets, int B, int T, int *map, const float *start, float *end, int D,
                    int *status) {
    __shared__ int mark[kMapThreads], far[32], empty[kMapThreads], empties;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long w0 = (long long)blockIdx.x * kMapThreads;
    pdl_trigger();  // the scan waits for this kernel's end before it reads the table
    mark[tid] = -1;
    int upto = 0;  // the furthest end so far
    for (int s0 = 0; s0 < B; s0 += kMapThreads) {
        const int s = s0 + tid;
        int a = 0, b = 0;
        bool good = false;
        if (s < B) {
            a = offsets[s];
            b = offsets[s + 1];
            good = a >= 0 && b >= a && b <= T;
        }
        int most = good ? b : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, most, off);
            if (lane >= off) most = max(most, y);
        }
        if (lane == 31) far[warp] = most;
        if (tid == 0) empties = 0;
        __syncthreads();
        int before = upto;  // the furthest end before this sequence
        for (int w = 0; w < warp; ++w) before = max(before, far[w]);
        const int prev = __shfl_up_sync(0xffffffffu, most, 1);
        if (lane) before = max(before, prev);
        for (int w = 0; w < 32; ++w) upto = max(upto, far[w]);
        if (s < B) {
            good = good && a >= before;
            if (!good && blockIdx.x == 0 && status) atomicOr(status, kStatusBounds);
            if (good && b > a) {
                if (b > w0 && a < w0 + kMapThreads) mark[a > w0 ? a - w0 : 0] = s;
            } else if (end && s % gridDim.x == blockIdx.x) {
                empty[atomicAdd(&empties, 1)] = s;
            }
        }
        __syncthreads();
        for (int i = 0; i < empties; ++i) {
            const long long at = (long long)empty[i] * D;
            for (int c = tid; c < D; c += kMapThreads) end[at + c] = start ? start[at + c] : 0.f;
        }
        __syncthreads();
    }
    __syncthreads();
    // the last sequence that starts at or before each token
    int q = mark[tid];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, q, off);
        if (lane >= off) q = max(q, y);
    }
    if (lane == 31) far[warp] = q;
    __syncthreads();
    for (int w = 0; w < warp; ++w) q = max(q, far[w]);
    const long long t = w0 + tid;
    if (t < T) map[t] = q >= 0 && t < offsets[q + 1] ? q : -1;
}

// ------------------------------------------------------------------ one token

// A thread takes eight channels, all of its loads before any arithmetic.
constexpr int kStepThreads = 128;
template <typename T, bool SIG>
__global__ void __launch_bounds__(kStepThreads)
    scan_step_kernel(const T *x, const typename GateType<T, SIG>::type *gate, const float *h,
                     float *h_out, T *y, long long pieces, int per, long long ldx, long long ldg) {
    using G = typename GateType<T, SIG>::type;
    const long long i = (long long)blockIdx.x * kStepThreads + threadIdx.x;
    // the previous step's states are complete before the first read
    pdl_wait();
    if (i >= pieces) return;
    const long long row = pieces >> 31 ? i / per : (long long)((unsigned)i / (unsigned)per);
    const int c = (int)(i - row * per) * 8;
    Vec8<T> xv;
    Vec8<G> gv;
    Pair xs[4], s[4], a[4], b[4];
    xv.load(x + row * ldx + c);
    gv.load(gate + row * ldg + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = load2(h + i * 8 + 2 * e);
    pdl_trigger();
    get4(xv, xs);
    if constexpr (SIG && sizeof(T) == 2) {
        gate_ab2(gv.a.x, a[0], b[0]);
        gate_ab2(gv.a.y, a[1], b[1]);
        gate_ab2(gv.a.z, a[2], b[2]);
        gate_ab2(gv.a.w, a[3], b[3]);
    } else {
        get4(gv, a);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 g = split(a[e]);
            float2 u, v;
            gate_ab<SIG>(g.x, u.x, v.x);
            gate_ab<SIG>(g.y, u.y, v.y);
            a[e] = pair(u.x, u.y);
            b[e] = pair(v.x, v.y);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = fma2(a[e], s[e], SIG ? mul2(b[e], xs[e]) : xs[e]);
    Vec8<float> hv;
    set4(hv, s);
    put8(h_out + i * 8, hv);
    if (y) {
        Vec8<T> yv;
        set4(yv, s);
        put8(y + i * 8, yv);
    }
}

// ------------------------------------------------------------------ host

// [tokens, D] with the token stride ld, in boxes of 64 channels x rows tokens.
template <typename E> bool box_map(CUtensorMap *m, const void *p, long long tokens, int D, long long ld, int rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)tokens};
    cuuint64_t strides[1] = {(cuuint64_t)ld * sizeof(E)};
    cuuint32_t box[2] = {kChannels, (cuuint32_t)rows}, es[2] = {1, 1};
    return enc(m, sizeof(E) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
               const_cast<void *>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the tokens lie in streams, tiles and clusters.
struct ScanPlan {
    bool masked;
    int streams, cluster;
    ScanRun run;
};
ScanPlan scan_plan(const ScanArgs &a, int tile, int most, const int *map) {
    ScanPlan s = {};
    ScanRun &r = s.run;
    const int nsm = sm_count() > 0 ? sm_count() : 152;
    r.h0 = a.h0; r.dh_T = a.dh_T; r.states = a.states; r.h = a.h; r.h_T = a.h_T;
    r.dx = a.dx; r.dgate = a.dgate; r.dh0 = a.dh0;
    r.map = map;
    r.D = a.D;
    r.groups = (a.D + kChannels - 1) / kChannels;
    r.T = a.T;
    r.blocks = (a.T + kScanBlock - 1) / kScanBlock;
    r.total = a.offsets ? a.T : a.B * a.T;
    r.status = device_status_ptr();
    r.step = tile;
    if (a.offsets) {
        s.masked = true;
        s.streams = 1;
        r.stream = a.T;
    } else if (a.T <= kScanBlock && a.B > 1) {
        // whole sequences in a tile, and tiles of as many streams as the SMs take at once
        s.masked = true;
        const int per = tile / a.T, tiles = (a.B + per - 1) / per;
        r.step = per * a.T;
        long long streams = (2LL * nsm + r.groups - 1) / r.groups;
        if (streams > tiles) streams = tiles;
        const int each = (int)((tiles + streams - 1) / streams);
        s.streams = (tiles + each - 1) / each;
        r.stream = each * r.step;
        // such tiles have nothing to tell each other, so no clusters (with two tiles a stream
        // clusters of two put them side by side, and cost their start and end and the totals:
        // 11 sequences of 64 float32 tokens and 2048 channels 13.8 us, one CTA for both 8.8)
        most = 1;
    } else {
        s.streams = a.B;
        r.stream = a.T;
    }
    r.rows = r.step < r.stream ? r.step : r.stream;
    const int tiles = (r.stream + r.step - 1) / r.step;
    s.cluster = 1;
    while (s.cluster < most && 2 * s.cluster <= tiles &&
           2LL * r.groups * s.streams * s.cluster < 3LL * nsm)
        s.cluster *= 2;
    r.cluster = s.cluster;
    return s;
}

template <typename K, typename... A>
cudaError_t launch_clustered(K kern, uintptr_t (&set)[64], const ScanPlan &s, size_t smem,
                             bool after_map, cudaStream_t st, const A &...args) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set[dev] != context_key()) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        set[dev] = context_key();
    }
    const long long grid = (long long)s.run.groups * s.streams * s.cluster;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (s.cluster > 1) {
        cudaLaunchAttribute &x = attr[cfg.numAttrs++];
        x.id = cudaLaunchAttributeClusterDimension;
        x.val.clusterDim.x = s.cluster;
        x.val.clusterDim.y = x.val.clusterDim.z = 1;
    }
    if (after_map) {  // its first loads do not wait for the table
        cudaLaunchAttribute &x = attr[cfg.numAttrs++];
        x.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        x.val.programmaticStreamSerializationAllowed = 1;
    }
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, bool SIG, bool MASKED, bool CLUSTER, typename RUN>
cudaError_t forward(const ScanArgs &a, const ScanPlan &s, const RUN &run, bool after_map, cudaStream_t st) {
    using S = Shape<T, SIG, false>;
    static uintptr_t set[64] = {};
    CUtensorMap mx, mg;
    if (!box_map<T>(&mx, a.x, s.run.total, a.D, a.ldx, s.run.rows) ||
        !box_map<typename S::G>(&mg, a.gate, s.run.total, a.D, a.ldg, s.run.rows))
        return cudaErrorInvalidValue;
    return launch_clustered(scan_kernel<T, SIG, MASKED, CLUSTER, RUN>, set, s, S::kStages * S::kStage,
                            after_map, st, mx, mg, run);
}
template <typename T, bool SIG, bool MASKED, bool CLUSTER, typename RUN>
cudaError_t backward(const ScanArgs &a, const ScanPlan &s, const RUN &run, bool after_map, cudaStream_t st) {
    using S = Shape<T, SIG, true>;
    static uintptr_t set[64] = {};
    CUtensorMap mx, mg, md;
    if (!box_map<T>(&mx, a.x, s.run.total, a.D, a.ldx, s.run.rows) ||
        !box_map<typename S::G>(&mg, a.gate, s.run.total, a.D, a.ldg, s.run.rows) ||
        !box_map<T>(&md, a.dh, s.run.total, a.D, a.D, s.run.rows))
        return cudaErrorInvalidValue;
    return launch_clustered(scan_backward_kernel<T, SIG, MASKED, CLUSTER, RUN>, set, s, S::kStages * S::kStage,
                            after_map, st, mx, mg, md, run);
}

template <typename T, bool SIG, bool BACK, bool MASKED, bool CLUSTER, typename RUN>
cudaError_t launch_one(const ScanArgs &a, const ScanPlan &s, const RUN &run, bool after_map, cudaStream_t st) {
    if constexpr (BACK) return backward<T, SIG, MASKED, CLUSTER>(a, s, run, after_map, st);
    else return forward<T, SIG, MASKED, CLUSTER>(a, s, run, after_map, st);
}
template <typename T, bool SIG, bool BACK>
cudaError_t launch_any(const ScanArgs &a, const int *map, bool after_map, cudaStream_t st) {
    const ScanPlan s = scan_plan(a, Shape<T, SIG, BACK>::kTokens, Shape<T, SIG, BACK>::kCluster, map);
    if (s.masked)
        return s.cluster > 1 ? launch_one<T, SIG, BACK, true, true>(a, s, s.run, after_map, st)
                             : launch_one<T, SIG, BACK, true, false>(a, s, s.run, after_map, st);
    return s.cluster > 1 ? launch_one<T, SIG, BACK, false, true>(a, s, s.run, after_map, st)
                         : launch_one<T, SIG, BACK, false, false>(a, s, s.run, after_map, st);
}
template <bool BACK> cudaError_t launch_lost(const ScanArgs &a, long long limit, int lost, cudaStream_t st) {
    using T = __nv_bfloat16;
    const ScanPlan s = scan_plan(a, Shape<T, true, BACK>::kTokens, Shape<T, true, BACK>::kCluster, nullptr);
    LostRun run;
    static_cast<ScanRun &>(run) = s.run;
    run.limit = limit;
    run.lost = lost;
    if (s.masked) return launch_one<T, true, BACK, true, false>(a, s, run, false, st);
    return s.cluster > 1 ? launch_one<T, true, BACK, false, true>(a, s, run, false, st)
                         : launch_one<T, true, BACK, false, false>(a, s, run, false, st);
}
// after_map: the launch comes directly after the table's.
template <bool BACK>
cudaError_t launch_type(const ScanArgs &a, gdn_dtype dt, const int *map, bool after_map, cudaStream_t st) {
    if (dt == GDN_BF16)
        return a.sigmoid ? launch_any<__nv_bfloat16, true, BACK>(a, map, after_map, st)
                         : launch_any<__nv_bfloat16, false, BACK>(a, map, after_map, st);
    return a.sigmoid ? launch_any<float, true, BACK>(a, map, after_map, st)
                     : launch_any<float, false, BACK>(a, map, after_map, st);
}

// The table of packed tokens, and what sequences without tokens end with.
cudaError_t launch_map(const ScanArgs &a, int *map, const float *start, float *end, cudaStream_t st) {
    scan_map_kernel<<<(unsigned)((a.T + (long long)kMapThreads - 1) / kMapThreads), kMapThreads, 0, st>>>(
        a.offsets, a.B, a.T, map, start, end, a.D, device_status_ptr());
    return cudaGetLastError();
}

template <typename T, bool SIG>
cudaError_t step(const void *x, const void *gate, const float *h, float *h_out, void *y, int B, int D,
                 long long ldx, long long ldg, cudaStream_t st) {
    using G = typename GateType<T, SIG>::type;
    const long long pieces = (long long)B * (D / 8), grid = (pieces + kStepThreads - 1) / kStepThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return launch_pdl(scan_step_kernel<T, SIG>, (unsigned)grid, kStepThreads, 0, st,
                      static_cast<const T *>(x), static_cast<const G *>(gate), h, h_out,
                      static_cast<T *>(y), pieces, D / 8, ldx, ldg);
}

}  // namespace

size_t scan_map_bytes(int T) { return ((size_t)T * sizeof(int) + 255) & ~size_t(255); }

cudaError_t launch_scan(const ScanArgs &a, gdn_dtype dt, void *workspace, cudaStream_t st) {
    int *const map = a.offsets ? static_cast<int *>(workspace) : nullptr;
    if (map) {
        const cudaError_t e = launch_map(a, map, a.h0, a.h_T, st);
        if (e != cudaSuccess) return e;
    }
    return launch_type<false>(a, dt, map, map != nullptr, st);
}

cudaError_t launch_scan_backward(const ScanArgs &a, gdn_dtype dt, void *workspace, cudaStream_t st) {
    int *const map = a.offsets ? static_cast<int *>(workspace) : nullptr;
    if (map) {
        const cudaError_t e = launch_map(a, map, a.dh_T, a.dh0, st);
        if (e != cudaSuccess) return e;
    }
    ScanArgs b = a;
    if (!b.states) {  // a forward pass that only keeps them
        ScanArgs f = a;
        f.states = b.states = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                                        (map ? scan_map_bytes(a.T) : 0));
        const cudaError_t e = launch_type<false>(f, dt, map, map != nullptr, st);
        if (e != cudaSuccess) return e;
    }
    return launch_type<true>(b, dt, map, map && a.states, st);
}

cudaError_t launch_scan_lost(const ScanArgs &a, long long limit, int lost, cudaStream_t st) {
    return a.dh ? launch_lost<true>(a, limit, lost, st) : launch_lost<false>(a, limit, lost, st);
}

cudaError_t launch_scan_step(const void *x, const void *gate, const float *h, float *h_out, void *y,
                             int B, int D, long long ldx, long long ldg, bool sigmoid, gdn_dtype dt,
                             cudaStream_t st) {
    if (dt == GDN_BF16)
        return sigmoid ? step<__nv_bfloat16, true>(x, gate, h, h_out, y, B, D, ldx, ldg, st)
                       : step<__nv_bfloat16, false>(x, gate, h, h_out, y, B, D, ldx, ldg, st);
    return sigmoid ? step<float, true>(x, gate, h, h_out, y, B, D, ldx, ldg, st)
                   : step<float, false>(x, gate, h, h_out, y, B, D, ldx, ldg, st);
}

}  // namespace gdn
