// Layer norm of rows with the sum that runs past a layer, and its gradients:
//
//     s = x + residual,  y = (s - m) r .* w + b
//     n = (s - m) r,  g = w .* dy
//     dx = r (g - mean g - n mean(g n)) + ds,  dw = sum dy .* n,  db = sum dy
//
// Bound by memory: every input read once, every output written once (8 bytes a
// value with the sum, 4 without; gradients 8 or 6, in bf16).  A team (a warp, or
// the threads of one wide row) has a ring of one to four blocks of rows in shared memory,
// which one thread fills by bulk copies: what is in flight does not depend on
// registers.  (Rows fetched ahead into registers spilled: 124 us for 32768 rows of
// 2048 bf16 channels with the sum.)  With one block only, outputs fetch the next as soon as
// it is in registers; gradients read it twice and fetch after that, so that a team's loads
// do not overlap its own arithmetic, only the other teams'.  The deviation is taken from the mean, not from
// the squares' sum: a row about a large mean keeps it.
#include <type_traits>

#include "gdn_pair.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr long long kWaitLimit = 2000000000LL;  // about 1 s of SM clocks
constexpr long long kDrainLimit = kWaitLimit / 16;
constexpr long long kLostAnswer = -2;

// Threads of a row and pieces of 8 channels of a thread.  A team is a warp, of one
// row or several, or the threads of a row; ALONE: one row at a time.
template <int TPR_, int VPT_, bool ALONE_ = false> struct RowShape {
    enum {
        TPR = TPR_,
        VPT = VPT_,
        ALONE = ALONE_,
        kTeam = TPR < 32 ? 32 : TPR,
        kAbreast = kTeam / TPR,  // rows side by side in a team
        // Outputs: one CTA an SM, of up to 20 warps, fewer where the rows are few (24
        // warps spilled; two CTAs of 8 would each hold the weights).  Of 20 warps float32
        // rows with the sum of up to 128 channels spill 20 bytes a thread, of 16 warps
        // float32 rows above 8192 channels 20, with the sum 28.  Gradients: 16
        // warps an SM (24 spilled: 94 -> 116 us for 512 channels).
        kTeams = kTeam < 640 ? 640 / kTeam : 1,
        kThreads = kTeams * kTeam,
        kBackThreads = kTeam < 256 ? 256 : kTeam,
        kBackTeams = kBackThreads / kTeam,
        kBackCtas = 512 / kBackThreads
    };
};
// Rows of a thread at once: their chains of sums overlap, and one meeting of a
// team's warps serves them all.  (Gradients of 5120 bf16 channels: two rows 88 us, one
// 119.)
template <typename T, typename S> constexpr int rows_at_once(bool back) {
    if (S::ALONE) return 1;
    const int pieces = back && S::TPR > 32 && sizeof(T) == 2 || !back ? 4 : 2;
    return S::VPT < pieces ? pieces / S::VPT : 1;
}
constexpr int kMaxSlots = 4;  // blocks of a team in shared memory (gradients), at most

// Sums of U values over the threads of a row, the same in all of them and in a
// fixed order.  Rows of several warps meet at a barrier of their team's; the two
// buffers of `red` take turns.
template <int TPR, int U> struct RowSum {
    static constexpr int kWarps = TPR / 32;
    float (*red)[(kWarps > 0 ? kWarps : 1) * U];  // [2][warps x U], the team's
    int team, turn;
    // Half of the values for the lanes with the bit `off`, half for those without:
    // each lane adds what its partner has of its half.
    template <int N>
    static __device__ __forceinline__ void share(float (&x)[N], int off) {
        const bool high = threadIdx.x & off;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float mine = high ? x[i + N / 2] : x[i], its = high ? x[i] : x[i + N / 2];
            x[i] = mine + __shfl_xor_sync(0xffffffffu, its, off);
        }
    }
    // The sum of value lane / (32 / U) over a warp (of four values in 6 exchanges, one
    // by one 20).
    static __device__ __forceinline__ float shared_out(const float (&x)[U]) {
        static_assert(U == 1 || U == 2 || U == 4 || U == 8, "a power of two of values");
        float y[8] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) y[u] = x[u];
        int off = 16;
        if constexpr (U == 8) {
            share<8>(y, off);
            off >>= 1;
        }
        if constexpr (U >= 4) {
            share<4>(reinterpret_cast<float (&)[4]>(y), off);
            off >>= 1;
        }
        if constexpr (U >= 2) {
            share<2>(reinterpret_cast<float (&)[2]>(y), off);
            off >>= 1;
        }
        float r = y[0];
#pragma unroll
        for (int o = 16 / U; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
        return r;
    }
    __device__ __forceinline__ void operator()(float (&x)[U]) {
        if constexpr (TPR < 32) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int off = TPR / 2; off > 0; off >>= 1) x[u] += __shfl_xor_sync(0xffffffffu, x[u], off);
        } else {
            const float r = shared_out(x);
            const int lane = threadIdx.x & 31;
            if constexpr (TPR == 32) {
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = __shfl_sync(0xffffffffu, r, u * (32 / U));
            } else {
                const int warp = (threadIdx.x % TPR) >> 5;
                if (lane % (32 / U) == 0) red[turn][warp * U + lane / (32 / U)] = r;
                sm100::named_sync(team + 1, TPR);
                // lanes add the warps' sums of value lane % U, and hand them round
                constexpr int ALL = kWarps * U;
                float z = red[turn][lane % ALL];
#pragma unroll
                for (int i = 32; i < ALL; i += 32) z += red[turn][i + lane];
#pragma unroll
                for (int o = U; o < (ALL < 32 ? ALL : 32); o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = __shfl_sync(0xffffffffu, z, u);
                turn ^= 1;
            }
        }
    }
};

struct NormArgs {
    const void *x, *res;  // backward: s and ds
    const void *dy;
    const float *w, *b;
    void *y, *s;          // backward: dx
    float *stats, *parts;
    long long N;
    int D;
    long long ldx, ldr;
    float eps;
    int rows, slots;      // of a block; blocks of a team
    bool more;            // outputs: CTAs take over others
    int *status;
};
// Self-test (kernels of their own): the clocks of a wait; the row whose block is not copied,
// or kLostAnswer: CTAs to take over are not asked for.
struct LostArgs : NormArgs {
    long long limit, lost;
};
__device__ __forceinline__ long long wait_limit(const NormArgs &) { return kWaitLimit; }
__device__ __forceinline__ long long wait_limit(const LostArgs &p) { return p.limit; }
__device__ __forceinline__ bool is_lost(const NormArgs &, long long, int) { return false; }
__device__ __forceinline__ bool is_lost(const LostArgs &p, long long row0, int n) {
    return p.lost >= row0 && p.lost < row0 + n;
}
__device__ __forceinline__ bool unasked(const NormArgs &) { return false; }
__device__ __forceinline__ bool unasked(const LostArgs &p) { return p.lost == kLostAnswer; }

// A team's ring: block i of the team's is in slot i % slots, its tensors one after
// another, the rows dense.
template <typename T, int TENSORS> struct Ring {
    uint8_t *base;
    uint64_t *full;
    const T *src[TENSORS];
    long long ld[TENSORS];
    int bytes;  // of a slot's tensor
    // by one thread
    template <typename A> __device__ __forceinline__ void fetch(const A &p, int slot, long long row0) const {
        if (row0 >= p.N) return;
        const int n = (int)min((long long)p.rows, p.N - row0), row = p.D * (int)sizeof(T);
        uint8_t *const at = base + slot * TENSORS * bytes;
        sm100::mbar_arrive_expect_tx(&full[slot], TENSORS * n * row);
        if (is_lost(p, row0, n)) return;
#pragma unroll
        for (int t = 0; t < TENSORS; ++t) {
            const T *const from = src[t] + row0 * ld[t];
            if (ld[t] == p.D) {
                sm100::bulk_load(at + t * bytes, from, n * row, &full[slot]);
            } else {
                for (int i = 0; i < n; ++i)
                    sm100::bulk_load(at + t * bytes + i * row, from + i * ld[t], row, &full[slot]);
            }
        }
    }
    __device__ __forceinline__ const T *row(const NormArgs &p, int slot, int tensor, int i) const {
        return reinterpret_cast<const T *>(base + (slot * TENSORS + tensor) * bytes) + (long long)i * p.D;
    }
};
// Waits with a limit; after one that ran out nothing more is fetched, and no barrier whose
// phase is open is arrived at again.  The threads of a team go on alike all the same, with
// what the slot holds, so that none is left behind at a barrier of theirs.
__device__ __forceinline__ void gave_up(int *abort, int *status) {
    *static_cast<volatile int *>(abort) = 1;
    if (status) atomicOr(status, kStatusTimeout);
}
// Where the blocks are dealt out: the first wait that runs out ends all others of the CTA.
template <typename A>
__device__ __forceinline__ void wait_dealt(uint64_t *bar, uint32_t parity, int *abort, const A &p) {
    volatile int *const flag = abort;
    if (!sm100::mbar_wait_or_abort(bar, parity, wait_limit(p), flag) && !*flag) gave_up(abort, p.status);
}
// Where they are drawn: the team's first thread says which block it is before the barrier
// completes, or that there is none, once its own waits (two of the limit) have run out.
template <typename A>
__device__ __forceinline__ bool wait_drawn(uint64_t *bar, uint32_t parity, int *abort, const A &p) {
    const bool ok = sm100::mbar_wait(bar, parity, 4 * wait_limit(p));
    if (!ok) gave_up(abort, p.status);
    return ok;
}
// Copies in flight land before the CTA ends (where nothing went wrong none are).
__device__ __forceinline__ void drain(uint64_t *full, int slots) {
    for (int i = 0; i < slots; ++i) {
        sm100::mbar_wait(&full[i], 0, kDrainLimit);
        sm100::mbar_wait(&full[i], 1, kDrainLimit);
    }
}
// Outputs: the chunks of a CTA, one block a team each, which the teams draw one by one.
// With the sum to form the grid has as many CTAs as there are chunks; one that runs
// takes over others that have not started, so that an SM with more of the memory's
// bandwidth gets more of them: dealt out evenly the last SM ended 13 % after the mean
// (32768 rows of 2048 bf16 channels 92 us, taken over 85).  Without the sum half as much
// moves, and the questions cost what they bring (512 channels: dealt out 46 us, taken
// over 48; 2048: 47 and 46).  Who draws a chunk's first block asks for the next chunk.
constexpr int kOutSlots = 2;   // blocks of a team, at most
constexpr int kAsked = 4;  // chunks asked for and not yet handed out
struct Chunks {
    alignas(16) unsigned long long answer[kAsked][2];
    uint64_t ready[kAsked];
    int taken[kAsked];  // how often the answer has been read
    int drawn;          // blocks drawn from the chunk that the CTA started with on
};
// One thread; chunk k >= 1.  (A question that is on its way when another thread gives up is
// answered long before the CTA's copies and answers have been waited for.)
template <typename A>
__device__ __forceinline__ void ask(Chunks &q, int k, int teams, int *abort, const A &p) {
    const int e = (k - 1) % kAsked, before = (k - 1) / kAsked * teams;
    volatile int *const taken = &q.taken[e], *const flag = abort;
    const long long t0 = clock64();
    while (*taken != before) {  // the entry's last answer has been read by all
        if (*flag) return;
        if (clock64() - t0 > wait_limit(p)) return gave_up(abort, p.status);
    }
    if (*flag) return;
    sm100::fence_proxy_async_smem();
    sm100::mbar_arrive_expect_tx(&q.ready[e], 16);
    if (unasked(p)) return;
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            sm100::smem_u32(q.answer[e])),
        "r"(sm100::smem_u32(&q.ready[e]))
        : "memory");
}
// A team's next block, or one past the rows where there is none (by one thread of the
// team, which draws no more then: all teams have read the last answer before the CTA
// ends).  Without taking over, a CTA's chunks lie a grid apart.
template <typename A>
__device__ __forceinline__ long long draw(Chunks &q, int teams, int *abort, const A &p) {
    volatile int *const flag = abort;
    if (*flag) return -1;
    const int n = atomicAdd(&q.drawn, 1), k = n / teams;
    if (!p.more) return ((long long)k * gridDim.x + blockIdx.x) * teams + n % teams;
    const int e = (k - 1) % kAsked;
    if (!sm100::mbar_wait_or_abort(&q.ready[e], ((k - 1) / kAsked) & 1, wait_limit(p), flag)) {
        gave_up(abort, p.status);
        return -1;
    }
    uint32_t ok, chunk;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t"
        "ld.shared.v2.b64 {lo, hi}, [%2];\n\tmov.b128 r, {lo, hi};\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(ok), "=r"(chunk)
        : "r"(sm100::smem_u32(q.answer[e]))
        : "memory");
    __threadfence_block();
    atomicAdd(&q.taken[e], 1);
    if (!ok) return -1;
    // (after an answer that there is none no other may be asked for)
    if (n % teams == 0) ask(q, k + 1, teams, abort, p);
    return (long long)chunk * teams + n % teams;
}

// From here on the values are unpacked again: kept as floats from one phase to the
// next, they took twice the registers and spilled.
__device__ __forceinline__ void repack(Vec8<float> &) {}
__device__ __forceinline__ void repack(Vec8<__nv_bfloat16> &v) {
    asm volatile("" : "+r"(v.a.x), "+r"(v.a.y), "+r"(v.a.z), "+r"(v.a.w));
}

// A thread's channels of a weight: eight from `p` (or `other` where there is none).
__device__ __forceinline__ void column(Pair (&v)[4], const float *p, float other, int c, int D) {
    if (p && c < D) {
        Vec8<float> q;
        q.load_cached(p + c);
        get4(q, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = both(other);
    }
}
// Where w and b of a piece come from: a thread's registers, where it has one piece, or
// where the row has all threads of an SM; shared memory, staged once by the CTA, up to
// 8192 channels; else (gradients) the L1 cache.
enum { kRegisters, kStaged, kCached };
template <typename S> constexpr int weights_in(bool back) {
    if (back) return S::VPT <= 2 ? kRegisters : kCached;
    return S::VPT == 1 || S::TPR * S::VPT * 8 > 8192 ? kRegisters : kStaged;
}
// Staged: the lower and the upper four channels of every piece apart, so that
// neighbouring lanes read neighbouring 16 bytes.
template <int PIECES>
__device__ __forceinline__ void stage_column(float4 *dst, const float *p, float other, int D) {
    for (int i = threadIdx.x; i < PIECES; i += blockDim.x) {
        float4 lo = make_float4(other, other, other, other), hi = lo;
        if (p && 8 * i < D) {
            lo = reinterpret_cast<const float4 *>(p)[2 * i];
            hi = reinterpret_cast<const float4 *>(p)[2 * i + 1];
        }
        dst[i] = lo;
        dst[PIECES + i] = hi;
    }
}
template <int PIECES> __device__ __forceinline__ void staged(Pair (&v)[4], const float4 *src, int i) {
    const float4 lo = src[i], hi = src[PIECES + i];
    v[0] = pair(lo.x, lo.y);
    v[1] = pair(lo.z, lo.w);
    v[2] = pair(hi.x, hi.y);
    v[3] = pair(hi.z, hi.w);
}
__device__ __forceinline__ float sum2(Pair x) {
    const float2 f = split(x);
    return f.x + f.y;
}

template <typename T, typename S, bool RES, typename A>
__global__ void __launch_bounds__(S::kThreads, 1)
    layer_norm_kernel(const A p) {
    constexpr int TPR = S::TPR, VPT = S::VPT, U = rows_at_once<T, S>(false);
    constexpr int TENSORS = RES ? 2 : 1, BATCH = U * S::kAbreast;
    constexpr int kWeights = weights_in<S>(false), PIECES = TPR * VPT;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[S::kTeams][2][(TPR >= 32 ? TPR / 32 : 1) * U];
    __shared__ uint64_t full[S::kTeams][kOutSlots];
    __shared__ long long row_of[S::kTeams][kOutSlots];
    __shared__ Chunks chunks;
    __shared__ int abort;
    const int team = threadIdx.x / S::kTeam, lead = threadIdx.x % S::kTeam == 0;
    const int l = threadIdx.x % TPR, c0 = l * 8, abreast = threadIdx.x % S::kTeam / TPR;
    Ring<T, TENSORS> ring;
    ring.bytes = p.rows * p.D * (int)sizeof(T);
    float4 *const weights = reinterpret_cast<float4 *>(smem);
    ring.base = smem + (kWeights == kStaged ? 64 * PIECES : 0) + (size_t)team * p.slots * TENSORS * ring.bytes;
    ring.full = full[team];
    ring.src[0] = static_cast<const T *>(p.x);
    ring.ld[0] = p.ldx;
    if constexpr (RES) {
        ring.src[1] = static_cast<const T *>(p.res);
        ring.ld[1] = p.ldr;
    }
    const int teams = blockDim.x / S::kTeam;
    // The team's next block: its rows on the way, or word that it has none (of the last
    // chunk) or that there is none.  open: the slot's last copies have not come.  Then nothing
    // is drawn any more, and the phase is not arrived at: who waits for the next one goes on at
    // once, or when its wait runs out, and finds the word, which the team's meeting for the
    // block's second sum has shown to all.
    constexpr long long kEnd = -1, kEmpty = -2;
    bool ended = false;
    auto fetch = [&](int slot, long long block, bool open) {
        const long long row0 = block < 0 ? kEnd : block * p.rows < p.N ? block * p.rows : p.more ? kEmpty : kEnd;
        row_of[team][slot] = row0;
        ended = row0 == kEnd;
        if (row0 >= 0) ring.fetch(p, slot, row0);
        else if (!open) sm100::mbar_arrive(&full[team][slot]);
    };
    auto next = [&](int slot, bool ok) {
        fetch(slot, ended ? -1 : draw(chunks, teams, &abort, p), !ok);
    };
    if (threadIdx.x == 0) {
        abort = 0;
        chunks.drawn = teams;
        for (int e = 0; e < kAsked; ++e) {
            chunks.taken[e] = 0;
            sm100::mbar_init(&chunks.ready[e], 1);
        }
    }
    if (lead) {
        for (int i = 0; i < p.slots; ++i) sm100::mbar_init(&full[team][i], 1);
        sm100::fence_mbar_init();
        fetch(0, (long long)blockIdx.x * teams + team, false);
    }
    RowSum<TPR, U> sum = {red[team], team, 0};
    const float inv = 1.f / p.D;
    constexpr bool kHold = kWeights == kRegisters;
    Pair w[kHold ? VPT : 1][4], b[kHold ? VPT : 1][4];
    if constexpr (kHold) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            column(w[k], p.w, 1.f, c0 + k * TPR * 8, p.D);
            column(b[k], p.b, 0.f, c0 + k * TPR * 8, p.D);
        }
    } else {
        stage_column<PIECES>(weights, p.w, 1.f, p.D);
        stage_column<PIECES>(weights + 2 * PIECES, p.b, 0.f, p.D);
    }
    T *const y = static_cast<T *>(p.y), *const sums = static_cast<T *>(p.s);
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    for (bool begin = true;; begin = false) {
        const bool ok = wait_drawn(&full[team][slot], parity, &abort, p);
        const long long block = row_of[team][slot];
        if (block == kEnd) break;
        if (begin) {
            // (the first block of the first team has rows; the CTAs of the first round have
            // started by the time that these are here)
            if (threadIdx.x == 0 && p.more) ask(chunks, 1, teams, &abort, p);
            if (lead)
                for (int i = 1; i < p.slots; ++i) next(i, true);
        }
        const int at = slot;
        if (++slot == p.slots) {
            slot = 0;
            parity ^= 1;
        }
        if (block == kEmpty) {
            if constexpr (TPR <= 32) __syncwarp();
            else sm100::named_sync(team + 1, TPR);
            if (lead) next(at, ok);
            continue;
        }
        const int n = (int)min((long long)p.rows, p.N - block);
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            Vec8<T> sv[U][VPT];
            float m[U], q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * S::kAbreast + abreast;
                Pair t = both(0.f);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = c0 + k * TPR * 8;
                    sv[u][k] = {};
                    if (i < n && c < p.D) {
                        from_shared(sv[u][k], ring.row(p, at, 0, i) + c);
                        Pair f[4];
                        get4(sv[u][k], f);
                        if constexpr (RES) {
                            Vec8<T> rv;
                            Pair r[4];
                            from_shared(rv, ring.row(p, at, 1, i) + c);
                            get4(rv, r);
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e] = add2(f[e], r[e]);
                            set4(sv[u][k], f);
                            get4(sv[u][k], f);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) t = add2(t, f[e]);
                    }
                }
                m[u] = sum2(t);
            }
            sum(m);
            if (i0 + BATCH >= n) {  // the block is in registers
                if constexpr (TPR <= 32) __syncwarp();
                if (lead) next(at, ok);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m[u] *= inv;
                const Pair minus = both(-m[u]);
                Pair t = both(0.f);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (c0 + k * TPR * 8 < p.D) {
                        Pair f[4];
                        repack(sv[u][k]);
                        get4(sv[u][k], f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            f[e] = add2(f[e], minus);
                            t = fma2(f[e], f[e], t);
                        }
                    }
                }
                q[u] = sum2(t);
            }
            sum(q);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * S::kAbreast + abreast;
                if (i >= n) continue;
                const long long row = block + i;
                const float r = rsqrtf(fmaf(q[u], inv, p.eps));
                if (p.stats && l == 0) *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(m[u], r);
                const Pair minus = both(-m[u]), scale = both(r);
                T *const yr = y + (row * p.D + c0), *const sr = sums + (row * p.D + c0);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (c0 + k * TPR * 8 < p.D) {
                        if (RES && sums) put8(sr + k * TPR * 8, sv[u][k]);
                        const int at_w = kHold ? k : 0;
                        if constexpr (!kHold) {
                            staged<PIECES>(w[0], weights, k * TPR + l);
                            staged<PIECES>(b[0], weights + 2 * PIECES, k * TPR + l);
                        }
                        Pair f[4];
                        repack(sv[u][k]);
                        get4(sv[u][k], f);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[e] = fma2(mul2(add2(f[e], minus), scale), w[at_w][e], b[at_w][e]);
                        Vec8<T> out;
                        set4(out, f);
                        put8(yr + k * TPR * 8, out);
                    }
                }
            }
        }
    }
    if (lead && abort) drain(full[team], p.slots);
    if (threadIdx.x == 0 && abort) drain(chunks.ready, kAsked);
}

// A thread's rows leave their sums for dw and db in its registers; the CTA's row
// groups add theirs up in shared memory, in their order, and the CTA writes one row
// of `parts`.
template <typename T, typename S, bool PAST, typename A>
__global__ void __launch_bounds__(S::kBackThreads, S::kBackCtas)
    layer_norm_backward_kernel(const A p) {
    constexpr int TPR = S::TPR, VPT = S::VPT, U = rows_at_once<T, S>(true);
    constexpr int TENSORS = PAST ? 3 : 2, BATCH = U * S::kAbreast;
    constexpr bool kHold = weights_in<S>(true) == kRegisters;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[S::kBackTeams][2][(TPR >= 32 ? TPR / 32 : 1) * 2 * U];
    __shared__ uint64_t full[S::kBackTeams][kMaxSlots];
    __shared__ int abort;
    const int team = threadIdx.x / S::kTeam, lead = threadIdx.x % S::kTeam == 0;
    const int l = threadIdx.x % TPR, c0 = l * 8, abreast = threadIdx.x % S::kTeam / TPR;
    Ring<T, TENSORS> ring;
    ring.bytes = p.rows * p.D * (int)sizeof(T);
    ring.base = smem + (size_t)team * p.slots * TENSORS * ring.bytes;
    ring.full = full[team];
    ring.src[0] = static_cast<const T *>(p.x);
    ring.src[1] = static_cast<const T *>(p.dy);
    ring.ld[0] = p.ldx;
    ring.ld[1] = p.D;
    if constexpr (PAST) {
        ring.src[2] = static_cast<const T *>(p.res);
        ring.ld[2] = p.D;
    }
    const long long first = ((long long)blockIdx.x * S::kBackTeams + team) * p.rows;
    const long long step = (long long)gridDim.x * S::kBackTeams * p.rows;
    if (threadIdx.x == 0) abort = 0;
    if (lead) {
        for (int i = 0; i < p.slots; ++i) sm100::mbar_init(&full[team][i], 1);
        sm100::fence_mbar_init();
        for (int i = 0; i < p.slots; ++i) ring.fetch(p, i, first + i * step);
    }
    RowSum<TPR, 2 * U> sum = {red[team], team, 0};
    const float inv = 1.f / p.D;
    Pair w[kHold ? VPT : 1][4], dw[VPT][4], db[VPT][4];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        if constexpr (kHold) column(w[k], p.w, 1.f, c0 + k * TPR * 8, p.D);
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[k][e] = db[k][e] = both(0.f);
    }
    T *const dx = static_cast<T *>(p.y);
    float2 st[U];
    auto statistics = [&](long long block, int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * S::kAbreast + abreast;
            st[u] = make_float2(0.f, 0.f);
            if (i < p.rows && block + i < p.N) st[u] = *reinterpret_cast<const float2 *>(p.stats + 2 * (block + i));
        }
    };
    statistics(first, 0);
    __syncthreads();
    int slot = 0;
    uint32_t parity = 0;
    for (long long block = first; block < p.N; block += step) {
        const int n = (int)min((long long)p.rows, p.N - block);
        wait_dealt(&full[team][slot], parity, &abort, p);
        for (int i0 = 0; i0 < n; i0 += BATCH) {
            float2 now[U];
            float t[2 * U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * S::kAbreast + abreast;
                now[u] = st[u];
                const Pair minus = both(-now[u].x), scale = both(now[u].y);
                Pair t0 = both(0.f), t1 = t0;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = c0 + k * TPR * 8;
                    if (i < n && c < p.D) {
                        Vec8<T> sv, dv;
                        Pair f[4], d[4];
                        if constexpr (!kHold) column(w[0], p.w, 1.f, c, p.D);
                        from_shared(sv, ring.row(p, slot, 0, i) + c);
                        from_shared(dv, ring.row(p, slot, 1, i) + c);
                        get4(sv, f);
                        get4(dv, d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const Pair z = mul2(add2(f[e], minus), scale);
                            const Pair g = mul2(d[e], w[kHold ? k : 0][e]);
                            dw[k][e] = fma2(d[e], z, dw[k][e]);
                            db[k][e] = add2(db[k][e], d[e]);
                            t0 = add2(t0, g);
                            t1 = fma2(g, z, t1);
                        }
                    }
                }
                t[2 * u] = sum2(t0);
                t[2 * u + 1] = sum2(t1);
            }
            if (i0 + BATCH < n) statistics(block, i0 + BATCH);
            else statistics(block + step, 0);
            sum(t);
            if (i0 == 0) {  // the team has met: all of it is through with the block before
                if constexpr (TPR <= 32) __syncwarp();
                if (lead && block != first && p.slots > 1 && !abort)
                    ring.fetch(p, slot ? slot - 1 : p.slots - 1, block + (p.slots - 1) * step);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * S::kAbreast + abreast;
                if (i >= n) continue;
                const Pair minus = both(-now[u].x), scale = both(now[u].y);
                const Pair mg = both(-t[2 * u] * inv), mgn = both(-t[2 * u + 1] * inv);
                T *const xr = dx + ((block + i) * p.D + c0);
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int c = c0 + k * TPR * 8;
                    if (c < p.D) {
                        Vec8<T> sv, dv;
                        Pair f[4], d[4], past[4];
                        if constexpr (!kHold) column(w[0], p.w, 1.f, c, p.D);
                        from_shared(sv, ring.row(p, slot, 0, i) + c);
                        from_shared(dv, ring.row(p, slot, 1, i) + c);
                        get4(sv, f);
                        get4(dv, d);
                        if constexpr (PAST) {
                            from_shared(sv, ring.row(p, slot, 2, i) + c);
                            get4(sv, past);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const Pair z = mul2(add2(f[e], minus), scale);
                            const Pair v = fma2(z, mgn, fma2(d[e], w[kHold ? k : 0][e], mg));
                            if constexpr (PAST) f[e] = fma2(v, scale, past[e]);
                            else f[e] = mul2(v, scale);
                        }
                        set4(sv, f);
                        put8(xr + k * TPR * 8, sv);
                    }
                }
            }
        }
        if (p.slots == 1) {
            if constexpr (TPR <= 32) __syncwarp();
            else sm100::named_sync(team + 1, TPR);
            if (lead && !abort) ring.fetch(p, 0, block + step);
        }
        if (++slot == p.slots) {
            slot = 0;
            parity ^= 1;
        }
    }
    if (lead && abort) drain(full[team], p.slots);
    pdl_trigger();
    if (!p.parts) return;
    constexpr int kRowGroups = S::kBackThreads / TPR, W = TPR * 8;  // W: channels of a group's first pieces
    float *const acc = reinterpret_cast<float *>(smem);  // [groups - 1][2][8][TPR]
    const int group = threadIdx.x / TPR;
    if constexpr (kRowGroups > 1) {
        static_assert(VPT == 1, "several groups have one piece a thread");
        __syncthreads();
        if (group > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                store2(acc + ((group - 1) * 2) * W + (e * TPR + l) * 2, dw[0][e]);
                store2(acc + ((group - 1) * 2 + 1) * W + (e * TPR + l) * 2, db[0][e]);
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int q = 1; q < kRowGroups; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw[0][e] = add2(dw[0][e], load2(acc + ((q - 1) * 2) * W + (e * TPR + l) * 2));
                db[0][e] = add2(db[0][e], load2(acc + ((q - 1) * 2 + 1) * W + (e * TPR + l) * 2));
            }
    }
    float *const out = p.parts + (long long)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = c0 + k * TPR * 8;
        if (c < p.D) {
            Vec8<float> v;
            set4(v, dw[k]);
            put8(out + c, v);
            set4(v, db[k]);
            put8(out + p.D + c, v);
        }
    }
}

// dw and db: the sums of the rows of `parts`, in a fixed order.  32 warps a CTA
// of 32 columns: one warp alone would make a chain of some 300 loads.
__global__ void __launch_bounds__(1024)
    layer_norm_sum_kernel(const float *parts, int n, int D, float *dw, float *db) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    pdl_wait();  // launched beside the rows' kernel
    float s = 0.f;
    if (col < 2 * D) {
#pragma unroll 8
        for (int i = warp; i < n; i += 32) s += parts[(long long)i * 2 * D + col];
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < 2 * D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += red[i][lane];
        float *const dst = col < D ? dw : db;
        if (dst) dst[col < D ? col : col - D] = t;
    }
}

// Rows of a block, blocks of a team, CTAs, their threads and shared memory.  A
// team's block takes about 4 KB a warp and tensor (gradients of rows of several warps: 1
// KB, so that two to four fit); the rings of an SM's CTAs share its memory.  Many rows leave
// room for one block a team with the sum to form (but 12288 channels: two) and of 8192 bf16
// channels without it, in gradients up to 256 channels (1048576 rows of 64 bf16 channels 84
// us, 71 % of the copy bandwidth, with ds 95, 83 %) and of the widest float32 rows.
constexpr int kShared = 216 * 1024;  // of an SM
struct NormPlan {
    int rows, slots, grid, threads;
    bool more;
    size_t smem, most;  // of this call, and of any width of the shape
};
template <typename T, typename S> NormPlan norm_plan(long long N, int D, int tensors, bool back) {
    NormPlan r;
    const int nsm = sm_count() > 0 ? sm_count() : 152, ctas = back ? S::kBackCtas : 1;
    const int row = D * (int)sizeof(T), batch = rows_at_once<T, S>(back) * S::kAbreast;
    r.rows = (back && S::TPR > 32 ? 1024 : 4096) * (S::kTeam / 32) / row / batch * batch;
    if (r.rows < batch) r.rows = batch;
    const int fixed = !back && weights_in<S>(back) == kStaged ? 64 * S::TPR * S::VPT : 0;
    const int block = tensors * r.rows * row, room = kShared / ctas - fixed;
    int teams = back ? S::kBackTeams : S::kTeams;
    if (teams > room / block) teams = room / block;
    const long long blocks = (N + r.rows - 1) / r.rows;
    if (!back && blocks < (long long)teams * nsm) teams = (int)((blocks + nsm - 1) / nsm);
    r.threads = teams * S::kTeam;
    const int most_slots = back ? kMaxSlots : kOutSlots;
    r.slots = room / (teams * block) > most_slots ? most_slots : room / (teams * block);
    r.smem = fixed + (size_t)r.slots * teams * block;
    // the sums of the row groups but one, at the end
    const size_t sums = back ? (size_t)(S::kBackThreads / S::TPR - 1) * 16 * S::TPR * sizeof(float) : 0;
    if (r.smem < sums) r.smem = sums;
    r.most = kShared / ctas;
    const long long need = (blocks + teams - 1) / teams, most = (long long)ctas * nsm;
    r.more = !back && tensors == 2 && need > most && need <= 0x7fffffff;
    const long long grid = r.more || need < most ? need : most;
    r.grid = (int)grid;
    return r;
}

// f for the shape of D channels.  Outputs: a warp or less a row up to 2048 bf16
// channels, no barrier; above 8192 all threads of an SM, whose registers hold the weights
// (12288 and 16384 channels with the sum 85 and 90 us; rows of 256 threads that read the
// weights from the L1 cache 134 and 126); gradients: one piece a thread as far as it goes, for the
// sums in registers.
template <typename T, typename F> auto by_width(int D, F &&f) {
    const int pieces = D / 8;
    constexpr int V = 16 / (int)sizeof(T), W = 32 * 8 / V;  // pieces of a thread, threads of 256 pieces
    if (pieces <= 8) return f(RowShape<8, 1>());
    if (pieces <= 16) return f(RowShape<16, 1>());
    if (pieces <= 32) return f(RowShape<32, 1>());
    if (pieces <= 64) return f(RowShape<32, 2>());
    if (pieces <= 128) return f(RowShape<32, 4>());
    if (pieces <= 256) return f(RowShape<W, V>());
    if (pieces <= 512) return f(RowShape<2 * W, V>());
    if (pieces <= 1024) return f(RowShape<4 * W, V>());
    return f(RowShape<512, 4>());
}
// bf16 rows of three tensors that leave room for two blocks of two only go one at a time
// (8192 channels: two rows 109 us, one 95; without ds, three blocks, 71 and 85).
template <typename T, typename F> auto by_width_backward(int D, bool past, F &&f) {
    const int pieces = D / 8;
    if (pieces <= 8) return f(RowShape<8, 1>());
    if (pieces <= 16) return f(RowShape<16, 1>());
    if (pieces <= 32) return f(RowShape<32, 1>());
    if (pieces <= 64) return f(RowShape<64, 1>());
    if (pieces <= 128) return f(RowShape<128, 1>());
    if (pieces <= 256) return f(RowShape<256, 1>());
    if (pieces <= 512) return f(RowShape<256, 2>());
    if constexpr (sizeof(T) == 2)
        if (past && pieces > 768 && pieces <= 1024) return f(RowShape<512, 2, true>());
    if (pieces <= 1024) return f(RowShape<512, 2>());
    return f(RowShape<512, 4>());
}

template <typename K, typename A>
cudaError_t launch(K kern, uintptr_t (&set)[64], A p, const NormPlan &plan, cudaStream_t st) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set[dev] != context_key()) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan.most);
        if (e != cudaSuccess) return e;
        set[dev] = context_key();
    }
    p.rows = plan.rows;
    p.slots = plan.slots;
    p.more = plan.more;
    p.status = device_status_ptr();
    kern<<<plan.grid, plan.threads, plan.smem, st>>>(p);
    return cudaGetLastError();
}

template <typename T, typename S, typename A> cudaError_t forward_shape(const A &p, cudaStream_t st) {
    static uintptr_t set[2][64] = {};
    const NormPlan plan = norm_plan<T, S>(p.N, p.D, p.res ? 2 : 1, false);
    return p.res ? launch(layer_norm_kernel<T, S, true, A>, set[1], p, plan, st)
                 : launch(layer_norm_kernel<T, S, false, A>, set[0], p, plan, st);
}
template <typename T> cudaError_t forward(const NormArgs &p, cudaStream_t st) {
    return by_width<T>(p.D, [&](auto shape) { return forward_shape<T, decltype(shape)>(p, st); });
}

template <typename T, typename S, typename A>
cudaError_t backward_shape(const A &p, float *dw, float *db, cudaStream_t st) {
    static uintptr_t set[2][64] = {};
    const NormPlan plan = norm_plan<T, S>(p.N, p.D, p.res ? 3 : 2, true);
    auto rows = [&] {
        if constexpr (!S::ALONE && std::is_same<A, NormArgs>::value)
            if (!p.res) return launch(layer_norm_backward_kernel<T, S, false, A>, set[0], p, plan, st);
        return launch(layer_norm_backward_kernel<T, S, true, A>, set[1], p, plan, st);
    };
    const cudaError_t e = rows();
    if (e != cudaSuccess || !p.parts) return e;
    return launch_pdl(layer_norm_sum_kernel, (2 * p.D + 31) / 32, 1024, 0, st,
                      static_cast<const float *>(p.parts), plan.grid, p.D, dw, db);
}
template <typename T> cudaError_t backward(const NormArgs &p, float *dw, float *db, cudaStream_t st) {
    return by_width_backward<T>(p.D, p.res != nullptr, [&](auto shape) {
        return backward_shape<T, decltype(shape)>(p, dw, db, st);
    });
}

// The shapes that the self-test has: several rows a warp, a row a warp, rows of several
// warps, rows of all threads of a CTA.
template <typename F> cudaError_t by_width_tested(int D, F &&f) {
    switch (D) {
        case 64: return f(RowShape<8, 1>(), RowShape<8, 1>());
        case 2048: return f(RowShape<32, 8>(), RowShape<256, 1>());
        case 4096: return f(RowShape<64, 8>(), RowShape<256, 2>());
        case 16384: return f(RowShape<512, 4>(), RowShape<512, 4>());
    }
    return cudaErrorInvalidValue;
}

template <typename T> int most_parts(long long N, int D) {
    int most = 0;
    for (int tensors = 2; tensors <= 3; ++tensors) {
        const int n = by_width_backward<T>(D, tensors == 3, [&](auto shape) {
            return norm_plan<T, decltype(shape)>(N, D, tensors, true).grid;
        });
        most = most > n ? most : n;
    }
    return most;
}

}  // namespace

int layer_norm_parts(long long N, int D) {
    // the larger of the types' and the forms' grids
    const int a = most_parts<__nv_bfloat16>(N, D), b = most_parts<float>(N, D);
    return a > b ? a : b;
}

cudaError_t launch_layer_norm(const void *x, const void *res, const float *w, const float *b,
                              void *y, void *s, float *stats, long long N, int D, long long ldx,
                              long long ldr, float eps, gdn_dtype dt, cudaStream_t st) {
    NormArgs p = {};
    p.x = x; p.res = res; p.w = w; p.b = b; p.y = y; p.s = s; p.stats = stats;
    p.N = N; p.D = D; p.ldx = ldx; p.ldr = ldr; p.eps = eps;
    return dt == GDN_BF16 ? forward<__nv_bfloat16>(p, st) : forward<float>(p, st);
}

cudaError_t launch_layer_norm_backward(const void *s, const void *dy, const float *stats,
                                       const float *w, const void *ds, void *dx, float *dw,
                                       float *db, long long N, int D, long long lds, gdn_dtype dt,
                                       float *parts, cudaStream_t st) {
    NormArgs p = {};
    p.x = s; p.dy = dy; p.stats = const_cast<float *>(stats); p.w = w; p.res = ds; p.y = dx;
    p.parts = dw || db ? parts : nullptr;
    p.N = N; p.D = D; p.ldx = lds;
    return dt == GDN_BF16 ? backward<__nv_bfloat16>(p, dw, db, st) : backward<float>(p, dw, db, st);
}

cudaError_t launch_layer_norm_lost(const void *x, const void *res, void *y, float *stats, long long N,
                                   int D, long long limit, long long lost, cudaStream_t st) {
    LostArgs p = {};
    p.x = x; p.res = res; p.y = y; p.stats = stats; p.N = N; p.D = p.ldx = p.ldr = D; p.eps = 1e-5f;
    p.limit = limit;
    p.lost = lost < 0 ? kLostAnswer : lost;
    return by_width_tested(D, [&](auto shape, auto) {
        return forward_shape<__nv_bfloat16, decltype(shape)>(p, st);
    });
}
cudaError_t launch_layer_norm_backward_lost(const void *s, const void *dy, const float *stats,
                                            const void *ds, void *dx, float *dw, float *parts,
                                            long long N, int D, long long limit, long long lost,
                                            cudaStream_t st) {
    LostArgs p = {};
    p.x = s; p.dy = dy; p.stats = const_cast<float *>(stats); p.res = ds; p.y = dx; p.parts = parts;
    p.N = N; p.D = p.ldx = D;
    p.limit = limit;
    p.lost = lost;
    return by_width_tested(D, [&](auto, auto shape) {
        return backward_shape<__nv_bfloat16, decltype(shape)>(p, dw, nullptr, st);
    });
}

}  // namespace gdn
