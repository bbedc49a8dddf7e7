// Linear attention with a decay for each head on the tensor cores (bf16 q, k,
// v; K and V of 64 or 128), in chunks of C = 128 tokens.  With p the place of
// a token in scan order within its chunk and S the state at the chunk's start:
//
//     O = diag(read a^(p_t + 1)) [Q S^T + P V],
//         P_ts = write a^(p_t - p_s) / a^(p_t + 1) (q_t . k_s) where p_s <= p_t, else 0
//     S <- a^C S + D,   D = (diag(write a^(C - 1 - p_s)) V)^T K
//
// The row factor stands outside of both products, so that they share one
// accumulator.  It is held at 2^-64 and P takes the exact remaining power: what
// that mis-weights is S's part of rows that have decayed by more than 2^-64.
//
// Precision: P and S are rounded to bf16 as operands (a step of the bf16
// output each).  Where the state is a float32 result (`exact`) the weighted V
// goes in as three bf16 pieces that add up to it; gradients that return no state
// leave out the third (2^-16 of the value; with one piece alone their error was
// 1.6 times that of float32 arithmetic, with two it is 1.35 times: P's and S's
// rounding).  D is formed chunk by chunk from zero in the float32 accumulator, and S is kept in
// float32 registers, added to with rounding (an accumulator carried through all
// chunks would be cut, not rounded, at every product).
//
// One CTA runs one segment of one (sequence, head), 20 warps in groups of 4:
//   0-3   P: row t of Q K^T from TMEM, weighted, back to TMEM as bf16 (over the
//         columns that it came from) for the product with V.  (Eight warps that
//         shared P's columns and then O's: gradients of B = 8, T = 4096, H = 16,
//         128 x 128 took 4 us more than the 273 of now.)
//   4-7   O: row t from TMEM, scaled, to shared memory (in K's
//         place) and out by TMA (ragged chunks: plain stores)
//   8-15  state: two groups of 128 threads; each chunk's V in two halves of
//         tokens, transposed, weighted and split: two pieces to TMEM, the
//         lowest back to shared memory, all as operands of D; and S = a^C S + D
//         (thread v holds half of row v), as bf16 to shared memory for the next
//         chunk's Q S^T.  The first half of the next chunk's V goes before the
//         wait for D, so that D is formed while it runs.
//   16    loads K and V, two chunks ahead; 18 loads Q (as soon as the last
//         chunk's Q S^T is done)
//   17    issues the MMAs; 19 sends O
// Launched with 96 registers a thread (5 groups x 128 threads x 96 = 61440);
// the groups then share the same 480 registers a lane of the five as
// 2 x 96 + 2 x 128 + 32 (K = 64: 2 x 104 + 2 x 96 + 80), with which nothing
// spills: with some 20 registers of the rows spilled a chunk took half as long
// again.
// TMEM (512 columns): Q K^T and P 128 | O 128 | D 128 | V pieces 64 + 64.
#include <cstring>

#include "gdn_chunk.cuh"
#include "gdn_internal.cuh"
#include "gdn_linear.cuh"

namespace gdn {
namespace {

constexpr int kC = 128;             // tokens of a chunk
constexpr int kStages = 2;
constexpr int kWarps = 20;
constexpr int kBarP = 1, kBarS = 2;  // named barriers
constexpr uint32_t kColP = 0, kColO = 128, kColD = 256, kColHi = 384, kColMid = 448;

template <int K, int V>
struct LinLayout {
    static constexpr uint32_t QSLOT = kC * 2 * K;
    static constexpr uint32_t KSLOT = kC * 2 * K;
    static constexpr uint32_t VSLOT = kC * 2 * V;
    // as an operand of 128 rows the lowest pieces reach past V = 64 columns,
    // into what follows (rows that nothing reads)
    static constexpr uint32_t LOW = 0;
    static constexpr uint32_t Q = LOW + kC * 2 * V;
    static constexpr uint32_t KK = Q + QSLOT;
    static constexpr uint32_t VV = KK + kStages * KSLOT;
    static constexpr uint32_t S = VV + kStages * VSLOT;
    // O on its way out: the lowest pieces' place where there are none, K's slot
    // of the chunk where all of the memory is taken (K is read before O is
    // complete), else a place of its own
    static constexpr bool O_IN_K = K == 128 && V == 128;
    static constexpr uint32_t OUT = S + 2 * K * V;
    static constexpr uint32_t TABLE = OUT + (O_IN_K ? 0 : kC * 2 * V);  // column factors of P, weights of V
    static constexpr uint32_t SMEM = TABLE + 2 * kC * 4 + 1024;  // + alignment
};

template <int N> __device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of a warp whose lanes are all here.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}

// Products with descriptors given by their low words: the high word (stride
// 1024, version, swizzle) is the same for every tile here, and steps within a
// tile are additions to the address field.
constexpr uint32_t kDescHi = 0x40004040u;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHi)
        : "memory");
}

// Four 8 x 8 blocks of 16-bit values, transposed: a lane gets rows lane / 4
// (of the transposed blocks), columns 2 (lane % 4) and the next, of each.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The way back.
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                                uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// 16 TMEM lanes x 16 columns: register 4 c + 2 m + r of a lane goes to TMEM
// lane 8 r + lane / 4, column 8 c + 4 m + lane % 4.
__device__ __forceinline__ void tmem_st_16x128(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}
// The upper halves of two words, x's below y's.
__device__ __forceinline__ uint32_t upper_halves(float x, float y) {
    return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
__device__ __forceinline__ float upper_half(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}
// a *= f, b *= g as one packed product.
__device__ __forceinline__ void mul2(float &a, float &b, float f, float g) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(g));
}
// a = f a + c, b = f b + d as one packed operation.
__device__ __forceinline__ void fma2(float &a, float &b, float f, float c, float d) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %4};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(c), "f"(d));
}
// x -= upper_half(x), y -= upper_half(y) as one packed operation (exact).
__device__ __forceinline__ void drop_upper_halves(float &x, float &y) {
    const float u = upper_half(x), w = upper_half(y);
    asm("{\n\t.reg .b64 a, b, m;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "mov.b64 m, {%4, %4};\n\tfma.rn.f32x2 a, b, m, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(u), "f"(w), "f"(-1.f));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's 32 scores in TMEM times a^lag / rho (the way of strong decays): `lag0`
// is the first column's lag, which rises along the row (up) or falls.
__device__ __forceinline__ void weigh_each(uint32_t taddr, int lag0, bool up, float lg, float lrho) {
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
        uint32_t r[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr + c));
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int lag = up ? lag0 + c + e : lag0 - c - e;
            r[e] = __float_as_uint(__uint_as_float(r[e]) * ex2((float)max(lag, 0) * lg - lrho));
        }
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr + c),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    }
    tmem_st_wait();
}

// Block b of 32 columns of row t of a tile of kCols (64 or 32) columns, in the
// swizzle of its row length (128 or 64 bytes).
template <int kCols>
__device__ __forceinline__ void store_row_out(uint8_t *tile, int t, int b, const float (&x)[32]) {
    if constexpr (kCols == 64) {
        store_row<4>(tile, t, 4 * b, x);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4 *>(tile + t * 64 + ((c ^ ((t >> 1) & 3)) << 4)) =
                make_uint4(pack_bf16(x[8 * c], x[8 * c + 1]), pack_bf16(x[8 * c + 2], x[8 * c + 3]),
                           pack_bf16(x[8 * c + 4], x[8 * c + 5]), pack_bf16(x[8 * c + 6], x[8 * c + 7]));
    }
}

// mbar_try_wait that leaves the thread asleep until the phase completes, or
// for up to a millisecond: waits that spun took two fifths of all issued
// instructions.
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}

// acc stays 0 while the pairs of bf16 values that it meets are finite.
__device__ __forceinline__ void note_not_finite(uint32_t &acc, uint32_t pair) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(pair), "r"(0u));
}

struct LinBars {
    uint64_t kfull[kStages], vfull[kStages], used[kStages], sent[kStages], staged, qfull, qs, d0, dfree;
    uint64_t vw[2], scores, p, d, s, o, ofree, tail, out;
};

struct LinTcArgs {
    LinearScan a;
    SegPlan plan;
    const float *slots_in;
    float *slots_out;
    int *status;
};

// P V meets the values of V with the zeros of P's other triangle too, so that
// one that is not finite reaches the outputs of its channel from its chunk's
// first token on.  A warp forms those before it again, token by token from the
// segment's start (the rest are right, or not finite).  Such a value stays in
// the state, so that a segment's end tells whether there is one and nothing is
// looked at before (marks in the chunks' loop cost 2 to 9 % of the time).
template <int K, int V>
__device__ __forceinline__ void outputs_before_bad_value(const LinTcArgs &arg, const LinearItem &it, int h,
                                                      int f0, int tokens, int ch) {
    constexpr int C = K / 32;  // columns of a lane
    const LinearScan &p = arg.a;
    const int lane = threadIdx.x & 31;
    const bool rev = p.reverse, first = rev ? it.j == it.n - 1 : it.j == 0;
    const long long t0 = it.first + f0;
    const __nv_bfloat16 *const v = static_cast<const __nv_bfloat16 *>(p.v) + h / (p.H / p.Hv) * V + ch;
    auto token = [&](int y) { return t0 + (rev ? tokens - 1 - y : y); };
    int bad = -1;  // scan position of the first that is not finite
#pragma unroll 1
    for (int y0 = 0; y0 < tokens && bad < 0; y0 += 32) {
        const int y = y0 + lane;
        const float x = y < tokens ? __bfloat162float(v[token(y) * p.ldv]) : 0.f;
        const unsigned who = __ballot_sync(0xffffffffu, !(fabsf(x) < INFINITY));
        if (who) bad = y0 + __ffs(who) - 1;
    }
    if (bad < 0) return;
    // scan position of its chunk's first token
    const int at = (rev ? tokens - 1 - bad : bad) / kC * kC;
    const int from = rev ? tokens - min(tokens, at + kC) : at;
    const float a = p.alpha[h], lg = decay_log2(a);
    float S[C];
    auto add_row = [&](size_t row, float f) {
#pragma unroll
        for (int c = 0; c < C; ++c) S[c] = fmaf(f, arg.slots_in[(row * V + ch) * K + lane * C + c], S[c]);
    };
#pragma unroll
    for (int c = 0; c < C; ++c)
        S[c] = p.S0 && !arg.slots_in ? given_start(p.S0, p.s0_transposed, (size_t)it.seq * p.H + h, V, K,
                                                   ch, lane * C + c)
                                     : 0.f;
    if (arg.slots_in) {
        if (p.S0)
            add_row((size_t)(it.slot0 + (rev ? 0 : it.n - 1)) * p.H + h,
                    decay_power(start_steps(it, arg.plan.seg_len, rev), lg));
        for (int j = rev ? it.j + 1 : 0; j < (rev ? it.n : it.j); ++j)
            add_row((size_t)(it.slot0 + j) * p.H + h,
                    decay_power(tokens_between(j, it.j, it.len, arg.plan.seg_len, rev), lg));
    }
    const __nv_bfloat16 *const k =
        static_cast<const __nv_bfloat16 *>(p.k) + h / (p.H / p.Hk) * K + lane * C;
    const __nv_bfloat16 *const q =
        static_cast<const __nv_bfloat16 *>(p.q) + h / (p.H / p.Hq) * K + lane * C;
    auto take = [&](int y) {
        const long long t = token(y);
        const float w = p.write_scale * __bfloat162float(v[t * p.ldv]);
        const float d = rev && first && y == 0 ? 1.f : a;
#pragma unroll
        for (int c = 0; c < C; ++c) S[c] = fmaf(w, __bfloat162float(k[t * p.ldk + c]), d * S[c]);
    };
#pragma unroll 4
    for (int y = 0; y < from; ++y) take(y);
#pragma unroll 1
    for (int y = from; y < bad; ++y) {
        take(y);
        const long long t = token(y);
        float o = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) o = fmaf(S[c], __bfloat162float(q[t * p.ldq + c]), o);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) o += __shfl_xor_sync(0xffffffffu, o, off);
        if (lane == 0) {
            const size_t e = ((size_t)t * p.H + h) * V + ch;
            if (p.o_float) static_cast<float *>(p.o)[e] = p.read_scale * o;
            else static_cast<__nv_bfloat16 *>(p.o)[e] = __float2bfloat16_rn(p.read_scale * o);
        }
    }
}

template <int K, int V>
__global__ void __launch_bounds__(kWarps * 32, 1)
    linear_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                     const LinTcArgs arg) {
    using L = LinLayout<K, V>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ LinBars bar;
    __shared__ uint32_t tmem_at;
    __shared__ int abort_flag;
    volatile int *abort_v = &abort_flag;

    const LinearScan &p = arg.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % p.H;
    const LinearItem it =
        linear_item(p.offsets, p.B, p.T, arg.plan.seg_len, blockIdx.x / p.H, arg.status);
    if (it.seq < 0) return;
    const bool rev = p.reverse;
    const bool last = rev ? it.j == 0 : it.j == it.n - 1;  // segment, in scan order
    const bool first = rev ? it.j == it.n - 1 : it.j == 0;
    float *const slot = arg.slots_out
                            ? arg.slots_out + ((size_t)(it.slot0 + it.j) * p.H + h) * V * K
                            : nullptr;
    if (slot && last) {  // nothing starts from its end: the slot takes a copy of S0
        if (p.S0)
            for (int i = tid; i < V * K; i += kWarps * 32)
                slot[i] = given_start(p.S0, p.s0_transposed, (size_t)it.seq * p.H + h, V, K, i / K,
                                      i % K);
        return;
    }
    const bool want_o = p.o && !slot;
    float *const end = slot ? slot
                       : p.ST && last ? p.ST + ((size_t)it.seq * p.H + h) * V * K : nullptr;
    const int f0 = it.j * arg.plan.seg_len;
    const int tokens = min(it.len - f0, arg.plan.seg_len);
    const int nc = (tokens + kC - 1) / kC;
    // i-th chunk in scan order: first token (from the segment's first) and number
    auto chunk_at = [&](int i) { return (rev ? nc - 1 - i : i) * kC; };
    auto chunk_n = [&](int i) { return min(kC, tokens - chunk_at(i)); };
    // a reversed scan takes its start state up undecayed
    auto chunk_lead = [&](int i) { return rev && first && i == 0 ? 0 : 1; };
    const float lg = decay_log2(p.alpha[h]);

    if (warp == 17) {
        tmem_alloc(&tmem_at, 512);
        tmem_relinquish();
        if (lane == 0) {
            for (int s = 0; s < kStages; ++s) {
                mbar_init(&bar.kfull[s], 1);
                mbar_init(&bar.vfull[s], 1);
                mbar_init(&bar.used[s], 1);
                mbar_init(&bar.sent[s], 1);
            }
            mbar_init(&bar.staged, 4);
            mbar_init(&bar.qfull, 1);
            mbar_init(&bar.qs, 1);
            mbar_init(&bar.d0, 1);
            mbar_init(&bar.dfree, 8);
            mbar_init(&bar.scores, 1);
            mbar_init(&bar.p, 4);
            mbar_init(&bar.vw[0], 8);
            mbar_init(&bar.vw[1], 8);
            mbar_init(&bar.d, 1);
            mbar_init(&bar.s, 8);
            mbar_init(&bar.o, 1);
            mbar_init(&bar.ofree, 4);
            mbar_init(&bar.tail, 8);
            mbar_init(&bar.out, 1);
            abort_flag = 0;
            fence_mbar_init();
        }
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    const uint32_t quad = (uint32_t)(warp & 3) << 21;  // 32 TMEM lanes of this warp
    float *const colfac = reinterpret_cast<float *>(smem + L::TABLE);
    float *const vweight = colfac + kC;

    if (!want_o && tid < kC)
        vweight[tid] = p.write_scale * exp2f((float)(rev ? tid : kC - 1 - tid) * lg);
    __syncthreads();

    // After a wait has run out every later wait returns at once and nothing is
    // written any more, but the loops keep their barriers and end.
    bool dead = false;
    auto wait = [&](uint64_t *b, uint32_t parity) {
        if (dead || mbar_sleep_wait(b, parity & 1)) return;
        const uint32_t t0 = (uint32_t)clock();
#pragma unroll 1
        while (!mbar_sleep_wait(b, parity & 1))
            if (*abort_v || (uint32_t)clock() - t0 > (uint32_t)kSpinLimit) {
                *abort_v = 1;
                dead = true;
                return;
            }
    };
    // chunks whose D is formed: all but a last one whose end nobody wants
    auto updates = [&](int i) { return i + 1 < nc || end; };
    const bool o_in_k = L::O_IN_K && p.exact;
    auto o_place = [&](int i) {
        return smem + (o_in_k ? L::KK + (i % kStages) * L::KSLOT : L::O_IN_K ? L::LOW : L::OUT);
    };
    auto wait_warp = [&](uint64_t *b, uint32_t parity) {
        wait(b, parity);
        __syncwarp();
    };
    auto arrive_warp = [&](uint64_t *b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };

    // Half c of chunk i's V, by 4 warps for each half g of its tokens: a warp's
    // lanes of TMEM are 32 channels.  Lanes 8 j .. address block j: tokens
    // + 8 (j / 2), channels + 8 (j % 2).
    auto convert = [&](int i, int c, int g) {
        const uint32_t tok = g * 64 + (lane & 7) + ((lane >> 4) << 3);
        const float2 *w2 = reinterpret_cast<const float2 *>(vweight) + g * 32 + (lane & 3);
        // 32 tokens of this group's 64, as bf16 pieces, each the upper half of
        // what is left: three whose sum is the float32 product (exact), or two
        if ((warp & 3) * 32 < V) {
            float2 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = w2[16 * c + 4 * e];
#pragma unroll 1
            for (int r = 0; r < 2; ++r) {  // 16 channels
                const uint32_t col = (uint32_t)(warp & 3) * 32 + 16 * r + (lane & 8);
                const uint32_t off = (col >> 6) * (kC * 128) + swz128(tok, (col & 63) >> 3) + c * 4096;
                const uint32_t src = smem_u32(smem) + L::VV + (i % kStages) * L::VSLOT + off;
                const uint32_t at = tmem + quad + ((uint32_t)r << 20) + g * 32 + 16 * c;
                uint32_t hi[8], x[2][4];
                ldmatrix4_trans(x[0], src);
                ldmatrix4_trans(x[1], src + 2048);
                uint32_t mid[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint32_t &z = x[e >> 2][e & 3];
                    float u = __uint_as_float(z << 16);
                    float y = __uint_as_float(z & 0xffff0000u);
                    mul2(u, y, w[e >> 1].x, w[e >> 1].y);
                    hi[e] = upper_halves(u, y);
                    drop_upper_halves(u, y);
                    if (p.exact) {
                        mid[e] = upper_halves(u, y);
                        drop_upper_halves(u, y);
                        z = upper_halves(u, y);
                    } else {
                        mid[e] = pack_bf16(u, y);
                    }
                }
                tmem_st_16x128(at + kColMid, mid);
                if (p.exact) {
                    const uint32_t low = smem_u32(smem) + L::LOW + off;
                    stmatrix4_trans(low, x[0][0], x[0][1], x[0][2], x[0][3]);
                    stmatrix4_trans(low + 2048, x[1][0], x[1][1], x[1][2], x[1][3]);
                }
                tmem_st_16x128(at + kColHi, hi);
            }
            tmem_st_wait();
            fence_proxy_async_smem();
        }
    };
    // without outputs the rows' warps take the second halves
    const bool help = !want_o && tokens % kC == 0;

    if (warp < 8) {
        // ---------------------------------------------------------------- rows
        if constexpr (K == 64) reg_inc<104>();
        if (help) {
#pragma unroll 1
            for (int i = 0; i < nc && updates(i); ++i) {
                wait_warp(&bar.vfull[i % kStages], i / kStages);
                if (i > 0) wait_warp(&bar.d, i - 1);  // the pieces' places are free
                convert(i, 1, warp >> 2);
                tc_fence_before();
                arrive_warp(&bar.vw[1]);
            }
        }
        const int t = (warp & 3) * 32 + lane;
        if (want_o && warp < 4) {
            // the powers within a block of 32 columns; a row's factor of the block
            // takes the rest of the lag
            if (t < 32) colfac[t] = p.write_scale * exp2f((float)(rev ? t : 31 - t) * lg);
            named_sync(kBarP, 128);
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                const int n = chunk_n(i), lead = chunk_lead(i);
                const int pt = (rev ? n - 1 - t : t) + lead;
                const float lrho = fmaxf((float)pt * lg, -64.f);
                wait_warp(&bar.scores, i);
                tc_fence_after();
                // In blocks of 32 columns.  Rolled: twenty warps in their roles,
                // unrolled, missed the instruction cache at every chunk (a quarter
                // of all stalls).
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t w[16];
                    const bool blank = rev ? b < warp : b > warp;
                    float x[32];
                    // one power for the row and block: within the diagonal block
                    // it reaches a^-31, so that where a < 1/4 its scores are
                    // weighted one by one instead
                    const bool each = b == warp && lg < -2.f;
                    const int far = rev ? 32 * b - t : t - 32 * b - 31;
                    if (!blank) {
                        if (each) weigh_each(tmem + quad + kColP + 32 * b, rev ? far : far + 31, rev, lg, lrho);
                        tmem_ld32(tmem + quad + kColP + 32 * b, x);
                        tmem_ld_wait();
                    }
                    if (blank) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = 0;
                    } else {
                        const float rf = each ? p.write_scale : ex2((float)far * lg - lrho);
                        const float4 *f4 = reinterpret_cast<const float4 *>(colfac);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 f = each ? make_float4(1.f, 1.f, 1.f, 1.f) : f4[e];
                            mul2(x[4 * e], x[4 * e + 1], f.x, f.y);
                            mul2(x[4 * e + 2], x[4 * e + 3], f.z, f.w);
                            mul2(x[4 * e], x[4 * e + 1], rf, rf);
                            mul2(x[4 * e + 2], x[4 * e + 3], rf, rf);
                        }
                        pack_row(x, w);
                        if (b == warp) {  // the columns at or before this row, in scan order
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                // 16 bits of a pair for each of its columns that counts
                                const int bits = 16 * (rev ? 2 * e + 2 - lane : lane + 1 - 2 * e);
                                const uint32_t ones = __funnelshift_lc(0xffffffffu, 0u, max(bits, 0));
                                w[e] &= rev ? __brev(ones) : ones;
                            }
                        }
                    }
                    tmem_st16(tmem + quad + kColP + 16 * b, w);
                }
                tmem_st_wait();
                tc_fence_before();
                arrive_warp(&bar.p);
            }
        } else if (want_o) {
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                const int n = chunk_n(i);
                const int pt = (rev ? n - 1 - t : t) + chunk_lead(i);
                const float rho = p.read_scale * ex2(fmaxf((float)pt * lg, -64.f));
                const bool whole = n == kC && !p.o_float;
                constexpr int kCols = V / 2;  // of a tile on its way out
                uint8_t *const stage = o_place(i);
                if (!o_in_k && i > 0) wait_warp(&bar.sent[(i - 1) % kStages], (i - 1) / kStages);
                wait_warp(&bar.o, i);
                tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < V / 32; ++b) {
                    float x[32];
                    tmem_ld32(tmem + quad + kColO + 32 * b, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 16; ++e) mul2(x[2 * e], x[2 * e + 1], rho, rho);
                    if (whole) {
                        store_row_out<kCols>(stage + 32 * b / kCols * (kC * 2 * kCols), t, b % (kCols / 32), x);
                    } else if (t < n && !dead) {
                        const size_t at = ((size_t)(it.first + f0 + chunk_at(i) + t) * p.H + h) * V +
                                          32 * b;
                        if (p.o_float) {
                            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                        } else {
                            uint32_t w[16];
                            pack_row(x, w);
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + at);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                dst[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                        }
                    }
                    __syncwarp();
                }
                tc_fence_before();
                fence_proxy_async_smem();
                // first: O's columns free, another warp may come to stage the next chunk
                arrive_warp(&bar.staged);
                arrive_warp(&bar.ofree);
            }
        }
    } else if (warp < 16) {
        // ---------------------------------------------------------------- state
        if constexpr (K == 128) reg_inc<128>();
        constexpr int NS = K / 2;
        const int g = (warp - 8) >> 2;
        const int v = (warp & 3) * 32 + lane;
        const bool mine = (warp & 3) * 32 < V;  // V = 64: lanes 64.. carry nothing
        const int k0 = g * NS;
        float S[NS];
        if (!slot && mine) {
#pragma unroll
            for (int e = 0; e < NS; ++e) S[e] = 0.f;
            if (p.S0) {
                const float f = decay_power(start_steps(it, arg.plan.seg_len, rev), lg);
                if (arg.slots_in) {
                    const float4 *src = reinterpret_cast<const float4 *>(
                        arg.slots_in + (((size_t)(it.slot0 + (rev ? 0 : it.n - 1)) * p.H + h) * V + v) * K + k0);
#pragma unroll
                    for (int e = 0; e < NS / 4; ++e) {
                        const float4 x = src[e];
                        S[4 * e] = f * x.x; S[4 * e + 1] = f * x.y;
                        S[4 * e + 2] = f * x.z; S[4 * e + 3] = f * x.w;
                    }
                } else {
                    const size_t head = (size_t)it.seq * p.H + h;
#pragma unroll
                    for (int e = 0; e < NS; ++e)
                        S[e] = f * given_start(p.S0, p.s0_transposed, head, V, K, v, k0 + e);
                }
            }
            if (arg.slots_in) {
                for (int j = rev ? it.j + 1 : 0; j < (rev ? it.n : it.j); ++j) {
                    const int gap = tokens_between(j, it.j, it.len, arg.plan.seg_len, rev);
                    const float f = decay_power(gap, lg);
                    const float4 *src = reinterpret_cast<const float4 *>(
                        arg.slots_in + (((size_t)(it.slot0 + j) * p.H + h) * V + v) * K + k0);
#pragma unroll
                    for (int e = 0; e < NS / 4; ++e) {
                        const float4 x = src[e];
                        S[4 * e] = fmaf(f, x.x, S[4 * e]);
                        S[4 * e + 1] = fmaf(f, x.y, S[4 * e + 1]);
                        S[4 * e + 2] = fmaf(f, x.z, S[4 * e + 2]);
                        S[4 * e + 3] = fmaf(f, x.w, S[4 * e + 3]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < NS; ++e) S[e] = 0.f;
        }
        const int st = tid - 256;  // 0..255 of both groups
        int n_table = help ? kC : -1;
        auto store_state = [&] {
            if (mine) {
                // rows of 128 bytes hold 64 columns; K = 64: the groups share one row
#pragma unroll
                for (int e = 0; e < NS / 32; ++e) {
                    float x[32];
#pragma unroll
                    for (int y = 0; y < 32; ++y) x[y] = S[32 * e + y];
                    const int col = k0 + 32 * e;
                    store_row<4>(smem + L::S + (col / 64) * (V * 128), v, (col % 64) / 8, x);
                }
            }
            fence_proxy_async_smem();
            arrive_warp(&bar.s);
        };
        if (want_o && nc > 0) store_state();
        // step 2 i + c: half c of chunk i's V; S takes chunk i - 1 up after the
        // first half of chunk i is on its way
#pragma unroll 1
        for (int step = 0; step <= 2 * nc; ++step) {
            const int i = step >> 1, c = step & 1;
            if (c == 0 && i < nc) {
                const int n = chunk_n(i);
                wait_warp(&bar.vfull[i % kStages], i / kStages);
                if (n < kC) {
                    wait_warp(&bar.kfull[i % kStages], i / kStages);
                    // the rows behind the sequence's last token are another's, or none
                    const uint4 zero = make_uint4(0, 0, 0, 0);
                    uint8_t *kt = smem + L::KK + (i % kStages) * L::KSLOT,
                            *vt = smem + L::VV + (i % kStages) * L::VSLOT;
                    for (int x = st; x < (kC - n) * 8; x += 256) {
                        const int at = (n + x / 8) * 128 + (x % 8) * 16;
#pragma unroll
                        for (int b = 0; b < K / 64; ++b)
                            *reinterpret_cast<uint4 *>(kt + b * (kC * 128) + at) = zero;
#pragma unroll
                        for (int b = 0; b < V / 64; ++b)
                            *reinterpret_cast<uint4 *>(vt + b * (kC * 128) + at) = zero;
                    }
                    fence_proxy_async_smem();
                    named_sync(kBarS, 256);
                    arrive_warp(&bar.tail);
                }
                if (n != n_table && updates(i)) {  // both groups come here together
                    named_sync(kBarS, 256);
                    if (st < kC)
                        vweight[st] = st < n ? p.write_scale * exp2f((float)(rev ? st : n - 1 - st) * lg) : 0.f;
                    named_sync(kBarS, 256);
                    n_table = n;
                }
                if (i > 0 && updates(i)) wait_warp(&bar.d0, i - 1);  // the pieces' places are free
            }
            if (i < nc && updates(i) && !(help && c)) {
                convert(i, c, g);
                tc_fence_before();
                arrive_warp(&bar.vw[c]);
            }
            if (c == 0 && i > 0 && updates(i - 1)) {
                const float ac = exp2f((float)(chunk_n(i - 1) + chunk_lead(i - 1) - 1) * lg);
                wait_warp(&bar.d, i - 1);
                tc_fence_after();
                if (mine) {
#pragma unroll
                    for (int e = 0; e < NS / 32; ++e) {
                        float x[32];
                        tmem_ld32(tmem + quad + kColD + k0 + 32 * e, x);
                        tmem_ld_wait();
#pragma unroll
                        for (int y = 0; y < 32; y += 2)
                            fma2(S[32 * e + y], S[32 * e + y + 1], ac, x[y], x[y + 1]);
                    }
                }
                tc_fence_before();
                arrive_warp(&bar.dfree);
                if (want_o && i < nc) store_state();
            }
        }
        if (want_o && nc > 0 && g == 0 && (warp & 3) * 32 < V) {
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < NS; ++e) z = fmaf(S[e], 0.f, z);
            unsigned channels = __ballot_sync(0xffffffffu, z != 0.f);
            if (!end) {  // the last chunk has not been taken up
                const uint8_t *const vt = smem + L::VV + ((nc - 1) % kStages) * L::VSLOT +
                                          ((warp & 3) >> 1) * (kC * 128);
                uint32_t acc = 0;
#pragma unroll 1
                for (uint32_t tok = lane; tok < kC; tok += 32)
#pragma unroll
                    for (uint32_t x = 0; x < 4; ++x) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(
                            vt + swz128(tok, 4 * (warp & 1) + x));
                        note_not_finite(acc, y.x);
                        note_not_finite(acc, y.y);
                        note_not_finite(acc, y.z);
                        note_not_finite(acc, y.w);
                    }
                if (__any_sync(0xffffffffu, acc != 0)) channels = ~0u;
            }
            if (channels) {
                wait_warp(&bar.out, 0);  // all outputs are in memory
                if (!__any_sync(0xffffffffu, dead))
                    for (; channels; channels &= channels - 1)
                        outputs_before_bad_value<K, V>(arg, it, h, f0, tokens,
                                                       (warp & 3) * 32 + __ffs(channels) - 1);
            }
        }
        if (want_o) named_sync(kBarS, 256);  // the end states may take the start states' place
        if (end && mine && !dead) {
            // the state that a reversed scan returns has decayed once more
            const float f = !slot && rev && it.len > 0 ? exp2f(lg) : 1.f;
            float4 *dst = reinterpret_cast<float4 *>(end + (size_t)v * K + k0);
#pragma unroll
            for (int e = 0; e < NS / 4; ++e)
                dst[e] = make_float4(f * S[4 * e], f * S[4 * e + 1], f * S[4 * e + 2], f * S[4 * e + 3]);
        }
    } else {
        reg_dec<K == 128 ? 32 : 80>();
        // ---------------------------------------------------------------- loads
        auto token_at = [&](int i) { return (p.offsets ? it.base : 0) + f0 + chunk_at(i); };
        const int c3 = p.offsets ? 0 : it.seq;
        if (warp == 16 && elect_one()) {
            tma_prefetch_desc(&mk);
            tma_prefetch_desc(&mv);
            const int hk = h / (p.H / p.Hk), hv = h / (p.H / p.Hv);
            int vs = 0, ks = 0;  // loads issued
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                const int s = i % kStages;
                if (i >= kStages) wait(&bar.used[s], i / kStages - 1);
                if (dead) break;
                mbar_arrive_expect_tx(&bar.vfull[s], kC * 2 * V);
                vs = i + 1;
#pragma unroll
                for (int b = 0; b < V / 64; ++b)
                    tma_load_4d(smem + L::VV + s * L::VSLOT + b * (kC * 128), &mv, &bar.vfull[s],
                                64 * b, hv, token_at(i), c3);
                if (o_in_k && want_o && i >= kStages) wait(&bar.sent[s], i / kStages - 1);
                if (dead) break;
                mbar_arrive_expect_tx(&bar.kfull[s], kC * 2 * K);
                ks = i + 1;
#pragma unroll
                for (int b = 0; b < K / 64; ++b)
                    tma_load_4d(smem + L::KK + s * L::KSLOT + b * (kC * 128), &mk, &bar.kfull[s],
                                64 * b, hk, token_at(i), c3);
                // the next, whose place is not free yet, to the L2 cache
                if (i > 0 && i + 1 < nc) {
#pragma unroll
                    for (int b = 0; b < V / 64; ++b)
                        tma_prefetch_l2_4d(&mv, 64 * b, hv, token_at(i + 1), c3);
#pragma unroll
                    for (int b = 0; b < K / 64; ++b)
                        tma_prefetch_l2_4d(&mk, 64 * b, hk, token_at(i + 1), c3);
                }
            }
            // copies in flight land before the CTA ends (again with a limit)
            for (int i = vs > kStages ? vs - kStages : 0; i < vs; ++i)
                mbar_wait(&bar.vfull[i % kStages], (i / kStages) & 1, kSpinLimit);
            for (int i = ks > kStages ? ks - kStages : 0; i < ks; ++i)
                mbar_wait(&bar.kfull[i % kStages], (i / kStages) & 1, kSpinLimit);
        }
        if (warp == 18 && want_o && elect_one()) {
            tma_prefetch_desc(&mq);
            const int hq = h / (p.H / p.Hq);
            int issued = 0;
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                if (i > 0) wait(&bar.qs, i - 1);
                if (dead) break;
                mbar_arrive_expect_tx(&bar.qfull, kC * 2 * K);
                issued = i + 1;
#pragma unroll
                for (int b = 0; b < K / 64; ++b)
                {
                    tma_load_4d(smem + L::Q + b * (kC * 128), &mq, &bar.qfull, 64 * b, hq,
                                token_at(i), c3);
                    if (i + 1 < nc) tma_prefetch_l2_4d(&mq, 64 * b, hq, token_at(i + 1), c3);
                }
            }
            if (issued) mbar_wait(&bar.qfull, (issued - 1) & 1, kSpinLimit);
        }
        // ---------------------------------------------------------------- O out
        if (warp == 19 && want_o && elect_one()) {
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                wait(&bar.staged, i);
                if (chunk_n(i) == kC && !p.o_float && !dead) {
                    const uint8_t *stage = o_place(i);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        tma_store_4d(&mo, stage + b * (kC * V), b * (V / 2), h, token_at(i), c3);
                    bulk_commit_group();
                    bulk_wait_read_all();
                }
                mbar_arrive(&bar.sent[i % kStages]);
            }
            bulk_wait_all();
            mbar_arrive(&bar.out);
        }
        // ---------------------------------------------------------------- MMAs
        if (warp == 17 && elect_one()) {
            const uint32_t base = smem_u32(smem);
            constexpr uint32_t id_scores = idesc_bf16(128, 128, false, false);
            constexpr uint32_t id_qs = idesc_bf16(128, V, false, false);
            constexpr uint32_t id_pv = idesc_bf16(128, V, false, true);
            constexpr uint32_t id_d = idesc_bf16(128, K, false, true);
            constexpr uint32_t id_low = idesc_bf16(128, K, true, true);
            const uint32_t q = desc_lo(base + L::Q, 16), k_0 = desc_lo(base + L::KK, 16),
                           s_0 = desc_lo(base + L::S, 16), kt_0 = desc_lo(base + L::KK, kC * 128),
                           v_0 = desc_lo(base + L::VV, kC * 128), low = desc_lo(base + L::LOW, kC * 128);
#pragma unroll 1
            for (int i = 0; i < nc; ++i) {
                const int s = i % kStages;
                const uint32_t kt = kt_0 + s * (L::KSLOT >> 4);
                wait(&bar.kfull[s], i / kStages);
                wait(&bar.vfull[s], i / kStages);
                if (chunk_n(i) < kC) wait(&bar.tail, 0);  // one ragged chunk a segment
                if (want_o) {
                    const uint32_t k = k_0 + s * (L::KSLOT >> 4);
                    wait(&bar.qfull, i);
                    if (i > 0) wait(&bar.o, i - 1);  // P, in the scores' columns, is read
                    tc_fence_after();
                    if (dead) continue;
#pragma unroll 1
                    for (int y = 0; y < K / 64; ++y)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t off = y * (kC * 8) + 2 * x;
                            mma_ss(tmem + kColP, q + off, k + off, id_scores, y + x > 0);
                        }
                    mma_commit(&bar.scores);
                }
                // D's first half goes ahead of the state's way through shared memory
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    if (updates(i)) {
                        wait(&bar.vw[c], i);
                        if (c == 0 && i > 0) wait(&bar.dfree, i - 1);
                        tc_fence_after();
                        if (dead) break;
                        // the small pieces first: the sum is cut to its size at each product
#pragma unroll 1
                        for (int y = p.exact ? 0 : 1; y < 3; ++y) {
                            const uint32_t a = tmem + (y == 1 ? kColMid : kColHi);
                            const bool on = c > 0 || y == 2 || (y == 1 && p.exact);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {  // tokens 32 c .. and 64 + 32 c ..
                                const int z = 2 * c + (x & 1) + 4 * (x >> 1);
                                if (y == 0)
                                    mma_ss(tmem + kColD, low + z * (2048 >> 4), kt + z * (2048 >> 4),
                                           id_low, on || x > 0);
                                else
                                    mma_ts(tmem + kColD, a + 8 * z, kt + z * (2048 >> 4), id_d, on || x > 0);
                            }
                        }
                        mma_commit(c ? &bar.d : &bar.d0);
                    }
                    if (c == 0 && want_o) {
                        wait(&bar.s, i);
                        if (i > 0) wait(&bar.ofree, i - 1);
                        tc_fence_after();
                        if (dead) break;
#pragma unroll 1
                        for (int y = 0; y < K / 64; ++y)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                mma_ss(tmem + kColO, q + y * (kC * 8) + 2 * x,
                                       s_0 + y * (V * 8) + 2 * x, id_qs, y + x > 0);
                        mma_commit(&bar.qs);
                    }
                }
                if (want_o) {
                    wait(&bar.p, i);
                    tc_fence_after();
                    if (dead) continue;
                    const uint32_t v = v_0 + s * (L::VSLOT >> 4);
#pragma unroll 4
                    for (int x = 0; x < kC / 16; ++x)
                        mma_ts(tmem + kColO, tmem + kColP + 8 * x, v + x * (2048 >> 4), id_pv, 1);
                    mma_commit(&bar.o);
                }
                if (dead) continue;
                mma_commit(&bar.used[s]);
            }
            // every product is done before the tensor memory is given back
            if (nc > 0)
                mbar_wait(&bar.used[(nc - 1) % kStages], ((nc - 1) / kStages) & 1,
                          dead ? 1000000 : kSpinLimit);
        }
    }
    if (dead) *abort_v = 1;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*abort_v && tid == 0 && arg.status) atomicOr(arg.status, kStatusTimeout);
    if (warp == 17) tmem_dealloc(tmem, 512);
}

template <int K, int V>
cudaError_t launch_kv(const LinearScan &a, float *slots, cudaStream_t st) {
    using L = LinLayout<K, V>;
    static uintptr_t attr_set[64] = {};  // context the attribute was set in
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kern = linear_tc_kernel<K, V>;
    if (attr_set[dev] != context_key()) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = context_key();
    }
    const bool packed = a.offsets != nullptr;
    const int B = packed ? 1 : a.B;
    CUtensorMap mq, mk, mv, mo;
    if (!make_strided_token_map(&mk, a.k, B, a.T, a.ldk, a.ldk * a.T, a.Hk, K, kC) ||
        !make_strided_token_map(&mv, a.v, B, a.T, a.ldv, a.ldv * a.T, a.Hv, V, kC))
        return cudaErrorInvalidValue;
    mq = mk;
    mo = mv;
    if (a.o && !make_strided_token_map(&mq, a.q, B, a.T, a.ldq, a.ldq * a.T, a.Hq, K, kC))
        return cudaErrorInvalidValue;
    const long long ldo = (long long)a.H * V;
    if (a.o && !a.o_float && !make_strided_token_map(&mo, a.o, B, a.T, ldo, ldo * a.T, a.H, V, kC, V / 2))
        return cudaErrorInvalidValue;
    LinTcArgs arg = {a, linear_tc_plan(a.B, a.T, a.H, K, V, packed), nullptr, nullptr,
                     device_status_ptr()};
    const long long grid = (long long)arg.plan.items * a.H;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (arg.plan.items > a.B) {
        arg.slots_out = slots;
        kern<<<(unsigned)grid, kWarps * 32, L::SMEM, st>>>(mq, mk, mv, mo, arg);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        arg.slots_out = nullptr;
        arg.slots_in = slots;
    }
    kern<<<(unsigned)grid, kWarps * 32, L::SMEM, st>>>(mq, mk, mv, mo, arg);
    return cudaGetLastError();
}

}  // namespace

// The cost of a cut is counted in chunk times: a CTA (one an SM) takes its
// segment's chunks and about four more to start and end; a first pass over all
// but the last segments takes 0.6 of that, and its launch three.  (B = 1,
// T = 65536, H = 16, 128 x 128: 4 segments a sequence 622 us, 9 322 us.)  Packed
// sequences' lengths are not known here: the longest is taken for four times the
// mean, and the work for evenly spread.
SegPlan linear_tc_plan(int B, int T, int H, int K, int V, bool packed) {
    (void)K;
    (void)V;
    const int nsm = sm_count() > 0 ? sm_count() : 152;
    const long long longest = packed && 4LL * T / B < T ? 4LL * T / B : T;
    auto time = [&](long long items, long long len) {
        const double one = (double)((len + kC - 1) / kC) + 4;
        if (!packed) return one * (double)((items * H + nsm - 1) / nsm);
        const double all = ((double)T / kC + 4.0 * items) * H / nsm;
        return one > all ? one : all;
    };
    SegPlan best{T > 0 ? T : 1, B};
    double least = time(B, longest);
    for (int n = 2; n <= 64 && longest / n >= 2 * kC; ++n) {
        const long long len = (longest + (long long)n * kC - 1) / ((long long)n * kC) * kC;
        const long long per = ((packed ? T : longest) + len - 1) / len;
        const long long items = packed ? per + B : per * B;
        const double cost = time(items, len) * 1.6 + 3;
        if (cost < least) {
            least = cost;
            best = {(int)len, (int)items};
        }
    }
    return best;
}

cudaError_t launch_linear_tc(const LinearScan &a, float *slots, cudaStream_t stream) {
    if (a.K == 128 && a.V == 128) return launch_kv<128, 128>(a, slots, stream);
    if (a.K == 64 && a.V == 128) return launch_kv<64, 128>(a, slots, stream);
    if (a.K == 128 && a.V == 64) return launch_kv<128, 64>(a, slots, stream);
    if (a.K == 64 && a.V == 64) return launch_kv<64, 64>(a, slots, stream);
    return cudaErrorInvalidValue;
}

}  // namespace gdn
