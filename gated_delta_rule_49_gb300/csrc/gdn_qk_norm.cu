// Norms of queries and keys for each head with the position rotation in the
// same pass, and its backward pass.
//
// For one head's channels x of one token (D channels, R <= D of them rotated):
//
//     r = (c sum_i x_i^2 + eps)^(-1/2),  c = 1/D (RMS) or 1 (L2)
//     n = w .* x r
//     y = rotate(n): pairs (i, i + R/2) or (2i, 2i + 1), i < R/2, turned by
//         the angle pos * inv_freq[i]; channels >= R pass unchanged
//
// Backward, g = rotate^T(dy) and h = w .* g:
//
//     dw_i = sum over tokens and heads of g_i x_i r
//     dx   = r (h - c r^2 x (x . h))
//
// Bound by memory: x read once and y written once (backward: x and dy read,
// dx written).  A row of D channels is held by D / 16 lanes, two pieces of 8
// channels each, chosen so that a lane holds both channels of its pairs: only
// the sums over a row are exchanged by shuffles.  (With 8 consecutive channels a
// lane the half layout took 8 more shuffles a row, and the angles' reads met 8 a
// bank: 160 us where this takes 90 for B = 8, T = 4096, 16 + 16 heads of
// 128 channels in bf16.)  A thread has the loads of several rows in flight
// before it works on the first.
//
// The angles of a tile of tokens are formed once, in shared memory, and serve
// all of their heads.  Only the fraction of a turn counts, and positions are
// whole: a frequency is kept as inv_freq / 2 pi in 64-bit fixed point, whole
// turns dropped (formed in float64, once a CTA), and the product with the
// position in wrapping integers is that fraction to pos 2^-56 turns.  (In
// float32 an angle of 1e6 has lost 4 of its digits; in float64, at the 2 lanes
// a clock of an SM here, the products took a third of the pass.)
#include "gdn_vec8.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// CTAs of an SM, and rows in flight of a thread.  For B = 8, T = 4096, 16 + 16
// heads of 128 channels in bf16: forward, 2 CTAs of 4 rows 90 us, 3 CTAs 98 (2
// rows: 100), 4 CTAs of 2 rows 98; backward, 2 CTAs of 2 rows 157 us (3 rows: 166,
// 4: 200, spilled), 3 CTAs 160 (1 row) and 227.
constexpr int kNormCtas = 2;
constexpr int norm_rows(bool back, bool wide) { return (back ? 2 : 4) / (wide ? 2 : 1); }

// One of q and k: its rows are taken by CTAs of its own, so that nothing is
// chosen row by row (issue slots are what runs short beside memory).
struct QkSide {
    const void *x, *dy;
    const float *w;
    void *y;             // backward: dx
    long long ld;
    int heads, tokens;   // of a tile
    unsigned magic;      // ceil(2^32 / heads): divides a row of a tile (0: one head)
};
struct QkNormArgs {
    QkSide side[2];
    int first;           // CTAs of q, the rest are k's
    const long long *pos;
    const float *inv_freq;
    float *partial;      // backward: [grid][D]
    long long N;
    int R;
    float eps;
};

template <int LPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// Packed float32 operations: a *= f, b *= g, and a = a f + c, b = b g + d.
__device__ __forceinline__ void mul2(float &a, float &b, float f, float g) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(g));
}
__device__ __forceinline__ void fma2(float &a, float &b, float f, float g, float c, float d) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f), "f"(g), "f"(c), "f"(d));
}
// The two pieces of a lane's channels.
__device__ __forceinline__ float (&lower(float (&x)[16]))[8] { return reinterpret_cast<float(&)[8]>(x[0]); }
__device__ __forceinline__ float (&upper(float (&x)[16]))[8] { return reinterpret_cast<float(&)[8]>(x[8]); }
// sum of x_i y_i
__device__ __forceinline__ float dot16(const float (&x)[16], const float (&y)[16]) {
    float s0 = x[0], s1 = x[1];
    mul2(s0, s1, y[0], y[1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) {
        float a = x[i], b = x[i + 1];
        fma2(a, b, y[i], y[i + 1], s0, s1);
        s0 = a;
        s1 = b;
    }
    return s0 + s1;
}

// First channels of lane c's two pieces: of a half layout's rotated lanes 8 c
// and R/2 + 8 c, else 16 c and 16 c + 8.
template <bool HALF> __device__ __forceinline__ int piece_a(int c, int R) {
    return HALF && 16 * c < R ? 8 * c : 16 * c;
}
template <bool HALF> __device__ __forceinline__ int piece_b(int c, int R) {
    return HALF && 16 * c < R ? (R >> 1) + 8 * c : 16 * c + 8;
}

// The lane's pairs turned by frequencies 8 c .. 8 c + 7 of `cs` (a token's
// angles: cosines, then sines; of each the lanes' first four side by side, then
// their last four); BACK: turned back.
template <bool HALF, bool BACK>
__device__ __forceinline__ void rotate16(float (&x)[16], const float4 *cs, int R, int c) {
    if (16 * c >= R) return;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const float4 u = cs[j * (R >> 4) + c], v = cs[(R >> 3) + j * (R >> 4) + c];
        const float co[4] = {u.x, u.y, u.z, u.w};
        float si[4] = {v.x, v.y, v.z, v.w};
        if constexpr (BACK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) si[i] = -si[i];
        }
        if constexpr (HALF) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const int a = 4 * j + i, b = 8 + a;
                float a0 = x[a], a1 = x[a + 1];
                float t0 = -x[b], t1 = -x[b + 1];
                mul2(t0, t1, si[i], si[i + 1]);
                fma2(x[a], x[a + 1], co[i], co[i + 1], t0, t1);
                mul2(a0, a1, si[i], si[i + 1]);
                fma2(x[b], x[b + 1], co[i], co[i + 1], a0, a1);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[8 * j + 2 * i], b = x[8 * j + 2 * i + 1];
                x[8 * j + 2 * i] = fmaf(a, co[i], -b * si[i]);
                x[8 * j + 2 * i + 1] = fmaf(a, si[i], b * co[i]);
            }
        }
    }
}

// The frequencies in turns, 2^64 a turn; the lowest bit, else 0, says that one
// is not finite.
__device__ __forceinline__ void fill_turns(unsigned long long *turns, const QkNormArgs &p) {
    for (int f = threadIdx.x; f < (p.R >> 1); f += kThreads) {
        double x = (double)p.inv_freq[f] * 0.15915494309189533577;
        x -= floor(x);  // [0, 1), or NaN
        turns[f] = x == x ? (unsigned long long)(x * 9223372036854775808.0) << 1 : 1;
    }
}

// cos and sin of every angle of tokens [t0, t0 + nt).
__device__ __forceinline__ void fill_angles(float *cs, const unsigned long long *turns,
                                            const QkNormArgs &p, long long t0, int nt) {
    const int half = p.R >> 1;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const unsigned long long x = (unsigned long long)p.pos[t0 + t] * turns[f];
        float s, c;
        sincospif((float)(int)(x >> 32) * 0x1p-31f, &s, &c);
        if (turns[f] & 1) s = c = __int_as_float(0x7fffffff);
        const int at = ((f >> 2) & 1) * (half >> 1) + (f >> 3) * 4 + (f & 3);
        cs[2 * t * half + at] = c;
        cs[(2 * t + 1) * half + at] = s;
    }
}

// A CTA takes tiles of some tokens with all heads of q or of k, a lane group of
// D / 16 lanes U rows at a time.
template <typename T, int D, bool HALF, bool BACK>
__global__ void __launch_bounds__(kThreads, kNormCtas)
    qk_norm_kernel(const QkNormArgs p, float c_norm) {
    constexpr int LPR = D / 16;            // lanes of a row
    constexpr int ROWS = kThreads / LPR;   // rows at a time
    constexpr int U = norm_rows(BACK, sizeof(T) == 4);
    extern __shared__ __align__(16) unsigned long long turns[];
    float *const cs2 = reinterpret_cast<float *>(turns + (p.R >> 1));  // two tiles
    const bool isk = (int)blockIdx.x >= p.first;
    const QkSide &sd = p.side[isk];
    const int heads = sd.heads, TT = sd.tokens;
    const unsigned magic = sd.magic;
    const int c = threadIdx.x % LPR, gi = threadIdx.x / LPR;
    const int pa = piece_a<HALF>(c, p.R), pb = piece_b<HALF>(c, p.R);
    const T *const src = static_cast<const T *>(sd.x) + pa, *const gsrc = static_cast<const T *>(sd.dy) + pa;
    T *const dst = static_cast<T *>(sd.y) + pa;
    const int ab = pb - pa;
    const long long ld = sd.ld;
    const int ldy = heads * D;
    float w[16], dw[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        w[i] = sd.w ? sd.w[i < 8 ? pa + i : pb + i - 8] : 1.f;
        dw[i] = 0.f;
    }
    auto token_of = [&](int r) { return magic ? (int)__umulhi((unsigned)r, magic) : r; };
    fill_turns(turns, p);
    __syncthreads();
    const long long tile0 = (long long)(isk ? blockIdx.x - p.first : blockIdx.x) * TT;
    const long long step = (long long)(isk ? gridDim.x - p.first : p.first) * TT;
    Vec8<T> xa[U], xb[U], ga[BACK ? U : 1], gb[BACK ? U : 1];
    // row u of the batch from row r0 of the tile of tokens t0 ..
    auto fetch = [&](int u, long long t0, int r0) {
        const int r = r0 + u * ROWS + gi;
        if (t0 >= p.N || r >= (int)min((long long)TT, p.N - t0) * heads) return;
        const int t = token_of(r), h = r - t * heads;
        const T *x = src + ((t0 + t) * ld + h * D);
        xa[u].load(x);
        xb[u].load(x + ab);
        if constexpr (BACK) {
            x = gsrc + (t0 * ldy + r * D);
            ga[u].load(x);
            gb[u].load(x + ab);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, tile0, 0);
    int buf = 0;
    for (long long t0 = tile0; t0 < p.N; t0 += step) {
        const int nt = (int)min((long long)TT, p.N - t0);
        const int rows = nt * heads;
        float *const cs = cs2 + buf * TT * p.R;
        buf ^= 1;
        fill_angles(cs, turns, p, t0, nt);
        __syncthreads();  // two tiles of angles: the other is not read any more
        for (int r0 = 0; r0 < rows; r0 += U * ROWS) {
            const bool more = r0 + U * ROWS < rows;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * ROWS + gi;
                const bool live = r < rows;
                const int t = live ? token_of(r) : 0;
                float x[16] = {}, g[16] = {};
                if (live) {
                    xa[u].get(lower(x));
                    xb[u].get(upper(x));
                    if constexpr (BACK) {
                        ga[u].get(lower(g));
                        gb[u].get(upper(g));
                    }
                }
                // its place is free: the next batch's row, of the next tile at the end
                fetch(u, more ? t0 : t0 + step, more ? r0 + U * ROWS : 0);
                const float ss = row_sum<LPR>(dot16(x, x));
                // a lane group without a row has no norm: with eps = 0 it would be infinite,
                // and 0 times it would reach the weights' gradient
                const float rn = !BACK || live ? rsqrtf(fmaf(c_norm, ss, p.eps)) : 0.f;
                const float4 *ct = reinterpret_cast<const float4 *>(cs + t * p.R);
                if constexpr (!BACK) {
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        mul2(x[i], x[i + 1], rn, rn);
                        mul2(x[i], x[i + 1], w[i], w[i + 1]);
                    }
                    rotate16<HALF, false>(x, ct, p.R, c);
                } else {
                    rotate16<HALF, true>(g, ct, p.R, c);
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float d0 = x[i], d1 = x[i + 1];
                        mul2(d0, d1, rn, rn);
                        fma2(d0, d1, g[i], g[i + 1], dw[i], dw[i + 1]);
                        dw[i] = d0;
                        dw[i + 1] = d1;
                        mul2(g[i], g[i + 1], w[i], w[i + 1]);
                    }
                    const float f = -row_sum<LPR>(dot16(x, g)) * c_norm * rn * rn;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        fma2(x[i], x[i + 1], f, f, g[i], g[i + 1]);
                        mul2(x[i], x[i + 1], rn, rn);
                    }
                }
                if (live) {
                    T *y = dst + (t0 * ldy + r * D);
                    Vec8<T>::store(y, lower(x));
                    Vec8<T>::store(y + ab, upper(x));
                }
            }
        }
    }
    if constexpr (BACK) {
        if (!p.partial) return;
        // sums over this CTA's rows, in the fixed order of its threads
        float *red = cs2;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) red[gi * D + (i < 8 ? pa + i : pb + i - 8)] = dw[i];
        __syncthreads();
        for (int d = threadIdx.x; d < D; d += kThreads) {
            float s = 0.f;
            for (int r = 0; r < ROWS; ++r) s += red[r * D + d];
            p.partial[(long long)blockIdx.x * D + d] = s;
        }
    }
}

// dw[d] = sum over the CTAs of q (blocks of the first D columns) or of k, in a
// fixed order.  32 warps a CTA: the sums are a chain of loads, which one warp
// alone would make some 200 long.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const float *partial, int first, int n,
                                                          int D, float *dwq, float *dwk) {
    __shared__ float red[32][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool isk = (int)blockIdx.x * 32 >= D;
    const int col = blockIdx.x * 32 + lane - (isk ? D : 0);
    float *dst = isk ? dwk : dwq;
    if (!dst) return;
    float s = 0.f;
#pragma unroll 8
    for (int i = (isk ? first : 0) + w; i < (isk ? n : first); i += 32) s += partial[(long long)i * D + col];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += red[i][lane];
        dst[col] = t;
    }
}

int tile_tokens(int heads, int D) {
    // about 8 rows a lane group: the angles of a tile then cost one sincospi
    // or two a thread next to 8 rows of work (at most 2 x 16 KB of angles)
    const int tokens = heads ? 8 * kThreads / (D / 16) / heads : 1, most = 4096 / D;
    return tokens < 1 ? 1 : (tokens > most ? most : tokens);
}

// CTAs of q and of both: one a tile, and no more than fit, by their rows.
struct NormGrid {
    int first, all;
};
NormGrid norm_grid(long long N, int Hq, int Hk, int D) {
    const long long tq = Hq ? (N + tile_tokens(Hq, D) - 1) / tile_tokens(Hq, D) : 0;
    const long long tk = Hk ? (N + tile_tokens(Hk, D) - 1) / tile_tokens(Hk, D) : 0;
    const long long most = (long long)kNormCtas * (sm_count() > 0 ? sm_count() : 152);
    if (tq + tk <= most) return {(int)tq, (int)(tq + tk)};
    long long q = (most * Hq + (Hq + Hk) / 2) / (Hq + Hk);
    q = Hq && q < 1 ? 1 : Hk && q > most - 1 ? most - 1 : q;
    q = q < tq ? q : tq;
    const long long k = most - q < tk ? most - q : tk;
    return {(int)q, (int)(q + k)};
}

template <typename T, bool HALF, bool BACK>
cudaError_t launch_d(const QkNormArgs &p, int D, float c, int grid, size_t smem, cudaStream_t st) {
    switch (D) {
        case 32: qk_norm_kernel<T, 32, HALF, BACK><<<grid, kThreads, smem, st>>>(p, c); break;
        case 64: qk_norm_kernel<T, 64, HALF, BACK><<<grid, kThreads, smem, st>>>(p, c); break;
        case 128: qk_norm_kernel<T, 128, HALF, BACK><<<grid, kThreads, smem, st>>>(p, c); break;
        case 256: qk_norm_kernel<T, 256, HALF, BACK><<<grid, kThreads, smem, st>>>(p, c); break;
        default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

template <bool BACK>
cudaError_t launch_any(const QkNormArgs &p, int D, float c, bool half, gdn_dtype dt, int grid,
                       cudaStream_t st) {
    const int tokens = p.side[0].tokens > p.side[1].tokens ? p.side[0].tokens : p.side[1].tokens;
    size_t smem = (size_t)2 * tokens * p.R * sizeof(float);
    if (BACK && smem < kThreads * 16 * sizeof(float)) smem = kThreads * 16 * sizeof(float);
    smem += (p.R / 2) * sizeof(unsigned long long);
    if (dt == GDN_BF16)
        return half ? launch_d<__nv_bfloat16, true, BACK>(p, D, c, grid, smem, st)
                    : launch_d<__nv_bfloat16, false, BACK>(p, D, c, grid, smem, st);
    return half ? launch_d<float, true, BACK>(p, D, c, grid, smem, st)
                : launch_d<float, false, BACK>(p, D, c, grid, smem, st);
}

QkSide side(const void *x, const void *dy, const float *w, void *y, long long ld, int heads, int D) {
    return {x, dy, w, y, ld, heads, tile_tokens(heads, D),
            heads <= 1 ? 0 : (unsigned)((0x100000000ull + heads - 1) / heads)};
}

}  // namespace

int qk_norm_backward_grid(long long N, int Hq, int Hk, int D) {
    return norm_grid(N, Hq, Hk, D).all;
}

cudaError_t launch_qk_norm(const void *q, const void *k, const float *wq, const float *wk,
                           const long long *pos, const float *inv_freq, void *yq, void *yk,
                           long long N, int Hq, int Hk, int D, int R, long long ldq, long long ldk,
                           bool l2, bool half, float eps, gdn_dtype dt, cudaStream_t st) {
    const NormGrid g = norm_grid(N, Hq, Hk, D);
    const QkNormArgs p = {{side(q, nullptr, wq, yq, ldq, Hq, D), side(k, nullptr, wk, yk, ldk, Hk, D)},
                          g.first, pos, inv_freq, nullptr, N, R, eps};
    return launch_any<false>(p, D, l2 ? 1.f : 1.f / D, half, dt, g.all, st);
}

cudaError_t launch_qk_norm_backward(const void *q, const void *k, const float *wq,
                                    const float *wk, const long long *pos, const float *inv_freq,
                                    const void *dyq, const void *dyk, void *dq, void *dk,
                                    float *dwq, float *dwk, long long N, int Hq, int Hk, int D,
                                    int R, long long ldq, long long ldk, bool l2, bool half,
                                    float eps, gdn_dtype dt, float *partial, cudaStream_t st) {
    const bool want = dwq || dwk;
    const NormGrid g = norm_grid(N, Hq, Hk, D);
    const QkNormArgs p = {{side(q, dyq, wq, dq, ldq, Hq, D), side(k, dyk, wk, dk, ldk, Hk, D)},
                          g.first, pos, inv_freq, want ? partial : nullptr, N, R, eps};
    const cudaError_t e = launch_any<true>(p, D, l2 ? 1.f : 1.f / D, half, dt, g.all, st);
    if (e != cudaSuccess || !want) return e;
    qk_norm_dw_kernel<<<2 * D / 32, 1024, 0, st>>>(partial, g.first, g.all, D, dwq, dwk);
    return cudaGetLastError();
}

}  // namespace gdn
