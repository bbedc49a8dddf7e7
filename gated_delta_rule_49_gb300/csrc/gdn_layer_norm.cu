// Layer norm of rows with the sum that runs past a layer, and its gradients:
//
//     s = x + residual,  y = (s - m) r .* w + b
//     n = (s - m) r,  g = w .* dy
//     dx = r (g - mean g - n mean(g n)) + ds,  dw = sum dy .* n,  db = sum dy
//
// Bound by memory: every input read once, every output written once (8 bytes a
// value with the sum, 4 without; gradients 8 or 6, in bf16).  A row is held by a
// group of threads, each with 8 (up to 32) of its channels, so that a thread's
// channels are the same in every row: w, b and the sums for dw and db stay in its
// registers.  The deviation is taken from the mean, not from the squares' sum: a
// row about a large mean keeps it.  A group works on U rows at once: their loads
// are in flight together, the next rows' go out as soon as these are summed, and
// one exchange between the group's warps serves all U.
#include "gdn_vec8.cuh"

namespace gdn {
namespace {

// Threads of a row, pieces of 8 channels of a thread.  Up to 2048 channels a piece
// is all: a group is the next power of two of pieces, and as many groups as fill
// 256 threads are a CTA.
template <int TPR_, int VPT_> struct RowShape {
    static constexpr int TPR = TPR_, VPT = VPT_;
    static constexpr int kThreads = TPR < 256 ? 256 : TPR;
    static constexpr int kGroups = kThreads / TPR;
};
// Rows at once, by what a row takes of a thread's registers.
template <typename T, int VPT> constexpr int rows_at_once(bool back) {
    const int u = (back ? 2 : 4) / (VPT * (int)sizeof(T) / 2);
    return u < 1 ? 1 : u;
}
// CTAs of 256 threads an SM.
constexpr int kNormCtas = 2;
constexpr int resident(int threads) { return kNormCtas * 256 / threads < 1 ? 1 : kNormCtas * 256 / threads; }
// Whether the next rows' loads go out before these are done: their registers.
template <typename T, int VPT> constexpr bool fetch_ahead(bool back) {
    return VPT * (int)sizeof(T) <= (back ? 4 : 8);
}
// Gradients of more than 8192 channels: the sums for dw and db in shared memory.
template <int VPT> constexpr bool sums_shared() { return VPT > 2; }

// Sums of U values over a group of TPR threads, the same in all of them and in a
// fixed order.  Groups of several warps meet at a barrier of their own; the two
// buffers of `red` take turns.
template <int TPR, int U> struct GroupSum {
    static constexpr int kWarps = TPR / 32;
    float (*red)[kWarps > 0 ? kWarps : 1][U];  // [2][warps][U], the group's
    int group, turn;
    __device__ __forceinline__ void operator()(float (&x)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1)
                x[u] += __shfl_xor_sync(0xffffffffu, x[u], off);
        if constexpr (TPR > 32) {
            const int warp = (threadIdx.x % TPR) >> 5;
            if ((threadIdx.x & 31) == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) red[turn][warp][u] = x[u];
            }
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(TPR) : "memory");
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = red[turn][0][u];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] += red[turn][w][u];
            turn ^= 1;
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
};

template <typename T, int VPT>
__device__ __forceinline__ void load_columns(float (&v)[VPT][8], const float *p, float other, int first,
                                             int step, int D) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = first + k * step;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = other;
        if (p && c < D) {
            Vec8<float> q;
            q.load_cached(p + c);
            q.get(v[k]);
        }
    }
}
// Eight values rounded to the type, as held by Vec8.
__device__ __forceinline__ void round8(Vec8<float> &v, const float (&x)[8]) {
    v.a = make_float4(x[0], x[1], x[2], x[3]);
    v.b = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void round8(Vec8<__nv_bfloat16> &v, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    v.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(__nv_bfloat16 *p, const Vec8<__nv_bfloat16> &v) {
    *reinterpret_cast<uint4 *>(p) = v.a;
}
__device__ __forceinline__ void put8(float *p, const Vec8<float> &v) {
    reinterpret_cast<float4 *>(p)[0] = v.a;
    reinterpret_cast<float4 *>(p)[1] = v.b;
}

template <typename T, typename S, bool RES>
__global__ void __launch_bounds__(S::kThreads, resident(S::kThreads))
    layer_norm_kernel(const NormArgs p) {
    constexpr int TPR = S::TPR, VPT = S::VPT, U = rows_at_once<T, VPT>(false);
    constexpr bool kHold = VPT <= 2;  // w and b in registers
    __shared__ float red[S::kGroups][2][TPR >= 32 ? TPR / 32 : 1][U];
    const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, c0 = l * 8;
    GroupSum<TPR, U> sum = {red[group], group, 0};
    const float inv = 1.f / p.D;
    float w[kHold ? VPT : 1][8], b[kHold ? VPT : 1][8];
    if constexpr (kHold) {
        load_columns<T, VPT>(w, p.w, 1.f, c0, TPR * 8, p.D);
        load_columns<T, VPT>(b, p.b, 0.f, c0, TPR * 8, p.D);
    }
    const T *const x = static_cast<const T *>(p.x), *const res = static_cast<const T *>(p.res);
    T *const y = static_cast<T *>(p.y), *const sums = static_cast<T *>(p.s);
    Vec8<T> rx[U][VPT], rr[RES ? U : 1][VPT];
    auto fetch = [&](long long row0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = c0 + k * TPR * 8;
                if (row0 + u < p.N && c < p.D) {
                    rx[u][k].load(x + ((row0 + u) * p.ldx + c));
                    if constexpr (RES) rr[u][k].load(res + ((row0 + u) * p.ldr + c));
                }
            }
    };
    const long long first = ((long long)blockIdx.x * S::kGroups + group) * U;
    const long long step = (long long)gridDim.x * S::kGroups * U;
    // groups of a warp or less go round together: their shuffles name all lanes
    const long long end = TPR < 32 ? p.N + (long long)(group % (32 / (TPR < 32 ? TPR : 32))) * U : p.N;
    constexpr bool kAhead = fetch_ahead<T, VPT>(false);
    if constexpr (kAhead) fetch(first);
    for (long long row0 = first; row0 < end; row0 += step) {
        if constexpr (!kAhead) fetch(row0);
        Vec8<T> sv[U][VPT];
        float m[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float f[8] = {};
                if (row0 + u < p.N && c0 + k * TPR * 8 < p.D) {
                    rx[u][k].get(f);
                    if constexpr (RES) {
                        float r[8];
                        rr[u][k].get(r);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] += r[e];
                    }
                }
                round8(sv[u][k], f);
                if constexpr (RES) sv[u][k].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) m[u] += f[e];
            }
        }
        if constexpr (kAhead) fetch(row0 + step);
        sum(m);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            m[u] *= inv;
            q[u] = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                if (c0 + k * TPR * 8 >= p.D) continue;
                float f[8];
                sv[u][k].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) q[u] = fmaf(f[e] - m[u], f[e] - m[u], q[u]);
            }
        }
        sum(q);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = row0 + u;
            if (row >= p.N) continue;
            const float r = rsqrtf(fmaf(q[u], inv, p.eps));
            if (p.stats && l == 0) *reinterpret_cast<float2 *>(p.stats + 2 * row) = make_float2(m[u], r);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = c0 + k * TPR * 8;
                if (c >= p.D) continue;
                if (RES && sums) put8(sums + (row * p.D + c), sv[u][k]);
                float f[8], wk[1][8], bk[1][8];
                if constexpr (!kHold) {
                    load_columns<T, 1>(wk, p.w, 1.f, c, 0, p.D);
                    load_columns<T, 1>(bk, p.b, 0.f, c, 0, p.D);
                }
                sv[u][k].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    f[e] = fmaf((f[e] - m[u]) * r, kHold ? w[kHold ? k : 0][e] : wk[0][e],
                                kHold ? b[kHold ? k : 0][e] : bk[0][e]);
                Vec8<T>::store(y + (row * p.D + c), f);
            }
        }
    }
}

// A group's rows leave their sums for dw and db in its registers; the CTA's
// groups add theirs up in shared memory, in their order, and the CTA writes one
// row of `parts`.
template <typename T, typename S, bool PAST>
__global__ void __launch_bounds__(S::kThreads, resident(S::kThreads))
    layer_norm_backward_kernel(const NormArgs p) {
    constexpr int TPR = S::TPR, VPT = S::VPT, U = rows_at_once<T, VPT>(true);
    constexpr bool kHold = VPT <= 2;
    __shared__ float red[S::kGroups][2][TPR >= 32 ? TPR / 32 : 1][2 * U];
    extern __shared__ float acc[];  // [groups - 1][2][8][TPR], or [VPT][2][8][TPR]
    const int group = threadIdx.x / TPR, l = threadIdx.x % TPR, c0 = l * 8;
    GroupSum<TPR, 2 * U> sum = {red[group], group, 0};
    const float inv = 1.f / p.D;
    constexpr bool kShared = sums_shared<VPT>();
    float w[kHold ? VPT : 1][8], dw[VPT][8] = {}, db[VPT][8] = {};
    if constexpr (kShared)  // a thread's own channels: no other meets them
        for (int k = 0; k < VPT; ++k)
            for (int e = 0; e < 8; ++e) acc[(k * 16 + e) * TPR + l] = acc[(k * 16 + 8 + e) * TPR + l] = 0.f;
    if constexpr (kHold) load_columns<T, VPT>(w, p.w, 1.f, c0, TPR * 8, p.D);
    const T *const s = static_cast<const T *>(p.x), *const dy = static_cast<const T *>(p.dy);
    const T *const ds = static_cast<const T *>(p.res);
    T *const dx = static_cast<T *>(p.y);
    Vec8<T> rs[U][VPT], rd[U][VPT], rp[PAST ? U : 1][VPT];
    float2 st[U];
    auto fetch = [&](long long row0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = row0 + u;
            if (row >= p.N) continue;
            st[u] = *reinterpret_cast<const float2 *>(p.stats + 2 * row);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = c0 + k * TPR * 8;
                if (c >= p.D) continue;
                rs[u][k].load(s + (row * p.ldx + c));
                rd[u][k].load(dy + (row * p.D + c));
                if constexpr (PAST) rp[u][k].load(ds + (row * p.D + c));
            }
        }
    };
    const long long first = ((long long)blockIdx.x * S::kGroups + group) * U;
    const long long step = (long long)gridDim.x * S::kGroups * U;
    const long long end = TPR < 32 ? p.N + (long long)(group % (32 / (TPR < 32 ? TPR : 32))) * U : p.N;
    constexpr bool kAhead = fetch_ahead<T, VPT>(true);
    if constexpr (kAhead) fetch(first);
    for (long long row0 = first; row0 < end; row0 += step) {
        if constexpr (!kAhead) fetch(row0);
        Vec8<T> ns[U][VPT], nd[U][VPT], np[PAST ? U : 1][VPT];
        float2 nst[U];
        float t[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            nst[u] = st[u];
            t[2 * u] = t[2 * u + 1] = 0.f;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = c0 + k * TPR * 8;
                if (row0 + u >= p.N || c >= p.D) continue;
                ns[u][k] = rs[u][k];
                nd[u][k] = rd[u][k];
                if constexpr (PAST) np[u][k] = rp[u][k];
                float wk[1][8], f[8], d[8];
                if constexpr (!kHold) load_columns<T, 1>(wk, p.w, 1.f, c, 0, p.D);
                ns[u][k].get(f);
                nd[u][k].get(d);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = (f[e] - nst[u].x) * nst[u].y;
                    if constexpr (kShared) {
                        float *const at = acc + (k * 16 + e) * TPR + l;
                        at[0] = fmaf(d[e], n, at[0]);
                        at[8 * TPR] += d[e];
                    } else {
                        dw[k][e] = fmaf(d[e], n, dw[k][e]);
                        db[k][e] += d[e];
                    }
                    const float g = d[e] * (kHold ? w[kHold ? k : 0][e] : wk[0][e]);
                    t[2 * u] += g;
                    t[2 * u + 1] = fmaf(g, n, t[2 * u + 1]);
                }
            }
        }
        if constexpr (kAhead) fetch(row0 + step);
        sum(t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = row0 + u;
            if (row >= p.N) continue;
            const float mg = t[2 * u] * inv, mgn = t[2 * u + 1] * inv;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = c0 + k * TPR * 8;
                if (c >= p.D) continue;
                float wk[1][8], f[8], d[8], z[8] = {};
                if constexpr (!kHold) load_columns<T, 1>(wk, p.w, 1.f, c, 0, p.D);
                ns[u][k].get(f);
                nd[u][k].get(d);
                if constexpr (PAST) np[u][k].get(z);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = (f[e] - nst[u].x) * nst[u].y;
                    const float g = fmaf(d[e], kHold ? w[kHold ? k : 0][e] : wk[0][e], -mg);
                    const float v = fmaf(-n, mgn, g);
                    f[e] = PAST ? fmaf(v, nst[u].y, z[e]) : v * nst[u].y;
                }
                Vec8<T>::store(dx + (row * p.D + c), f);
            }
        }
    }
    if (!p.parts) return;
    constexpr int W = TPR * 8;  // channels of a group's first pieces
    if constexpr (S::kGroups > 1) {
        static_assert(VPT == 1, "several groups have one piece a thread");
        __syncthreads();
        if (group > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[((group - 1) * 2) * W + e * TPR + l] = dw[0][e];
                acc[((group - 1) * 2 + 1) * W + e * TPR + l] = db[0][e];
            }
        }
        __syncthreads();
        if (group > 0) return;
        for (int q = 1; q < S::kGroups; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[0][e] += acc[((q - 1) * 2) * W + e * TPR + l];
                db[0][e] += acc[((q - 1) * 2 + 1) * W + e * TPR + l];
            }
    }
    float *const out = p.parts + (long long)blockIdx.x * 2 * p.D;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = c0 + k * TPR * 8;
        if (c >= p.D) continue;
        if constexpr (kShared)
            for (int e = 0; e < 8; ++e) {
                dw[k][e] = acc[(k * 16 + e) * TPR + l];
                db[k][e] = acc[(k * 16 + 8 + e) * TPR + l];
            }
        Vec8<float>::store(out + c, dw[k]);
        Vec8<float>::store(out + p.D + c, db[k]);
    }
}

// dw and db: the sums of the rows of `parts`, in a fixed order.  32 warps a CTA
// of 32 columns: one warp alone would make a chain of some 300 loads.
__global__ void __launch_bounds__(1024)
    layer_norm_sum_kernel(const float *parts, int n, int D, float *dw, float *db) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
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

// CTAs: no more than fit at once, nor than there are rows.
template <typename T, typename S> int norm_grid(long long N, bool back) {
    const long long rows = (long long)S::kGroups * rows_at_once<T, S::VPT>(back);
    const long long need = (N + rows - 1) / rows;
    const long long most = (long long)resident(S::kThreads) * (sm_count() > 0 ? sm_count() : 152);
    return (int)(need < most ? need : most);
}

// f for the shape of D channels.
template <typename F> auto by_width(int D, F &&f) {
    const int pieces = D / 8;
    if (pieces <= 8) return f(RowShape<8, 1>());
    if (pieces <= 16) return f(RowShape<16, 1>());
    if (pieces <= 32) return f(RowShape<32, 1>());
    if (pieces <= 64) return f(RowShape<64, 1>());
    if (pieces <= 128) return f(RowShape<128, 1>());
    if (pieces <= 256) return f(RowShape<256, 1>());
    if (pieces <= 512) return f(RowShape<256, 2>());
    if (pieces <= 1024) return f(RowShape<512, 2>());
    return f(RowShape<512, 4>());
}

template <typename T> cudaError_t forward(const NormArgs &p, cudaStream_t st) {
    return by_width(p.D, [&](auto shape) {
        using S = decltype(shape);
        const int grid = norm_grid<T, S>(p.N, false);
        if (p.res) layer_norm_kernel<T, S, true><<<grid, S::kThreads, 0, st>>>(p);
        else layer_norm_kernel<T, S, false><<<grid, S::kThreads, 0, st>>>(p);
        return cudaGetLastError();
    });
}

// More shared memory than a launch may have without asking; once a context.
template <typename K> cudaError_t allow_smem(K kern, uintptr_t (&set)[64], size_t bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set[dev] == context_key()) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) set[dev] = context_key();
    return e;
}

template <typename T> cudaError_t backward(const NormArgs &p, float *dw, float *db, cudaStream_t st) {
    return by_width(p.D, [&](auto shape) {
        using S = decltype(shape);
        const int grid = norm_grid<T, S>(p.N, true);
        constexpr int kept = sums_shared<S::VPT>() ? S::VPT : S::kGroups - 1;
        constexpr size_t smem = (size_t)kept * 16 * S::TPR * sizeof(float);
        if constexpr (smem > 48 * 1024) {
            static uintptr_t set[2][64] = {};
            const cudaError_t e = p.res ? allow_smem(layer_norm_backward_kernel<T, S, true>, set[1], smem)
                                        : allow_smem(layer_norm_backward_kernel<T, S, false>, set[0], smem);
            if (e != cudaSuccess) return e;
        }
        if (p.res) layer_norm_backward_kernel<T, S, true><<<grid, S::kThreads, smem, st>>>(p);
        else layer_norm_backward_kernel<T, S, false><<<grid, S::kThreads, smem, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess || !p.parts) return e;
        layer_norm_sum_kernel<<<(2 * p.D + 31) / 32, 1024, 0, st>>>(p.parts, grid, p.D, dw, db);
        return cudaGetLastError();
    });
}

}  // namespace

int layer_norm_parts(long long N, int D) {
    // the larger of the two types' grids
    return by_width(D, [&](auto shape) {
        using S = decltype(shape);
        const int a = norm_grid<__nv_bfloat16, S>(N, true), b = norm_grid<float, S>(N, true);
        return a > b ? a : b;
    });
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

}  // namespace gdn
