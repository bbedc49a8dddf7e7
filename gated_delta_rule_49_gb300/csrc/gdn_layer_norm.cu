// Layer norm of rows with the sum that runs past a layer, and its gradients:
//
//     s = x + residual,  y = (s - m) r .* w + b
//     n = (s - m) r,  g = w .* dy
//     dx = r (g - mean g - n mean(g n)) + ds,  dw = sum dy .* n,  db = sum dy
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Sum over the CTA, in a fixed order; every thread has it.
__device__ __forceinline__ float cta_sum(float x) {
    __shared__ float red[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    return s;
}

// One CTA a row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_kernel(const T *x, const T *res, const float *w, const float *b, T *y, T *s,
                      float *stats, int D, long long ldx, long long ldr, float eps) {
    extern __shared__ float row[];
    const long long n = blockIdx.x;
    float sum = 0.f;
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float v = to_f32(x[n * ldx + i]);
        if (res) v = to_f32(from_f32<T>(v + to_f32(res[n * ldr + i])));
        row[i] = v;
        sum += v;
    }
    const float m = cta_sum(sum) / D;
    float sq = 0.f;
    for (int i = threadIdx.x; i < D; i += kThreads) sq += (row[i] - m) * (row[i] - m);
    const float r = rsqrtf(cta_sum(sq) / D + eps);
    if (stats && threadIdx.x == 0) {
        stats[2 * n] = m;
        stats[2 * n + 1] = r;
    }
    for (int i = threadIdx.x; i < D; i += kThreads) {
        if (s) s[n * D + i] = from_f32<T>(row[i]);
        y[n * D + i] = from_f32<T>(fmaf((row[i] - m) * r, w ? w[i] : 1.f, b ? b[i] : 0.f));
    }
}

// A CTA takes every gridDim.x-th row.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_backward_kernel(const T *s, const T *dy, const float *stats, const float *w,
                               const T *ds, T *dx, float *parts, long long N, int D, long long lds) {
    extern __shared__ float acc[];  // dw, db
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) acc[i] = 0.f;
    for (long long row = blockIdx.x; row < N; row += gridDim.x) {
        const float m = stats[2 * row], r = stats[2 * row + 1];
        float sg = 0.f, sgn = 0.f;
        for (int i = threadIdx.x; i < D; i += kThreads) {
            const float n = (to_f32(s[row * lds + i]) - m) * r, d = to_f32(dy[row * D + i]);
            const float g = w ? d * w[i] : d;
            sg += g;
            sgn += g * n;
            acc[i] += d * n;
            acc[D + i] += d;
        }
        sg = cta_sum(sg) / D;
        sgn = cta_sum(sgn) / D;
        for (int i = threadIdx.x; i < D; i += kThreads) {
            const float n = (to_f32(s[row * lds + i]) - m) * r, d = to_f32(dy[row * D + i]);
            float v = r * ((w ? d * w[i] : d) - sg - n * sgn);
            if (ds) v += to_f32(ds[row * D + i]);
            dx[row * D + i] = from_f32<T>(v);
        }
    }
    if (!parts) return;
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) parts[(long long)blockIdx.x * 2 * D + i] = acc[i];
}

__global__ void __launch_bounds__(kThreads)
    layer_norm_sum_kernel(const float *parts, int n, int D, float *dw, float *db) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= 2 * D) return;
    float *const dst = i < D ? dw : db;
    if (!dst) return;
    float s = 0.f;
    for (int k = 0; k < n; ++k) s += parts[(long long)k * 2 * D + i];
    dst[i < D ? i : i - D] = s;
}

// The CTAs' shared memory passes what a launch may have without asking; once a context.
template <typename K> cudaError_t allow_smem(K kern, uintptr_t (&set)[64], int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (set[dev] == context_key()) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) set[dev] = context_key();
    return e;
}

template <typename T>
cudaError_t forward(const void *x, const void *res, const float *w, const float *b, void *y, void *s,
                    float *stats, long long N, int D, long long ldx, long long ldr, float eps,
                    cudaStream_t st) {
    static uintptr_t set[64] = {};
    const cudaError_t e = allow_smem(layer_norm_kernel<T>, set, 16384 * 4);
    if (e != cudaSuccess) return e;
    if (N > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    layer_norm_kernel<T><<<(unsigned)N, kThreads, D * 4, st>>>(
        static_cast<const T *>(x), static_cast<const T *>(res), w, b, static_cast<T *>(y),
        static_cast<T *>(s), stats, D, ldx, ldr, eps);
    return cudaGetLastError();
}

template <typename T>
cudaError_t backward(const void *s, const void *dy, const float *stats, const float *w,
                     const void *ds, void *dx, float *parts, long long N, int D, long long lds,
                     cudaStream_t st) {
    static uintptr_t set[64] = {};
    const cudaError_t e = allow_smem(layer_norm_backward_kernel<T>, set, 16384 * 8);
    if (e != cudaSuccess) return e;
    layer_norm_backward_kernel<T><<<layer_norm_parts(N, D), kThreads, D * 8, st>>>(
        static_cast<const T *>(s), static_cast<const T *>(dy), stats, w, static_cast<const T *>(ds),
        static_cast<T *>(dx), parts, N, D, lds);
    return cudaGetLastError();
}

}  // namespace

int layer_norm_parts(long long N, int D) {
    (void)D;
    const long long most = 2LL * (sm_count() > 0 ? sm_count() : 152);
    return (int)(N < most ? N : most);
}

cudaError_t launch_layer_norm(const void *x, const void *res, const float *w, const float *b,
                              void *y, void *s, float *stats, long long N, int D, long long ldx,
                              long long ldr, float eps, gdn_dtype dt, cudaStream_t st) {
    return dt == GDN_BF16
               ? forward<__nv_bfloat16>(x, res, w, b, y, s, stats, N, D, ldx, ldr, eps, st)
               : forward<float>(x, res, w, b, y, s, stats, N, D, ldx, ldr, eps, st);
}

cudaError_t launch_layer_norm_backward(const void *s, const void *dy, const float *stats,
                                       const float *w, const void *ds, void *dx, float *dw,
                                       float *db, long long N, int D, long long lds, gdn_dtype dt,
                                       float *parts, cudaStream_t st) {
    if (!dw && !db) parts = nullptr;
    const cudaError_t e = dt == GDN_BF16 ? backward<__nv_bfloat16>(s, dy, stats, w, ds, dx, parts, N, D, lds, st)
                                         : backward<float>(s, dy, stats, w, ds, dx, parts, N, D, lds, st);
    if (e != cudaSuccess || !parts) return e;
    layer_norm_sum_kernel<<<(2 * D + kThreads - 1) / kThreads, kThreads, 0, st>>>(
        parts, layer_norm_parts(N, D), D, dw, db);
    return cudaGetLastError();
}

}  // namespace gdn
