// The gated linear recurrence, channel by channel:
//
//     h_t = a_t h_{t-1} + b_t x_t
//
// with a given and b = 1, or a = 1 / (1 + exp(-g)) and b = 1 - a, and its
// gradients
//
//     G_t = dh_t + a_{t+1} G_{t+1},  dx = b G,  da = G (h_{t-1} - [sigmoid] x),
//     dg = da a b,  dh0 = a_1 G_1
#include "gdn_vec8.cuh"
#include "gdn_linear_item.cuh"

namespace gdn {
namespace {

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

template <typename T, bool SIG> struct GateType { using type = T; };
template <typename T> struct GateType<T, false> { using type = float; };

// One thread a sequence and channel.
template <typename T, bool SIG>
__global__ void scan_kernel(const ScanArgs p, int *status) {
    using G = typename GateType<T, SIG>::type;
    const int seq = blockIdx.x, c = blockIdx.y * blockDim.x + threadIdx.x;
    const LinearItem it = linear_item(p.offsets, p.B, p.T, p.T, seq, blockIdx.y == 0 ? status : nullptr);
    if (c >= p.D || it.seq < 0) return;
    const long long at = (long long)seq * p.D + c;
    float h = p.h0 ? p.h0[at] : 0.f;
    const int blocks = (p.T + kScanBlock - 1) / kScanBlock;
    for (int i = 0; i < it.len; ++i) {
        const int t = it.base + i;  // packed: of all tokens
        const long long tok = it.first + i;
        if (p.states && t % kScanBlock == 0)
            p.states[((p.offsets ? 0 : (long long)seq * blocks) + t / kScanBlock) * p.D + c] = h;
        float a, b;
        gate_ab<SIG>(to_f32(static_cast<const G *>(p.gate)[tok * p.ldg + c]), a, b);
        h = fmaf(a, h, b * to_f32(static_cast<const T *>(p.x)[tok * p.ldx + c]));
        if (p.h) static_cast<T *>(p.h)[tok * p.D + c] = from_f32<T>(h);
    }
    if (p.h_T) p.h_T[at] = h;
}

template <typename T, bool SIG>
__global__ void scan_backward_kernel(const ScanArgs p, int *status) {
    using G = typename GateType<T, SIG>::type;
    const int seq = blockIdx.x, c = blockIdx.y * blockDim.x + threadIdx.x;
    const LinearItem it = linear_item(p.offsets, p.B, p.T, p.T, seq, blockIdx.y == 0 ? status : nullptr);
    if (c >= p.D || it.seq < 0) return;
    const long long at = (long long)seq * p.D + c;
    float u = p.dh_T ? p.dh_T[at] : 0.f;
    const int blocks = (p.T + kScanBlock - 1) / kScanBlock;
    const int t0 = it.base, t1 = it.base + it.len;
    const long long shift = it.first - it.base;
    float past[kScanBlock];
    for (int blk = (t1 - 1) / kScanBlock; it.len && blk >= t0 / kScanBlock; --blk) {
        const int lo = max(t0, blk * kScanBlock), hi = min(t1, (blk + 1) * kScanBlock);
        float h = lo == t0 ? (p.h0 ? p.h0[at] : 0.f)
                           : p.states[((p.offsets ? 0 : (long long)seq * blocks) + blk) * p.D + c];
        for (int t = lo; t < hi; ++t) {
            const long long tok = shift + t;
            float a, b;
            gate_ab<SIG>(to_f32(static_cast<const G *>(p.gate)[tok * p.ldg + c]), a, b);
            past[t - lo] = h;
            h = fmaf(a, h, b * to_f32(static_cast<const T *>(p.x)[tok * p.ldx + c]));
        }
        for (int t = hi - 1; t >= lo; --t) {
            const long long tok = shift + t;
            float a, b;
            gate_ab<SIG>(to_f32(static_cast<const G *>(p.gate)[tok * p.ldg + c]), a, b);
            const float x = to_f32(static_cast<const T *>(p.x)[tok * p.ldx + c]);
            const float g = to_f32(static_cast<const T *>(p.dh)[tok * p.D + c]) + u;
            static_cast<T *>(p.dx)[tok * p.D + c] = from_f32<T>(b * g);
            const float da = SIG ? g * (past[t - lo] - x) * a * b : g * past[t - lo];
            static_cast<G *>(p.dgate)[tok * p.D + c] = from_f32<G>(da);
            u = a * g;
        }
    }
    if (p.dh0) p.dh0[at] = u;
}

// One token: a thread takes eight channels, all of its loads before any arithmetic.
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
    float xs[8], gs[8], s[8];
    xv.load(x + row * ldx + c);
    gv.load(gate + row * ldg + c);
    const float4 lo = *reinterpret_cast<const float4 *>(h + i * 8);
    const float4 hi = *reinterpret_cast<const float4 *>(h + i * 8 + 4);
    pdl_trigger();
    s[0] = lo.x; s[1] = lo.y; s[2] = lo.z; s[3] = lo.w;
    s[4] = hi.x; s[5] = hi.y; s[6] = hi.z; s[7] = hi.w;
    xv.get(xs);
    gv.get(gs);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float a, b;
        gate_ab<SIG>(gs[e], a, b);
        s[e] = fmaf(a, s[e], b * xs[e]);
    }
    Vec8<float>::store(h_out + i * 8, s);
    if (y) Vec8<T>::store(y + i * 8, s);
}

template <typename F> cudaError_t by_type(gdn_dtype dt, bool sigmoid, F &&f) {
    if (dt == GDN_BF16) {
        if (sigmoid) f.template operator()<__nv_bfloat16, true>();
        else f.template operator()<__nv_bfloat16, false>();
    } else {
        if (sigmoid) f.template operator()<float, true>();
        else f.template operator()<float, false>();
    }
    return cudaGetLastError();
}

}  // namespace

size_t scan_map_bytes(int T) { return ((size_t)T * sizeof(int) + 255) & ~size_t(255); }

namespace {
struct Forward {
    const ScanArgs &a;
    cudaStream_t st;
    template <typename T, bool SIG> void operator()() {
        scan_kernel<T, SIG><<<dim3(a.B, (a.D + 63) / 64), 64, 0, st>>>(a, device_status_ptr());
    }
};
struct Backward {
    const ScanArgs &a;
    cudaStream_t st;
    template <typename T, bool SIG> void operator()() {
        scan_backward_kernel<T, SIG><<<dim3(a.B, (a.D + 63) / 64), 64, 0, st>>>(a, device_status_ptr());
    }
};
struct Step {
    const void *x, *gate;
    const float *h;
    float *h_out;
    void *y;
    int B, D;
    long long ldx, ldg;
    cudaStream_t st;
    cudaError_t e = cudaSuccess;
    template <typename T, bool SIG> void operator()() {
        const long long pieces = (long long)B * (D / 8);
        const long long grid = (pieces + kStepThreads - 1) / kStepThreads;
        using G = typename GateType<T, SIG>::type;
        e = grid > 0x7fffffffLL ? cudaErrorInvalidConfiguration
                                : launch_pdl(scan_step_kernel<T, SIG>, (unsigned)grid, kStepThreads, 0,
                                             st, static_cast<const T *>(x), static_cast<const G *>(gate),
                                             h, h_out, static_cast<T *>(y), pieces, D / 8, ldx, ldg);
    }
};
}  // namespace

cudaError_t launch_scan(const ScanArgs &a, gdn_dtype dt, void *workspace, cudaStream_t st) {
    (void)workspace;
    return by_type(dt, a.sigmoid, Forward{a, st});
}

cudaError_t launch_scan_backward(const ScanArgs &a, gdn_dtype dt, void *workspace,
                                 cudaStream_t st) {
    ScanArgs b = a;
    if (!b.states) {
        b.states = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                             (a.offsets ? scan_map_bytes(a.T) : 0));
        const cudaError_t e = by_type(dt, b.sigmoid, Forward{b, st});
        if (e != cudaSuccess) return e;
    }
    return by_type(dt, b.sigmoid, Backward{b, st});
}

cudaError_t launch_scan_step(const void *x, const void *gate, const float *h, float *h_out, void *y,
                             int B, int D, long long ldx, long long ldg, bool sigmoid, gdn_dtype dt,
                             cudaStream_t st) {
    Step f{x, gate, h, h_out, y, B, D, ldx, ldg, st};
    const cudaError_t e = by_type(dt, sigmoid, f);
    return f.e != cudaSuccess ? f.e : e;
}

}  // namespace gdn
