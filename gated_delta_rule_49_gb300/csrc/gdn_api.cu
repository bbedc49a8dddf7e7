// C ABI of libgdn.so: host-side validation and dispatch (declared in gdn.h).
#include <cstring>
#include <mutex>

#include <cuda.h>

#include "gdn_internal.cuh"

namespace gdn {

// Per-device status word.  Kernels OR kStatus* bits into it; the host reads
// and clears it in gdn_get_last_device_status.
static __device__ int g_device_status;

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_mu;
int *g_status_ptr[kMaxDevices];
uintptr_t g_status_ctx[kMaxDevices];  // the context g_status_ptr was looked up in
int g_sm_count[kMaxDevices];

int current_device() {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return -1;
    return dev;
}
}  // namespace

uintptr_t context_key() {
    // the driver entry point is fetched through the runtime, so the library
    // keeps no link-time dependency on libcuda (it loads on machines without
    // a driver; nothing here runs there)
    using GetCurrent = CUresult (*)(CUcontext *);
    static GetCurrent fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<GetCurrent>(p);
    }();
    CUcontext ctx = nullptr;
    if (!fn || fn(&ctx) != CUDA_SUCCESS) return 0;
    return reinterpret_cast<uintptr_t>(ctx);
}

int *device_status_ptr() {
    const int dev = current_device();
    if (dev < 0) return nullptr;
    std::lock_guard<std::mutex> lock(g_mu);
    const uintptr_t ctx = context_key();
    if (!g_status_ptr[dev] || ctx == 0 || g_status_ctx[dev] != ctx) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_device_status) != cudaSuccess) return nullptr;
        g_status_ptr[dev] = static_cast<int *>(p);
        g_status_ctx[dev] = context_key();  // current now that the lookup ran
    }
    return g_status_ptr[dev];
}

int sm_count() {
    const int dev = current_device();
    if (dev < 0) return 0;
    std::lock_guard<std::mutex> lock(g_mu);
    if (!g_sm_count[dev]) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
            return 0;
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

}  // namespace gdn

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool supported_kv(int K, int V) {
    return (K == 32 && V == 32) || (K == 64 && V == 128) || (K == 128 && V == 128);
}

int from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return GDN_OK;
    if (e == cudaErrorInvalidValue) return GDN_ERR_INVALID_ARG;
    return GDN_ERR_CUDA;
}

// The argument checks that the norm's forward and backward pass share.
int check_qk_norm(const void *q, const void *k, const float *wq, const float *wk,
                  const long long *pos, const float *inv_freq, long long N, int Hq, int Hk, int D,
                  int R, long long q_stride, long long k_stride, int norm, int pairing, float eps,
                  int dtype) {
    if (N < 0 || Hq < 0 || Hk < 0 || Hq > 16384 || Hk > 16384 || N > (1LL << 40))
        return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (norm != GDN_NORM_RMS && norm != GDN_NORM_L2) return GDN_ERR_INVALID_ARG;
    if (pairing != GDN_PAIR_HALF && pairing != GDN_PAIR_ADJACENT) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (D != 32 && D != 64 && D != 128 && D != 256) return GDN_ERR_UNSUPPORTED;
    if (R < 0 || R > D) return GDN_ERR_INVALID_ARG;
    if (R % 16) return GDN_ERR_UNSUPPORTED;
    const int unit = dtype == GDN_BF16 ? 8 : 4;  // elements of 16 bytes
    if ((Hq && (q_stride < (long long)Hq * D || q_stride % unit)) ||
        (Hk && (k_stride < (long long)Hk * D || k_stride % unit)))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, wq, wk, pos, inv_freq};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (N && ((Hq && !q) || (Hk && !k) || (R && Hq + Hk && (!pos || !inv_freq))))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

bool linear_kv(int K, int V) { return supported_kv(K, V) || (K == 64 && V == 64); }

// The checks of sizes that the linear attention calls share.
int check_linear(int B, int T, int Hq, int H, int K, int V, long long q_stride, long long k_stride,
                 long long v_stride, int dtype) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!linear_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (H && (Hq < 1 || H % Hq)) return GDN_ERR_INVALID_ARG;
    const int unit = dtype == GDN_BF16 ? 8 : 4;  // elements of 16 bytes
    if (H && (q_stride < (long long)Hq * K || k_stride < (long long)Hq * K ||
              v_stride < (long long)H * V || q_stride % unit || k_stride % unit || v_stride % unit))
        return GDN_ERR_INVALID_ARG;
    if ((long long)B * H > (1 << 24) || (long long)B * T > (1LL << 40)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

// The checks that the recurrence's calls share.
int check_scan(const void *x, const void *gate, int B, int T, int D, bool packed,
               long long x_stride, long long gate_stride, int kind, int dtype) {
    if (B < 0 || T < 0 || D < 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (kind != GDN_SCAN_DECAY && kind != GDN_SCAN_SIGMOID) return GDN_ERR_INVALID_ARG;
    if (D % 8) return GDN_ERR_UNSUPPORTED;
    const int unit = dtype == GDN_BF16 ? 8 : 4;  // elements of 16 bytes
    const int gate_unit = kind == GDN_SCAN_DECAY ? 4 : unit;
    // the strides' bound is a tensor map's
    if (x_stride < D || gate_stride < D || x_stride % unit || gate_stride % gate_unit ||
        x_stride > (1LL << 36) || gate_stride > (1LL << 36))
        return GDN_ERR_INVALID_ARG;
    // tokens and channels are 32-bit coordinates of a tile, rounded up to whole tiles
    const long long most = (1LL << 31) - 1024;
    if ((packed ? T : (long long)B * T) > most || B > most || D > most ||
        (long long)B * D > (1LL << 36))
        return GDN_ERR_INVALID_ARG;
    return aligned16(x) && aligned16(gate) ? GDN_OK : GDN_ERR_ALIGNMENT;
}

// Memory of a call: `rows` rows of `width` bytes, `pitch` bytes apart.  in_place: an output
// that may take the place of an input, or an input whose place may be taken.
struct Span {
    const void *p;
    long long rows, width, pitch;
    bool in_place;
};
// n * size bytes in one piece.
Span dense(const void *p, long long n, long long size, bool in_place = false) {
    const long long most = 1LL << 60;  // no tensor is larger
    const long long bytes = n > most / size ? most : n * size;
    return {p, 1, bytes, bytes, in_place};
}
// Rows of D elements of `size` bytes, `stride` elements apart.
Span strided(const void *p, long long rows, int D, long long stride, long long size,
             bool in_place = false) {
    const long long most = 1LL << 56;  // further than any two rows lie
    return {p, rows, D * size, (stride < most ? stride : most) * size, in_place};
}
// Whether `out`, which is dense, and x share a byte.
bool meet(const Span &out, const Span &x) {
    if (!out.p || !x.p || out.width <= 0 || x.width <= 0 || x.rows <= 0) return false;
    const long long lo =
        (long long)(reinterpret_cast<uintptr_t>(out.p) - reinterpret_cast<uintptr_t>(x.p));
    // the first row of x that ends behind the start of out
    const long long k = lo < x.width ? 0 : (lo - x.width) / x.pitch + 1;
    return k < x.rows && k * x.pitch < lo + out.width;
}
// Whether an output lies over an input or over another output.
template <int M, int N> bool clash(const Span (&outs)[M], const Span (&ins)[N]) {
    for (int i = 0; i < M; ++i) {
        for (const Span &x : ins)
            if (meet(outs[i], x) && !(outs[i].in_place && x.in_place && outs[i].p == x.p)) return true;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return true;
    }
    return false;
}

// The states before every 64th token, and their bytes rounded up.
long long scan_states(int B, int T, bool packed) {
    return (packed ? 1LL : B) * (((long long)T + gdn::kScanBlock - 1) / gdn::kScanBlock);
}
size_t scan_states_bytes(int B, int T, int D, bool packed) {
    return ((size_t)scan_states(B, T, packed) * D * sizeof(float) + 255) & ~size_t(255);
}
// Bytes of an element of x (h, y, dh, dx) and of the gates.
struct ScanSizes {
    long long x, gate;
    ScanSizes(int kind, int dtype)
        : x(dtype == GDN_BF16 ? 2 : 4), gate(kind == GDN_SCAN_DECAY ? 4 : x) {}
};

int check_layer_norm(long long N, int D, int dtype) {
    if (N < 0 || N > (1LL << 40) || D < 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    return D % 8 || D > 16384 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace

extern "C" {

int gdn_version(void) { return 100; }

const char *gdn_status_string(int status) {
    switch (status) {
        case GDN_OK: return "ok";
        case GDN_ERR_INVALID_ARG: return "invalid argument";
        case GDN_ERR_UNSUPPORTED: return "unsupported (K, V) variant or device";
        case GDN_ERR_ALIGNMENT: return "pointer not 16-byte aligned";
        case GDN_ERR_CUDA: return "CUDA runtime or launch error";
        case GDN_ERR_TIMEOUT: return "device wait timed out";
        case GDN_ERR_WORKSPACE: return "workspace missing or too small";
        case GDN_ERR_DEVICE_BOUNDS: return "device-side index check failed";
        case GDN_WARN_ZERO_STATE: return "warning: all-zero state (stable rank undefined, 0 returned)";
        case GDN_WARN_NOT_CONVERGED: return "warning: Jacobi sweeps stopped at max_sweeps before convergence";
        case GDN_WARN_RANK_DEFICIENT: return "warning: calibration matrix has rank < k (greedy choice kept, no swaps)";
        default: return "unknown status";
    }
}

size_t gdn_prefill_workspace_size(int B, int T, int H, int K, int V, gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || V != 128 || (K != 128 && K != 64) || dtype != GDN_BF16)
        return 0;
    if ((long long)B * H > 0x7fffffffLL) return 0;
    return gdn::segment_shape(B * H, T, K, gdn::sm_count()).workspace_bytes;
}

size_t gdn_prefill_two_pass_workspace_size(int B, int T, int H, int K, int V, gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || V != 128 || (K != 128 && K != 64) || dtype != GDN_BF16)
        return 0;
    if ((long long)B * H > 0x7fffffffLL) return 0;
    const gdn::SegShape sh = gdn::segment_shape(B * H, T, K, gdn::sm_count());
    return gdn::prefill_prep_offset(sh) + gdn::prefill_prep_bytes((long long)B * H, T) +
           gdn::prefill_x_bytes(sh, (long long)B * H, T);
}

namespace {
// T = 0: the final state is the start state (or zero).
int empty_prefill(const float *S0, float *S_T, int B, int H, int K, int V, cudaStream_t st) {
    if (!S_T) return GDN_OK;
    const size_t bytes = sizeof(float) * (size_t)B * H * V * K;
    cudaError_t e = S0 ? (S0 == S_T ? cudaSuccess
                                    : cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, st))
                       : cudaMemsetAsync(S_T, 0, bytes, st);
    return from_cuda(e);
}

// Which gate arrays a gate needs (non-NULL) and forbids (NULL).
bool gates_match(gdn_gate gate, const float *beta, const float *b, const float *w) {
    if (gate == GDN_GATE_GDN2) return !beta && b && w;
    return beta && !b && !w;
}
bool valid_gate(int gate) {
    return gate == GDN_GATE_SCALAR || gate == GDN_GATE_KDA || gate == GDN_GATE_GDN2;
}
}  // namespace

int gdn_prefill(const void *q, const void *k, const void *v, const float *alpha,
                const float *beta, const float *S0, void *o, float *S_T, int B, int T, int H,
                int K, int V, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !alpha || !beta)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, S0, o, S_T};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    const size_t need = gdn_prefill_workspace_size(B, T, H, K, V, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if ((long long)B * H == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    // bf16 at V = 128 runs on the tensor cores; float32 mode and the small
    // (32, 32) variant run the token-by-token CUDA-core kernel (scalar gate).
    if (dtype == GDN_BF16 && V == 128 && (K == 128 || K == 64))
        return from_cuda(gdn::launch_prefill_tc(q, k, v, alpha, beta, S0, o, S_T, B, T, T, H, K, V,
                                                workspace, workspace_bytes, st));
    return from_cuda(gdn::launch_prefill_gated(q, k, v, alpha, beta, nullptr, nullptr, S0, o, S_T,
                                               B, T, T, H, K, V, GDN_GATE_SCALAR, dtype, st));
}

size_t gdn_prefill_gathered_workspace_size(int B, int T, int H, int K_in, int K, int V,
                                           gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || K_in != 128 || K != 64 || V != 128 || dtype != GDN_BF16)
        return 0;
    if ((long long)B * H > 0x7fffffffLL) return 0;
    return gdn::gathered_layout(B, T, H).total;
}

int gdn_prefill_gathered(const void *q_full, const void *k_full, const int *idx, int K_in,
                         const void *v, const float *alpha, const float *beta, const float *S0,
                         void *o, float *S_T, int B, int T, int H, int K, int V, gdn_dtype dtype,
                         void *workspace, size_t workspace_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0 || K_in <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 || K_in != 128 || K != 64 || V != 128) return GDN_ERR_UNSUPPORTED;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q_full || !k_full || !idx || !v || !alpha || !beta)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q_full, k_full, idx, v, alpha, beta, S0, o, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    if ((long long)B * H == 0) return GDN_OK;
    if ((long long)B * H > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    const size_t need = gdn_prefill_gathered_workspace_size(B, T, H, K_in, K, V, dtype);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    return from_cuda(gdn::launch_prefill_gathered(q_full, k_full, idx, v, alpha, beta, S0, o, S_T,
                                                  B, T, H, workspace, workspace_bytes, st));
}

int gdn_decode_step(const void *q, const void *k, const void *v, const float *alpha,
                    const float *beta, float *S, void *o, int B, int H, int K, int V,
                    gdn_dtype dtype, void *stream) {
    if (B < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * H == 0) return GDN_OK;
    if (!q || !k || !v || !alpha || !beta || !S || !o) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, S, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_decode(q, k, v, alpha, beta, S, o, B, H, K, V, dtype,
                                        static_cast<cudaStream_t>(stream)));
}

int gdn_gather_normalize(const void *x, const int *idx, void *y, long long N, int H, int K_in,
                         int K_out, gdn_dtype dtype, void *stream) {
    if (N < 0 || H < 1 || (K_out != 32 && K_out != 64) || K_in < K_out || K_in > 1024)
        return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (N == 0) return GDN_OK;
    if (!x || !idx || !y) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, idx, y};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (N > (1LL << 40) / H) return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_gather_normalize(x, idx, y, N * H, H, K_in, K_out, dtype, 1e-12f,
                                                  static_cast<cudaStream_t>(stream)));
}

int gdn_decode_step_gathered(const void *q_full, const void *k_full, const int *idx, int K_in,
                             const void *v, const float *alpha, const float *beta, float *S,
                             void *o, int B, int H, int K, int V, gdn_dtype dtype, void *stream) {
    if (B < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (K_in < K || K_in > 1024) return GDN_ERR_INVALID_ARG;
    if ((long long)B * H == 0) return GDN_OK;
    if (!q_full || !k_full || !idx || !v || !alpha || !beta || !S || !o) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q_full, k_full, idx, v, alpha, beta, S, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_decode_gathered(q_full, k_full, idx, K_in, v, alpha, beta, S, o,
                                                 B, H, K, V, dtype, 1e-12f,
                                                 static_cast<cudaStream_t>(stream)));
}

int gdn_prefill_gated(const void *q, const void *k, const void *v, const float *alpha,
                      const float *beta, const float *b, const float *w, const float *S0,
                      void *o, float *S_T, int B, int T, int H, int K, int V, gdn_gate gate,
                      gdn_dtype dtype, void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!valid_gate(gate)) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !alpha || !gates_match(gate, beta, b, w)))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, b, w, S0, o, S_T};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    if ((long long)B * H == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    return from_cuda(gdn::launch_prefill_gated(q, k, v, alpha, beta, b, w, S0, o, S_T, B, T, T,
                                               H, K, V, gate, dtype, st));
}

size_t gdn_prefill_gated_chunked_workspace_size(int B, int T, int H, int K, int V,
                                                gdn_gate gate, gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || K != 128 || V != 128 || dtype != GDN_BF16) return 0;
    if (gate != GDN_GATE_KDA && gate != GDN_GATE_GDN2) return 0;
    if ((long long)B * H > 0x7fffffffLL) return 0;
    return gdn::prefill_gated_tc_workspace(B, T, H, gate);
}

int gdn_prefill_gated_chunked(const void *q, const void *k, const void *v, const float *alpha,
                              const float *beta, const float *b, const float *w, const float *S0,
                              void *o, float *S_T, int B, int T, int H, int K, int V,
                              gdn_gate gate, gdn_dtype dtype, void *workspace,
                              size_t workspace_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!valid_gate(gate)) return GDN_ERR_INVALID_ARG;
    if (gate == GDN_GATE_SCALAR || dtype != GDN_BF16 || K != 128 || V != 128)
        return GDN_ERR_UNSUPPORTED;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !alpha || !gates_match(gate, beta, b, w)))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, b, w, S0, o, S_T, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    if ((long long)B * H == 0) return GDN_OK;
    if ((long long)B * H > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    const size_t need = gdn_prefill_gated_chunked_workspace_size(B, T, H, K, V, gate, dtype);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    return from_cuda(gdn::launch_prefill_gated_tc(q, k, v, alpha, beta, b, w, S0, o, S_T, B, T, H,
                                                  gate, workspace, st));
}

int gdn_decode_step_gated(const void *q, const void *k, const void *v, const float *alpha,
                          const float *beta, const float *b, const float *w, float *S, void *o,
                          int B, int H, int K, int V, gdn_gate gate, gdn_dtype dtype,
                          void *stream) {
    if (B < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!valid_gate(gate)) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if ((long long)B * H == 0) return GDN_OK;
    if (!q || !k || !v || !alpha || !S || !o || !gates_match(gate, beta, b, w))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, b, w, S, o};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    if ((long long)B * H > 0x7fffffffLL) return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_decode_gated(q, k, v, alpha, beta, b, w, S, o, B, H, K, V, gate,
                                              dtype, static_cast<cudaStream_t>(stream)));
}

int gdn_state_truncate(float *S, int BH, int V, int K, int r, float *sigma, int max_sweeps,
                       void *stream) {
    if (BH < 0 || r < 1 || max_sweeps < 1 || max_sweeps > 1000) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (BH == 0) return GDN_OK;
    if (!S) return GDN_ERR_INVALID_ARG;
    if (!aligned16(S) || (sigma && !aligned16(sigma))) return GDN_ERR_ALIGNMENT;
    if (r >= (K < V ? K : V) && !sigma) return GDN_OK;  // nothing to cut, nothing asked
    return from_cuda(gdn::launch_state_truncate(S, BH, V, K, r, sigma, max_sweeps,
                                                static_cast<cudaStream_t>(stream)));
}

int gdn_prefill_truncated(const void *q, const void *k, const void *v, const float *alpha,
                          const float *beta, const float *S0, void *o, float *S_T, int B, int T,
                          int H, int K, int V, gdn_dtype dtype, int seg_len, int r,
                          int max_sweeps, void *workspace, size_t workspace_bytes,
                          void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (seg_len < 1 || r < 1 || max_sweeps < 1 || max_sweeps > 1000) return GDN_ERR_INVALID_ARG;
    if (!S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !alpha || !beta)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, beta, S0, o, S_T};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    // windows are seg_len tokens long, the last one possibly shorter
    const int L = seg_len < T ? seg_len : T, tail = T % seg_len;
    size_t need = gdn_prefill_workspace_size(B, L, H, K, V, dtype);
    if (tail > 0) {
        const size_t need_tail = gdn_prefill_workspace_size(B, tail, H, K, V, dtype);
        if (need_tail > need) need = need_tail;
    }
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if ((long long)B * H == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    const size_t esz = dtype == GDN_BF16 ? 2 : 4;
    const bool tc = dtype == GDN_BF16 && V == 128 && (K == 128 || K == 64);
    const float *start = S0;
    for (int t0 = 0; t0 < T; t0 += seg_len) {
        const int n = T - t0 < seg_len ? T - t0 : seg_len;
        const size_t tok = (size_t)t0 * H;  // token-head offset of the window
        const char *qw = static_cast<const char *>(q) + tok * K * esz;
        const char *kw = static_cast<const char *>(k) + tok * K * esz;
        const char *vw = static_cast<const char *>(v) + tok * V * esz;
        char *ow = o ? static_cast<char *>(o) + tok * V * esz : nullptr;
        cudaError_t e = tc ? gdn::launch_prefill_tc(qw, kw, vw, alpha + tok, beta + tok, start, ow,
                                                    S_T, B, n, T, H, K, V, workspace,
                                                    workspace_bytes, st)
                           : gdn::launch_prefill_gated(qw, kw, vw, alpha + tok, beta + tok,
                                                       nullptr, nullptr, start, ow, S_T, B, n, T,
                                                       H, K, V, GDN_GATE_SCALAR, dtype, st);
        if (e != cudaSuccess) return from_cuda(e);
        start = S_T;
        if (t0 + n < T && r < (K < V ? K : V)) {
            e = gdn::launch_state_truncate(S_T, B * H, V, K, r, nullptr, max_sweeps, st);
            if (e != cudaSuccess) return from_cuda(e);
        }
    }
    return GDN_OK;
}

size_t gdn_channel_gram_workspace_size(int B, int T, int H, int K) {
    if (B <= 0 || T <= 0 || H <= 0 || K != 128) return 0;
    return (size_t)H * gdn::gram_splits(B, T, H) * 128 * 128 * sizeof(float);
}

int gdn_channel_gram(const void *k, const void *q, int B, int T, int H, int K, gdn_dtype dtype,
                     float *G, void *workspace, size_t workspace_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (K != 128 || dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
    if (H == 0) return GDN_OK;
    if (!G) return GDN_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((long long)B * T == 0)
        return from_cuda(cudaMemsetAsync(G, 0, sizeof(float) * (size_t)H * K * K, st));
    if (!k || !q) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {k, q, G, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    if ((long long)B * ((T + 63) / 64) > 0x7fffffffLL || H > 65535) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_channel_gram_workspace_size(B, T, H, K);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    return from_cuda(gdn::launch_channel_gram(k, q, B, T, H, G, workspace, st));
}

int gdn_drrqr_select(const float *G, int H, int n, int k, float f, int max_swaps, int *idx,
                     float *rho_max, int *swaps, void *stream) {
    if (H < 0 || n < 2 || n > 128 || k < 1 || k >= n) return GDN_ERR_INVALID_ARG;
    if (!(f >= 1.f) || !(f < 3.0e38f) || max_swaps < 0 || max_swaps > 100000)
        return GDN_ERR_INVALID_ARG;
    if (H == 0) return GDN_OK;
    if (!G || !idx) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {G, idx, rho_max, swaps};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_drrqr_select(G, H, n, k, f, max_swaps, idx, rho_max, swaps,
                                              static_cast<cudaStream_t>(stream)));
}

size_t gdn_prefill_host_workspace_size(int B, int T, int H, int K, int V, gdn_dtype dtype,
                                       int window) {
    if (B <= 0 || T < 0 || H <= 0 || window < 1 || !supported_kv(K, V)) return 0;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return 0;
    if ((long long)B * H > 0x7fffffffLL) return 0;
    return gdn::host_layout(B, T, H, K, V, dtype, window).total;
}

int gdn_prefill_host(const void *q, const void *k, const void *v, const float *alpha,
                     const float *beta, const float *S0, void *o, float *S_T, int B, int T, int H,
                     int K, int V, gdn_dtype dtype, int window, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (B < 0 || T < 0 || H < 0 || K <= 0 || V <= 0 || window < 1) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP32) return GDN_ERR_INVALID_ARG;
    if (!supported_kv(K, V)) return GDN_ERR_UNSUPPORTED;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !alpha || !beta)) return GDN_ERR_INVALID_ARG;
    if ((long long)B * H == 0) return GDN_OK;
    const size_t need = gdn_prefill_host_workspace_size(B, T, H, K, V, dtype, window);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_prefill_host(q, k, v, alpha, beta, S0, o, S_T, B, T, H, K, V,
                                              dtype, window, workspace,
                                              static_cast<cudaStream_t>(stream)));
}

int gdn_state_rank(const float *S, int BH, int V, int K, float *fro2, float *sigma1,
                   float *stable_rank, int max_iter, float tol, void *stream) {
    if (BH < 0 || V < 1 || K < 1 || V > 128 || K > 128) return GDN_ERR_INVALID_ARG;
    if (max_iter < 1 || !(tol >= 0.f)) return GDN_ERR_INVALID_ARG;
    if (BH == 0) return GDN_OK;
    if (!S || !fro2 || !sigma1 || !stable_rank) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {S, fro2, sigma1, stable_rank};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_state_rank(S, BH, V, K, fro2, sigma1, stable_rank, max_iter,
                                            tol, static_cast<cudaStream_t>(stream)));
}

int gdn_qk_norm_rotate(const void *q, const void *k, const float *wq, const float *wk,
                       const long long *pos, const float *inv_freq, void *yq, void *yk,
                       long long N, int Hq, int Hk, int D, int R, long long q_stride,
                       long long k_stride, gdn_norm norm, gdn_pairing pairing, float eps,
                       gdn_dtype dtype, void *stream) {
    const int e = check_qk_norm(q, k, wq, wk, pos, inv_freq, N, Hq, Hk, D, R, q_stride, k_stride,
                                norm, pairing, eps, dtype);
    if (e != GDN_OK || N == 0 || Hq + Hk == 0) return e;
    if ((Hq && !yq) || (Hk && !yk)) return GDN_ERR_INVALID_ARG;
    if (!aligned16(yq) || !aligned16(yk)) return GDN_ERR_ALIGNMENT;
    // in place only where the rows lie as the outputs do
    if ((yq == q && Hq && q_stride != (long long)Hq * D) ||
        (yk == k && Hk && k_stride != (long long)Hk * D))
        return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_qk_norm(q, k, wq, wk, pos, inv_freq, yq, yk, N, Hq, Hk, D, R,
                                         q_stride, k_stride, norm == GDN_NORM_L2,
                                         pairing == GDN_PAIR_HALF, eps, dtype,
                                         static_cast<cudaStream_t>(stream)));
}

size_t gdn_qk_norm_rotate_backward_workspace_size(long long N, int Hq, int Hk, int D) {
    if (N <= 0 || Hq < 0 || Hk < 0 || Hq + Hk <= 0 || D <= 0) return 0;
    return (size_t)gdn::qk_norm_backward_grid(N, Hq, Hk, D) * D * sizeof(float);
}

int gdn_qk_norm_rotate_backward(const void *q, const void *k, const float *wq, const float *wk,
                                const long long *pos, const float *inv_freq, const void *dyq,
                                const void *dyk, void *dq, void *dk, float *dwq, float *dwk,
                                long long N, int Hq, int Hk, int D, int R, long long q_stride,
                                long long k_stride, gdn_norm norm, gdn_pairing pairing, float eps,
                                gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                                void *stream) {
    const int e = check_qk_norm(q, k, wq, wk, pos, inv_freq, N, Hq, Hk, D, R, q_stride, k_stride,
                                norm, pairing, eps, dtype);
    if (e != GDN_OK) return e;
    if ((dwq && !wq) || (dwk && !wk)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {dyq, dyk, dq, dk, dwq, dwk, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0 || Hq + Hk == 0) {  // sums over nothing
        cudaError_t c = cudaSuccess;
        if (dwq) c = cudaMemsetAsync(dwq, 0, sizeof(float) * D, st);
        if (dwk && c == cudaSuccess) c = cudaMemsetAsync(dwk, 0, sizeof(float) * D, st);
        return from_cuda(c);
    }
    if ((Hq && (!dyq || !dq)) || (Hk && (!dyk || !dk))) return GDN_ERR_INVALID_ARG;
    if ((dwq || dwk) &&
        (!workspace || workspace_bytes < gdn_qk_norm_rotate_backward_workspace_size(N, Hq, Hk, D)))
        return GDN_ERR_WORKSPACE;
    return from_cuda(gdn::launch_qk_norm_backward(
        q, k, wq, wk, pos, inv_freq, dyq, dyk, dq, dk, dwq, dwk, N, Hq, Hk, D, R, q_stride,
        k_stride, norm == GDN_NORM_L2, pairing == GDN_PAIR_HALF, eps, dtype,
        static_cast<float *>(workspace), st));
}

size_t gdn_linear_prefill_workspace_size(int B, int T, int H, int K, int V, int packed,
                                         gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || !linear_kv(K, V)) return 0;
    return gdn::linear_scan_workspace(B, T, H, K, V, packed != 0, dtype);
}

int gdn_linear_prefill(const void *q, const void *k, const void *v, const float *alpha,
                       const float *S0, void *o, float *S_T, const int *offsets, int B, int T,
                       int Hq, int H, int K, int V, long long q_stride, long long k_stride,
                       long long v_stride, float scale, gdn_dtype dtype, void *workspace,
                       size_t workspace_bytes, void *stream) {
    const int e = check_linear(B, T, Hq, H, K, V, q_stride, k_stride, v_stride, dtype);
    if (e != GDN_OK) return e;
    if (!o && !S_T) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, S0, o, S_T, offsets, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (B == 0 || H == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(S0, S_T, B, H, K, V, st);
    if ((!q && o) || !k || !v || !alpha) return GDN_ERR_INVALID_ARG;
    if (workspace_bytes < gdn_linear_prefill_workspace_size(B, T, H, K, V, offsets != nullptr, dtype) ||
        (!workspace && workspace_bytes))
        return GDN_ERR_WORKSPACE;
    gdn::LinearScan a = {};
    a.q = q; a.k = k; a.v = v;
    a.alpha = alpha; a.S0 = S0; a.o = o; a.ST = S_T; a.offsets = offsets;
    a.B = B; a.T = T; a.H = H; a.Hq = a.Hk = Hq; a.Hv = H; a.K = K; a.V = V;
    a.ldq = q_stride; a.ldk = k_stride; a.ldv = v_stride;
    a.write_scale = 1.f;
    a.read_scale = scale;
    a.exact = true;
    return from_cuda(gdn::launch_linear_scan(&a, 1, dtype, workspace, st));
}

namespace {
// The scans' slots, rounded up so that what follows is aligned: on the tensor
// cores one scan runs after another, on the CUDA cores all at once.
size_t linear_backward_slots(int B, int T, int H, int K, int V, bool packed, gdn_dtype dtype) {
    const size_t dv = gdn::linear_scan_workspace(B, T, H, K, V, packed, dtype);
    const size_t dqk = gdn::linear_scan_workspace(B, T, H, V, K, packed, dtype);
    const size_t n = !gdn::linear_on_tensor_cores(T, K, V, dtype) ? 2 * dqk + dv : dqk > dv ? dqk : dv;
    return (n + 255) & ~size_t(255);
}
// One head's part of a gradient that a group of heads shares, in float32 (bytes).
size_t linear_part(int B, int T, int H, int K, bool packed) {
    return ((size_t)(packed ? 1 : B) * T * H * K * sizeof(float) + 255) & ~size_t(255);
}
}  // namespace

size_t gdn_linear_backward_workspace_size(int B, int T, int Hq, int H, int K, int V, int packed,
                                          gdn_dtype dtype) {
    if (B <= 0 || T <= 0 || H <= 0 || Hq <= 0 || !linear_kv(K, V)) return 0;
    const size_t n = linear_backward_slots(B, T, H, K, V, packed != 0, dtype);
    if (Hq == H) return n;
    return n + (gdn::linear_on_tensor_cores(T, K, V, dtype) ? 1 : 2) * linear_part(B, T, H, K, packed != 0);
}

int gdn_linear_backward(const void *q, const void *k, const void *v, const float *alpha,
                        const void *dO, const float *S0, const float *dS_T, void *dq, void *dk,
                        void *dv, float *dS0, const int *offsets, int B, int T, int Hq, int H,
                        int K, int V, long long q_stride, long long k_stride, long long v_stride,
                        float scale, gdn_dtype dtype, void *workspace, size_t workspace_bytes,
                        void *stream) {
    const int e = check_linear(B, T, Hq, H, K, V, q_stride, k_stride, v_stride, dtype);
    if (e != GDN_OK) return e;
    if (!dq && !dk && !dv && !dS0) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, dO, S0, dS_T, dq, dk, dv, dS0, offsets, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (B == 0 || H == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return empty_prefill(dS_T, dS0, B, H, K, V, st);
    if (!q || !k || !v || !alpha || !dO) return GDN_ERR_INVALID_ARG;
    const size_t need =
        gdn_linear_backward_workspace_size(B, T, Hq, H, K, V, offsets != nullptr, dtype);
    if (workspace_bytes < need || (!workspace && workspace_bytes)) return GDN_ERR_WORKSPACE;
    const long long tokens = offsets ? T : (long long)B * T;
    char *const parts = static_cast<char *>(workspace) +
                        linear_backward_slots(B, T, H, K, V, offsets != nullptr, dtype);
    const bool together = !gdn::linear_on_tensor_cores(T, K, V, dtype);
    const int group = H / Hq;
    float *const part_q = reinterpret_cast<float *>(parts);
    float *const part_k = together ? reinterpret_cast<float *>(
                                         parts + linear_part(B, T, H, K, offsets != nullptr))
                                   : part_q;
    const long long ldo = (long long)H * V;

    gdn::LinearScan base = {};
    base.alpha = alpha; base.offsets = offsets;
    base.B = B; base.T = T; base.H = H;
    gdn::LinearScan scans[3];
    int n = 0;
    // dq and dk go out in float32, one part a head, where a group of heads shares them
    if (dq) {
        gdn::LinearScan &a = scans[n++] = base;
        a.q = dO; a.ldq = ldo; a.Hq = H;
        a.k = v; a.ldk = v_stride; a.Hk = H;
        a.v = k; a.ldv = k_stride; a.Hv = Hq;
        a.K = V; a.V = K;
        a.S0 = S0; a.s0_transposed = true; a.reverse = false;
        a.write_scale = 1.f; a.read_scale = scale;
        a.o = group > 1 ? part_q : dq;
        a.o_float = group > 1 || dtype == GDN_FP32;
    }
    if (dk) {
        gdn::LinearScan &a = scans[n++] = base;
        a.q = v; a.ldq = v_stride; a.Hq = H;
        a.k = dO; a.ldk = ldo; a.Hk = H;
        a.v = q; a.ldv = q_stride; a.Hv = Hq;
        a.K = V; a.V = K;
        a.S0 = dS_T; a.s0_transposed = true; a.reverse = true;
        a.write_scale = scale; a.read_scale = 1.f;
        a.o = group > 1 ? part_k : dk;
        a.o_float = group > 1 || dtype == GDN_FP32;
    }
    const int shared = n;
    if (dv || dS0) {
        gdn::LinearScan &a = scans[n++] = base;
        a.q = k; a.ldq = k_stride; a.Hq = Hq;
        a.k = q; a.ldk = q_stride; a.Hk = Hq;
        a.v = dO; a.ldv = ldo; a.Hv = H;
        a.K = K; a.V = V;
        a.S0 = dS_T; a.s0_transposed = false; a.reverse = true;
        a.write_scale = scale; a.read_scale = 1.f;
        a.o = dv; a.ST = dS0; a.exact = dS0 != nullptr; a.o_float = dtype == GDN_FP32;
    }
    cudaError_t c = cudaSuccess;
    // all at once where nothing keeps them apart: dS0 may take dS_T's place, which dk's scan
    // reads, and the launch takes two scans of one width first
    if (together && n == 3 && (!dS0 || (dS0 != dS_T && dS0 != S0))) {
        c = gdn::launch_linear_scan(scans, 3, dtype, workspace, st);
        if (c == cudaSuccess && group > 1)
            c = gdn::launch_group_sum(part_q, part_k, dq, dk, tokens, Hq, group, K, dtype, st);
        return from_cuda(c);
    }
    for (int i = 0; i < n && c == cudaSuccess; ++i) {
        c = gdn::launch_linear_scan(&scans[i], 1, dtype, workspace, st);
        if (c == cudaSuccess && i < shared && group > 1)
            c = gdn::launch_group_sum(static_cast<const float *>(scans[i].o), nullptr,
                                      i == 0 && dq ? dq : dk, nullptr, tokens, Hq, group, K, dtype,
                                      st);
    }
    return from_cuda(c);
}

int gdn_linear_decode_step(const void *q, const void *k, const void *v, const float *alpha,
                           const float *S, float *S_out, void *o, int B, int Hq, int H, int K,
                           int V, float scale, gdn_dtype dtype, void *stream) {
    const int e = check_linear(B, 1, Hq, H, K, V, (long long)Hq * K, (long long)Hq * K,
                               (long long)H * V, dtype);
    if (e != GDN_OK || B == 0 || H == 0) return e;
    if (!q || !k || !v || !alpha || !S || !S_out || !o) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {q, k, v, alpha, S, S_out, o};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    return from_cuda(gdn::launch_linear_decode(q, k, v, alpha, S, S_out, o, B, Hq, H, K, V, scale,
                                               dtype, static_cast<cudaStream_t>(stream)));
}

size_t gdn_scan_prefill_workspace_size(int B, int T, int D, int packed) {
    if (B <= 0 || T <= 0 || D <= 0 || !packed) return 0;
    return gdn::scan_map_bytes(T);
}

int gdn_scan_prefill(const void *x, const void *gate, const float *h0, void *h, float *h_T,
                     float *states, const int *offsets, int B, int T, int D, long long x_stride,
                     long long gate_stride, gdn_scan_kind kind, gdn_dtype dtype, void *workspace,
                     size_t workspace_bytes, void *stream) {
    const bool packed = offsets != nullptr;
    const int e = check_scan(x, gate, B, T, D, packed, x_stride, gate_stride, kind, dtype);
    if (e != GDN_OK) return e;
    const void *ptrs[] = {h0, h, h_T, states, offsets, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (B == 0 || D == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long state = (long long)B * D, tokens = packed ? T : (long long)B * T;
    if (T == 0) {
        const Span end[] = {dense(h_T, state, 4, true)}, start[] = {dense(h0, state, 4, true)};
        if (clash(end, start)) return GDN_ERR_INVALID_ARG;
        return empty_prefill(h0, h_T, B, 1, D, 1, st);
    }
    if (!x || !gate || (!h && !h_T && !states)) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_scan_prefill_workspace_size(B, T, D, packed);
    if (workspace_bytes < need || (need && !workspace)) return GDN_ERR_WORKSPACE;
    // every tensor is read while others are written; h_T may take the place of h0
    const ScanSizes z(kind, dtype);
    const Span outs[] = {dense(h, tokens * D, z.x), dense(h_T, state, 4, true),
                         dense(states, scan_states(B, T, packed) * D, 4), dense(workspace, need, 1)};
    const Span ins[] = {strided(x, tokens, D, x_stride, z.x), strided(gate, tokens, D, gate_stride, z.gate),
                        dense(h0, state, 4, true), dense(offsets, B + 1LL, 4)};
    if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
    gdn::ScanArgs a = {};
    a.x = x; a.gate = gate; a.h0 = h0; a.h = h; a.h_T = h_T; a.states = states;
    a.offsets = offsets; a.B = B; a.T = T; a.D = D; a.ldx = x_stride; a.ldg = gate_stride;
    a.sigmoid = kind == GDN_SCAN_SIGMOID;
    return from_cuda(gdn::launch_scan(a, dtype, workspace, st));
}

size_t gdn_scan_backward_workspace_size(int B, int T, int D, int packed, int kept) {
    if (B <= 0 || T <= 0 || D <= 0) return 0;
    return (packed ? gdn::scan_map_bytes(T) : 0) +
           (kept ? 0 : scan_states_bytes(B, T, D, packed != 0));
}

int gdn_scan_backward(const void *x, const void *gate, const void *dh, const float *h0,
                      const float *dh_T, const float *states, void *dx, void *dgate, float *dh0,
                      const int *offsets, int B, int T, int D, long long x_stride,
                      long long gate_stride, gdn_scan_kind kind, gdn_dtype dtype, void *workspace,
                      size_t workspace_bytes, void *stream) {
    const bool packed = offsets != nullptr;
    const int e = check_scan(x, gate, B, T, D, packed, x_stride, gate_stride, kind, dtype);
    if (e != GDN_OK) return e;
    const void *ptrs[] = {dh, h0, dh_T, states, dx, dgate, dh0, offsets, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (B == 0 || D == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long state = (long long)B * D, tokens = packed ? T : (long long)B * T;
    if (T == 0) {
        const Span end[] = {dense(dh0, state, 4, true)}, start[] = {dense(dh_T, state, 4, true)};
        if (clash(end, start)) return GDN_ERR_INVALID_ARG;
        return empty_prefill(dh_T, dh0, B, 1, D, 1, st);
    }
    if (!x || !gate || !dh || !dx || !dgate) return GDN_ERR_INVALID_ARG;
    const size_t need = gdn_scan_backward_workspace_size(B, T, D, packed, states != nullptr);
    if (workspace_bytes < need || (need && !workspace)) return GDN_ERR_WORKSPACE;
    // every tile's inputs are read while the outputs of others are written
    const ScanSizes z(kind, dtype);
    const Span outs[] = {dense(dx, tokens * D, z.x), dense(dgate, tokens * D, z.gate), dense(dh0, state, 4),
                         dense(workspace, need, 1)};
    const Span ins[] = {strided(x, tokens, D, x_stride, z.x), strided(gate, tokens, D, gate_stride, z.gate),
                        dense(dh, tokens * D, z.x), dense(h0, state, 4), dense(dh_T, state, 4),
                        dense(states, scan_states(B, T, packed) * D, 4), dense(offsets, B + 1LL, 4)};
    if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
    gdn::ScanArgs a = {};
    a.x = x; a.gate = gate; a.dh = dh; a.h0 = h0; a.dh_T = dh_T; a.states = const_cast<float *>(states);
    a.dx = dx; a.dgate = dgate; a.dh0 = dh0;
    a.offsets = offsets; a.B = B; a.T = T; a.D = D; a.ldx = x_stride; a.ldg = gate_stride;
    a.sigmoid = kind == GDN_SCAN_SIGMOID;
    return from_cuda(gdn::launch_scan_backward(a, dtype, workspace, st));
}

int gdn_scan_decode_step(const void *x, const void *gate, const float *h, float *h_out, void *y,
                         int B, int D, long long x_stride, long long gate_stride,
                         gdn_scan_kind kind, gdn_dtype dtype, void *stream) {
    const int e = check_scan(x, gate, B, 1, D, false, x_stride, gate_stride, kind, dtype);
    if (e != GDN_OK) return e;
    if (!aligned16(h) || !aligned16(h_out) || !aligned16(y)) return GDN_ERR_ALIGNMENT;
    if (B == 0 || D == 0) return GDN_OK;
    if (!x || !gate || !h || !h_out) return GDN_ERR_INVALID_ARG;
    // threads read what others write unless h_out is h; x and gate have rows and types of
    // their own
    const ScanSizes z(kind, dtype);
    const long long n = (long long)B * D;
    const Span outs[] = {dense(h_out, n, 4, true), dense(y, n, z.x)};
    const Span ins[] = {strided(x, B, D, x_stride, z.x), strided(gate, B, D, gate_stride, z.gate),
                        dense(h, n, 4, true)};
    if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_scan_step(x, gate, h, h_out, y, B, D, x_stride, gate_stride,
                                           kind == GDN_SCAN_SIGMOID, dtype,
                                           static_cast<cudaStream_t>(stream)));
}

int gdn_layer_norm(const void *x, const void *residual, const float *w, const float *b, void *y,
                   void *s, float *stats, long long N, int D, long long x_stride,
                   long long residual_stride, float eps, gdn_dtype dtype, void *stream) {
    const int e = check_layer_norm(N, D, dtype);
    if (e != GDN_OK) return e;
    if (!(eps >= 0.f)) return GDN_ERR_INVALID_ARG;
    const int unit = dtype == GDN_BF16 ? 8 : 4;  // elements of 16 bytes
    if (x_stride < D || x_stride % unit ||
        (residual && (residual_stride < D || residual_stride % unit)))
        return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, residual, w, b, y, s, stats};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (N == 0 || D == 0) return GDN_OK;
    if (!x || !y || (s && !residual)) return GDN_ERR_INVALID_ARG;
    // rows are read while others are written; in place only where they lie as the outputs do
    const long long z = dtype == GDN_BF16 ? 2 : 4;
    const Span outs[] = {dense(y, N * D, z, true), dense(s, N * D, z, true), dense(stats, N * 2, 4)};
    const Span ins[] = {strided(x, N, D, x_stride, z, x_stride == D),
                        strided(residual, N, D, residual_stride, z, residual_stride == D),
                        dense(w, D, 4), dense(b, D, 4)};
    if (clash(outs, ins)) return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_layer_norm(x, residual, w, b, y, s, stats, N, D, x_stride,
                                            residual_stride, eps, dtype,
                                            static_cast<cudaStream_t>(stream)));
}

size_t gdn_layer_norm_backward_workspace_size(long long N, int D) {
    if (N <= 0 || D <= 0 || D > 16384) return 0;
    return (size_t)gdn::layer_norm_parts(N, D) * 2 * D * sizeof(float);
}

int gdn_layer_norm_backward(const void *s, const void *dy, const float *stats, const float *w,
                            const void *ds, void *dx, float *dw, float *db, long long N, int D,
                            long long s_stride, gdn_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    const int e = check_layer_norm(N, D, dtype);
    if (e != GDN_OK) return e;
    if (s_stride < D || s_stride % (dtype == GDN_BF16 ? 8 : 4)) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {s, dy, stats, w, ds, dx, dw, db, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return GDN_ERR_ALIGNMENT;
    if (D == 0) return GDN_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) {  // sums over nothing
        cudaError_t c = cudaSuccess;
        if (dw) c = cudaMemsetAsync(dw, 0, sizeof(float) * D, st);
        if (db && c == cudaSuccess) c = cudaMemsetAsync(db, 0, sizeof(float) * D, st);
        return from_cuda(c);
    }
    if (!s || !dy || !stats || !dx) return GDN_ERR_INVALID_ARG;
    const size_t need = dw || db ? gdn_layer_norm_backward_workspace_size(N, D) : 0;
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    // rows are read while others are written; dx in place only where they lie as its own do;
    // dw and db are written when all else has been read
    const long long z = dtype == GDN_BF16 ? 2 : 4;
    const Span rows[] = {dense(dx, N * D, z, true), dense(workspace, need, 1)};
    const Span sums[] = {dense(dw, D, 4), dense(db, D, 4)};
    const Span ins[] = {strided(s, N, D, s_stride, z, s_stride == D), dense(dy, N * D, z, true),
                        dense(ds, N * D, z, true), dense(stats, N * 2, 4), dense(w, D, 4)};
    if (clash(rows, ins) || clash(sums, rows)) return GDN_ERR_INVALID_ARG;
    return from_cuda(gdn::launch_layer_norm_backward(s, dy, stats, w, ds, dx, dw, db, N, D, s_stride,
                                                     dtype, static_cast<float *>(workspace), st));
}

int gdn_get_last_device_status(void *stream) {
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return GDN_ERR_CUDA;
    int word = 0;
    if (cudaMemcpyFromSymbol(&word, gdn::g_device_status, sizeof(int)) != cudaSuccess)
        return GDN_ERR_CUDA;
    const int zero = 0;
    if (word != 0 && cudaMemcpyToSymbol(gdn::g_device_status, &zero, sizeof(int)) != cudaSuccess)
        return GDN_ERR_CUDA;
    if (word & gdn::kStatusTimeout) return GDN_ERR_TIMEOUT;
    if (word & gdn::kStatusBounds) return GDN_ERR_DEVICE_BOUNDS;
    if (word & gdn::kStatusNotConverged) return GDN_WARN_NOT_CONVERGED;
    if (word & gdn::kStatusRankDeficient) return GDN_WARN_RANK_DEFICIENT;
    if (word & gdn::kStatusZeroState) return GDN_WARN_ZERO_STATE;
    return GDN_OK;
}

}  // extern "C"
