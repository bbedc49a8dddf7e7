// Self-tests of the bounded waits: a wait on an mbarrier that never completes must give up,
// record the timeout in the device status word and return (no trap, no hang); a kernel that
// lacks one of its copies must end the same way.
#include "gdn_internal.cuh"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

__global__ void wait_timeout_kernel(long long limit, int *status) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        sm100::mbar_init(&bar, 1);
        sm100::fence_mbar_init();
        // nothing ever arrives: the phase with parity 0 never completes
        if (!sm100::mbar_wait(&bar, 0, limit) && status) atomicOr(status, kStatusTimeout);
    }
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_selftest_wait_timeout(long long limit_cycles, void *stream) {
    if (limit_cycles < 1 || limit_cycles > (1LL << 31)) return GDN_ERR_INVALID_ARG;
    gdn::wait_timeout_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(
        limit_cycles, gdn::device_status_ptr());
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_selftest_lost_copy(gdn_selftest_call call, long long limit_cycles, long long lost,
                                      void *buffer, size_t bytes, int rows, int T, int D,
                                      void *stream) {
    if (limit_cycles < 1 || limit_cycles > (1LL << 31) || lost < 0 || !buffer || rows < 1 || T < 1 ||
        D < 8 || D % 8 || (reinterpret_cast<uintptr_t>(buffer) & 15))
        return GDN_ERR_INVALID_ARG;
    // each tensor has the room of float32 values (the states before every 64th token are float32)
    const long long tokens = (long long)rows * T, part = ((tokens * D * 4) + 255) / 256 * 256;
    if (tokens > (1 << 24) || D > 16384) return GDN_ERR_INVALID_ARG;
    if (bytes < (size_t)part * 6) return GDN_ERR_WORKSPACE;
    char *const at = static_cast<char *>(buffer);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaErrorInvalidValue;
    if (call == GDN_SELFTEST_SCAN || call == GDN_SELFTEST_SCAN_BACKWARD) {
        gdn::ScanArgs a = {};
        a.x = at;
        a.gate = at + part;
        a.states = reinterpret_cast<float *>(at + 2 * part);
        a.B = rows; a.T = T; a.D = D;
        a.ldx = a.ldg = D;
        a.sigmoid = true;
        if (call == GDN_SELFTEST_SCAN) {
            a.h = at + 3 * part;
        } else {
            a.dh = at + 3 * part;
            a.dx = at + 4 * part;
            a.dgate = at + 5 * part;
        }
        e = gdn::launch_scan_lost(a, limit_cycles, (int)(lost < tokens ? lost : tokens), st);
    }
    if (call >= GDN_SELFTEST_NORM && call <= GDN_SELFTEST_NORM_BACKWARD) {
        const long long half = part / 2;
        float *const stats = reinterpret_cast<float *>(at + 4 * half);
        if (call == GDN_SELFTEST_NORM_BACKWARD)
            e = gdn::launch_layer_norm_backward_lost(
                at, at + half, stats, at + 2 * half, at + 3 * half,
                reinterpret_cast<float *>(at + 5 * part), reinterpret_cast<float *>(at + 3 * part),
                tokens, D, limit_cycles, lost, st);
        else
            e = gdn::launch_layer_norm_lost(at, call == GDN_SELFTEST_NORM ? nullptr : at + half,
                                            at + 2 * half, stats, tokens, D, limit_cycles,
                                            call == GDN_SELFTEST_NORM_ANSWER ? -1 : lost, st);
    }
    if (e == cudaErrorInvalidValue) return GDN_ERR_INVALID_ARG;
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
