// One scan of linear attention with a decay a = alpha[h] for each head, as
// both the prompt pass and each of the three gradients need it:
//
//     S <- a S + write_scale v_t k_t^T
//     o_t = read_scale S q_t
//
// over the tokens of a sequence, first to last, or last to first (`reverse`).
// The gradients of o_t = scale S_t q_t are scans of the same form:
//
//     dq_t = scale S_t^T do_t            first to last on (q, k, v) = (do, v, k)
//     dk_t = R_t^T v_t,  dv_t = R_t k_t  last to first on (v, do, q) and (k, q, do)
//     R_t  = a R_{t+1} + scale do_t q_t^T,  dS0 = a R_1
//
// with the states transposed where k and v change places (s0_transposed: the
// start state is given as [K, V]).  What differs in a reversed scan: R takes
// dS_T up before the last token without a decay, and the state that is
// returned has decayed once more (dS0 = a R_1).
//
// Sequences are cut into segments of seg_len tokens when there are few of
// them: the end state is linear in what was written, so a first pass finds
// each segment's end state from a zero start, and the second starts each
// segment from the decayed sum of the others'.
#pragma once

#include "gdn_internal.cuh"
#include "gdn_linear_item.cuh"

namespace gdn {

struct SegPlan {
    int seg_len;  // tokens of a segment
    int items;    // upper bound of the segments of all sequences (dense: the number)
};

// log2 of a decay; 0 becomes a number whose multiples exp2 takes to 0 while
// 0 times it stays 0 (a^0 = 1).
// A decay that is not a number stays one.
__device__ __forceinline__ float decay_log2(float a) {
    const float x = log2f(a);
    return x < -1e30f ? -1e30f : x;
}
// a^n from its log2; a^0 = 1 whatever a is.
__device__ __forceinline__ float decay_power(int n, float lg) {
    return n == 0 ? 1.f : exp2f((float)n * lg);
}

// Tokens between the end of segment i and the start (in scan order) of
// segment j of a sequence, i before j in scan order.
__device__ __forceinline__ int tokens_between(int i, int j, int len, int seg_len, bool reverse) {
    if (!reverse) return (j - i - 1) * seg_len;
    const int end = (j + 1) * seg_len < len ? (j + 1) * seg_len : len;
    return i * seg_len - end;
}

// One element of the start state that the caller gives.
__device__ __forceinline__ float given_start(const float *S0, bool transposed, size_t head, int V,
                                             int K, int v, int k) {
    const float *p = S0 + head * V * K;
    return transposed ? p[(size_t)k * V + v] : p[(size_t)v * K + k];
}

// How often S0 has decayed before a segment: a segment starts from S0 and the
// end states of the segments before it in scan order, in the workspace's slots
// ([slot][H][V][K]).  The slot of a sequence's last segment in scan order, whose
// end nothing starts from, holds a copy of S0: the end states may be written
// over S0 while segments start.
__device__ __forceinline__ int start_steps(const LinearItem &it, int seg_len, bool reverse) {
    if (!reverse) return it.j * seg_len;
    // a reversed scan takes its start state up undecayed
    return it.j == it.n - 1 ? 0 : it.len - (it.j + 1) * seg_len - 1;
}

// The scan on the tensor cores (bf16, K and V of 64 or 128); the segments it
// takes.
SegPlan linear_tc_plan(int B, int T, int H, int K, int V, bool packed);
cudaError_t launch_linear_tc(const LinearScan &a, float *slots, cudaStream_t stream);

}  // namespace gdn
