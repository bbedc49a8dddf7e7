// Which segment of which sequence a CTA takes.  Plain index arithmetic: nothing
// is included here, so that a test can run it on the CPU.
#pragma once

namespace gdn {

// One segment of one sequence.
struct LinearItem {
    int seq;           // -1: nothing to do
    int base;          // the sequence's first token (packed; else 0)
    long long first;   // base in tokens from the start of the tensors
    int len;           // tokens of the sequence
    int j, n;          // this segment and the number of them (>= 1)
    int slot0;         // slot of segment 0 in the workspace
};

// The item-th segment, found by the calling warp (every lane returns it).
// Bad offsets give an empty sequence and the bounds bit of the status: a pair
// that falls, passes T, or starts before the end of an earlier one (of those
// that rise and stay within T).  The sequences that are left do not overlap, so
// that their segments are at most ceil(T / seg_len) + B, whatever the offsets
// hold: the slots of the workspace and the CTAs of the launch.
__device__ __forceinline__ LinearItem linear_item(const int *offsets, int B, int T, int seg_len,
                                                  int item, int *status) {
    LinearItem r;
    if (!offsets) {
        const int n = T > seg_len ? (T + seg_len - 1) / seg_len : 1;
        r.seq = item / n;
        r.j = item - r.seq * n;
        r.n = n;
        r.slot0 = r.seq * n;
        r.len = T;
        r.first = (long long)r.seq * T;
        r.base = 0;
        if (r.seq >= B) r.seq = -1;
        return r;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;  // segments of the sequences before this warp-wide piece
    int upto = 0;    // the furthest end among them
    r.seq = -1;
    for (int s0 = 0; s0 < B; s0 += 32) {
        const int s = s0 + lane;
        int a = 0, len = 0, n = 0, end = 0;
        bool good = true;
        if (s < B) {
            a = offsets[s];
            const int b = offsets[s + 1];
            good = a >= 0 && b >= a && b <= T;
            if (good) {
                end = b;
                len = b - a;
            }
        }
        int far = end;  // the furthest end up to this sequence
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) far = max(far, __shfl_up_sync(0xffffffffu, far, off));
        const int prev = __shfl_up_sync(0xffffffffu, far, 1);
        good = good && a >= (lane ? max(upto, prev) : upto);
        upto = max(upto, __shfl_sync(0xffffffffu, far, 31));
        if (s < B) {
            if (!good) {
                if (status) atomicOr(status, kStatusBounds);
                a = len = 0;
            }
            n = len > seg_len ? (len + seg_len - 1) / seg_len : 1;
        }
        int incl = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const int excl = before + incl - n;
        const bool mine = n > 0 && item >= excl && item < excl + n;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            const int l = __ffs(who) - 1;
            r.seq = s0 + l;
            r.base = __shfl_sync(0xffffffffu, a, l);
            r.len = __shfl_sync(0xffffffffu, len, l);
            r.n = __shfl_sync(0xffffffffu, n, l);
            r.slot0 = __shfl_sync(0xffffffffu, excl, l);
            r.j = item - r.slot0;
            r.first = r.base;
            return r;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return r;
}

}  // namespace gdn
