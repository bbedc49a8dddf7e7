// linear_item on the CPU: a warp is 32 threads that meet at every shuffle.
// Arguments: B T seg_len items packed [offsets ...].  Prints, for each item,
// "seq base first len j n slot0" and the status last; exits 1 where the lanes
// of a warp disagree.
#include <atomic>
#include <barrier>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline
namespace gdn {
constexpr int kStatusBounds = 2;
}
struct Dim { int x; };
static thread_local Dim threadIdx;
static std::barrier<> meet(32);
static int values[32];

static int exchange(int v, int from) {
    values[threadIdx.x] = v;
    meet.arrive_and_wait();
    const int r = values[from];
    meet.arrive_and_wait();
    return r;
}
static int __shfl_up_sync(unsigned, int v, int off) {
    const int lane = threadIdx.x;
    return exchange(v, lane >= off ? lane - off : lane);
}
static int __shfl_sync(unsigned, int v, int from) { return exchange(v, from); }
static unsigned __ballot_sync(unsigned, bool yes) {
    values[threadIdx.x] = yes;
    meet.arrive_and_wait();
    unsigned r = 0;
    for (int i = 0; i < 32; ++i) r |= (unsigned)values[i] << i;
    meet.arrive_and_wait();
    return r;
}
static int __ffs(unsigned x) { return __builtin_ffs((int)x); }
template <typename T> static T max(T a, T b) { return a > b ? a : b; }
static void atomicOr(int *p, int v) { std::atomic_ref<int>(*p).fetch_or(v); }

#include "gdn_linear_item.cuh"

int main(int argc, char **argv) {
    const int B = atoi(argv[1]), T = atoi(argv[2]), seg_len = atoi(argv[3]), items = atoi(argv[4]);
    const bool packed = atoi(argv[5]);
    std::vector<int> offsets;
    for (int i = 6; i < argc; ++i) offsets.push_back(atoi(argv[i]));
    if (packed && (int)offsets.size() != B + 1) return 2;
    int status = 0;
    std::vector<std::vector<gdn::LinearItem>> got(items, std::vector<gdn::LinearItem>(32));
    std::vector<std::thread> warp;
    for (int lane = 0; lane < 32; ++lane)
        warp.emplace_back([&, lane] {
            threadIdx.x = lane;
            for (int i = 0; i < items; ++i)
                got[i][lane] = gdn::linear_item(packed ? offsets.data() : nullptr, B, T, seg_len, i, &status);
        });
    for (auto &t : warp) t.join();
    for (int i = 0; i < items; ++i) {
        const gdn::LinearItem &a = got[i][0];
        for (const gdn::LinearItem &b : got[i])
            if (a.seq != b.seq || (a.seq >= 0 && (a.first != b.first || a.len != b.len || a.j != b.j ||
                                                  a.n != b.n || a.slot0 != b.slot0)))
                return 1;
        if (a.seq < 0) printf("-1 0 0 0 0 0 0\n");
        else printf("%d %d %lld %d %d %d %d\n", a.seq, a.base, a.first, a.len, a.j, a.n, a.slot0);
    }
    printf("%d\n", status);
    return 0;
}
