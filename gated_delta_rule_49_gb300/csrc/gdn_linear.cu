// Linear attention with a decay for each head on the CUDA cores: the token by
// token scan (float32 runs and the (32, 32) variant), the single-token step,
// and the dispatch of a scan.
#include "gdn_linear.cuh"
#include "gdn_vec8.cuh"

namespace gdn {
namespace {

// ------------------------------------------------------------------ scan
//
// Value channels are independent: row v of the state is S_v <- a S_v +
// (write_scale v_t) k_t, o_v = read_scale S_v . q_t.  A warp keeps 8 rows in
// registers (a lane holds K / 32 columns of each), so a token costs 2 fused
// multiply-adds and a product for each element and 9 shuffles for the 8 dot
// products; a CTA of 4 warps covers 32 rows.  Tiles of 16 tokens go through
// shared memory as float32, the next tile's loads in flight during this
// one's arithmetic.  Bound by the float32 pipes: 3 K V instructions-lanes a
// token and head, as many as a chunk form without tensor cores would need.
constexpr int kScanThreads = 128;
constexpr int kTile = 16;      // tokens
constexpr int kRows = 8;       // rows of a warp
constexpr int kCtaRows = 32;

template <int C> struct Cols;  // C consecutive floats of a row
template <> struct Cols<1> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[1]) { x[0] = p[0]; }
};
template <> struct Cols<2> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[2]) {
        const float2 y = *reinterpret_cast<const float2 *>(p);
        x[0] = y.x; x[1] = y.y;
    }
};
template <> struct Cols<4> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[4]) {
        const float4 y = *reinterpret_cast<const float4 *>(p);
        x[0] = y.x; x[1] = y.y; x[2] = y.z; x[3] = y.w;
    }
};

//
// Up to three scans run in one launch (a backward pass: they do not depend on
// one another, and a small one is all start-up: B = 2, T = 391, 4 heads of 64 x
// 128 take 73 us as six launches and two sums, 49 us as two and one).
struct TokenScan {
    LinearScan p;
    SegPlan plan;
    float *slots;  // NULL: not cut
};
struct TokenScans {
    TokenScan scan[3];
    int count;
};
template <int K> constexpr int token_smem() { return kTile * (2 * K + kCtaRows); }  // floats

template <typename T, int K>
__device__ __forceinline__ void token_scan(const LinearScan &p, const SegPlan &plan,
                                           const float *slots_in, float *slots_out, float *sm,
                                           int *status) {
    constexpr int C = K / 32;             // columns of a lane
    constexpr int QV = kTile * K / 8;     // 8-element pieces of a q or k tile
    constexpr int QN = (QV + kScanThreads - 1) / kScanThreads;
    float(*const qs)[K] = reinterpret_cast<float(*)[K]>(sm);
    float(*const ks)[K] = qs + kTile;
    float(*const vs)[kCtaRows] = reinterpret_cast<float(*)[kCtaRows]>(ks + kTile);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = p.V / kCtaRows;
    const int blk = blockIdx.x % blocks;
    const int h = blockIdx.x / blocks % p.H;
    const int item = blockIdx.x / blocks / p.H;
    const LinearItem it = linear_item(p.offsets, p.B, p.T, plan.seg_len, item, status);
    if (it.seq < 0) return;
    const bool last = p.reverse ? it.j == 0 : it.j == it.n - 1;  // in scan order
    if (slots_out && last && !p.S0) return;  // nothing starts from its end
    const bool want_o = p.o && !slots_out;
    const int f0 = it.j * plan.seg_len;
    // tokens; the last segment's slot only takes a copy of S0
    const int n = slots_out && last ? 0 : min(it.len - f0, plan.seg_len);
    const float a = p.alpha[h], lg = decay_log2(a);
    const size_t VK = (size_t)p.V * K;
    const int row0 = blk * kCtaRows + warp * kRows;
    const int hq = h / (p.H / p.Hq), hk = h / (p.H / p.Hk), hv = h / (p.H / p.Hv);

    // the start state: the loads of a slot together, one slot after another
    float S[kRows][C];
    auto add_slot = [&](int at, float f) {
        const float *src = slots_in + ((size_t)at * p.H + h) * VK + (size_t)row0 * K + lane * C;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float x[C];
            Cols<C>::load(src + r * K, x);
#pragma unroll
            for (int c = 0; c < C; ++c) S[r][c] = fmaf(f, x[c], S[r][c]);
        }
    };
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
            S[r][c] = p.S0 && (slots_out ? last : !slots_in)
                          ? given_start(p.S0, p.s0_transposed, (size_t)it.seq * p.H + h, p.V, K,
                                        row0 + r, lane * C + c)
                          : 0.f;
    if (slots_in) {
        if (p.S0) add_slot(it.slot0 + (p.reverse ? 0 : it.n - 1),
                           decay_power(start_steps(it, plan.seg_len, p.reverse), lg));
#pragma unroll 4
        for (int i = p.reverse ? it.j + 1 : 0; i < (p.reverse ? it.n : it.j); ++i)
            add_slot(it.slot0 + i,
                     decay_power(tokens_between(i, it.j, it.len, plan.seg_len, p.reverse), lg));
    }
    const T *qp = static_cast<const T *>(p.q) + (long long)hq * K;
    const T *kp = static_cast<const T *>(p.k) + (long long)hk * K;
    const T *vp = static_cast<const T *>(p.v) + (long long)hv * p.V + blk * kCtaRows;
    // token of scan position i
    auto token = [&](int i) { return it.first + f0 + (p.reverse ? n - 1 - i : i); };

    Vec8<T> rq[QN], rk[QN], rv;
    auto fetch = [&](int i0) {
#pragma unroll
        for (int x = 0; x < QN; ++x) {
            const int piece = threadIdx.x + x * kScanThreads;
            const int t = piece / (K / 8), c = piece % (K / 8);
            if (piece < QV && i0 + t < n) {
                const long long tok = token(i0 + t);
                if (want_o) rq[x].load_cached(qp + tok * p.ldq + 8 * c);
                rk[x].load_cached(kp + tok * p.ldk + 8 * c);
            }
        }
        const int t = threadIdx.x / 4, c = threadIdx.x % 4;
        if (threadIdx.x < kTile * 4 && i0 + t < n)
            rv.load_cached(vp + token(i0 + t) * p.ldv + 8 * c);
    };
    auto put = [&](int i0) {
        float x8[8];
#pragma unroll
        for (int x = 0; x < QN; ++x) {
            const int piece = threadIdx.x + x * kScanThreads;
            const int t = piece / (K / 8), c = piece % (K / 8);
            if (piece < QV && i0 + t < n) {
                if (want_o) {
                    rq[x].get(x8);
                    Vec8<float>::store(&qs[t][8 * c], x8);
                }
                rk[x].get(x8);
                Vec8<float>::store(&ks[t][8 * c], x8);
            }
        }
        const int t = threadIdx.x / 4, c = threadIdx.x % 4;
        if (threadIdx.x < kTile * 4 && i0 + t < n) {
            rv.get(x8);
#pragma unroll
            for (int e = 0; e < 8; ++e) x8[e] *= p.write_scale;
            Vec8<float>::store(&vs[t][8 * c], x8);
        }
    };

    // the row whose dot product this lane holds after the transposing sums
    const int my_row = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
    // a reversed scan takes its start state up undecayed
    bool lead = !(p.reverse && it.j == it.n - 1);
    if (n > 0) fetch(0);
    for (int i0 = 0; i0 < n; i0 += kTile) {
        __syncthreads();
        put(i0);
        __syncthreads();
        if (i0 + kTile < n) fetch(i0 + kTile);
        const int m = min(kTile, n - i0);
#pragma unroll 4
        for (int t = 0; t < m; ++t) {
            float kk[C], qq[C], w[kRows], acc[kRows];
            Cols<C>::load(&ks[t][lane * C], kk);
            Cols<4>::load(&vs[t][warp * kRows], *reinterpret_cast<float(*)[4]>(&w[0]));
            Cols<4>::load(&vs[t][warp * kRows + 4], *reinterpret_cast<float(*)[4]>(&w[4]));
            const float at = lead ? a : 1.f;
            lead = true;
#pragma unroll
            for (int r = 0; r < kRows; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c) S[r][c] = fmaf(w[r], kk[c], at * S[r][c]);
            if (!want_o) continue;
            Cols<C>::load(&qs[t][lane * C], qq);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                acc[r] = S[r][0] * qq[0];
#pragma unroll
                for (int c = 1; c < C; ++c) acc[r] = fmaf(S[r][c], qq[c], acc[r]);
            }
            // sums over the warp, halving the rows a lane holds at each step
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                const int half = 4 >> s, bit = 16 >> s;
                const bool up = lane & bit;
#pragma unroll
                for (int r = 0; r < half; ++r) {
                    const float give = up ? acc[r] : acc[r + half];
                    const float keep = up ? acc[r + half] : acc[r];
                    acc[r] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
                }
            }
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 2);
            acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], 1);
            if ((lane & 3) == 0) {
                const float o = p.read_scale * acc[0];
                const long long at_o = (token(i0 + t) * p.H + h) * p.V + row0 + my_row;
                if (p.o_float) static_cast<float *>(p.o)[at_o] = o;
                else static_cast<T *>(p.o)[at_o] = from_f32<T>(o);
            }
        }
    }
    float *end = slots_out ? slots_out + ((size_t)(it.slot0 + it.j) * p.H + h) * VK
                 : p.ST && last ? p.ST + ((size_t)it.seq * p.H + h) * VK : nullptr;
    if (!end) return;
    // the state that a reversed scan returns has decayed once more
    const float f = !slots_out && p.reverse && it.len > 0 ? a : 1.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) end[(size_t)(row0 + r) * K + lane * C + c] = f * S[r][c];
}

// Scans 0 .. count - 1 in the y blocks; the last of three has its own width.
template <typename T, int KA, int KB>
__global__ void __launch_bounds__(kScanThreads)
    linear_token_kernel(const __grid_constant__ TokenScans a, bool first_pass, int *status) {
    constexpr int kFloats = token_smem<(KA > KB ? KA : KB)>();
    __shared__ __align__(16) float sm[kFloats];
    const TokenScan &s = a.scan[blockIdx.y];
    if (first_pass && !s.slots) return;
    const float *in = first_pass ? nullptr : s.slots;
    float *out = first_pass ? s.slots : nullptr;
    if (KA == KB || blockIdx.y < 2) token_scan<T, KA>(s.p, s.plan, in, out, sm, status);
    else token_scan<T, KB>(s.p, s.plan, in, out, sm, status);
}

// Cuts as in linear_tc_plan, counted in token times: about six CTAs run on an
// SM, one needs its segment's tokens and about 32 more to start and end, and a
// first pass as long again.
SegPlan token_plan(int B, int T, int H, int V, bool packed) {
    const int nsm = sm_count() > 0 ? sm_count() : 152;
    const long long longest = packed && 4LL * T / B < T ? 4LL * T / B : T;
    auto waves = [&](long long items) {
        return (double)((items * H * (V / kCtaRows) + 6 * nsm - 1) / (6 * nsm));
    };
    SegPlan best{T > 0 ? T : 1, B};
    double least = waves(B) * (longest + 32);
    for (int n = 2; n <= 64 && longest / n >= kTile; ++n) {
        const long long len = (longest + (long long)n * kTile - 1) / ((long long)n * kTile) * kTile;
        const long long per = ((packed ? T : longest) + len - 1) / len;
        const long long items = packed ? per + B : per * B;
        const double cost = waves(items) * (len + 32) * 2;
        if (cost < least) {
            least = cost;
            best = {(int)len, (int)items};
        }
    }
    return best;
}

size_t token_slots(const LinearScan &p) {
    const SegPlan plan = token_plan(p.B, p.T, p.H, p.V, p.offsets != nullptr);
    return plan.items > p.B ? (size_t)plan.items * p.H * p.V * p.K : 0;
}

template <typename T>
cudaError_t launch_token(const LinearScan *p, int count, float *slots, cudaStream_t st) {
    TokenScans a = {};
    a.count = count;
    long long grid = 0;
    bool cut = false;
    for (int i = 0; i < count; ++i) {
        a.scan[i].p = p[i];
        a.scan[i].plan = token_plan(p[i].B, p[i].T, p[i].H, p[i].V, p[i].offsets != nullptr);
        const size_t n = token_slots(p[i]);
        a.scan[i].slots = n ? slots : nullptr;
        slots += n;
        cut = cut || n;
        const long long g = (long long)a.scan[i].plan.items * p[i].H * (p[i].V / kCtaRows);
        grid = g > grid ? g : grid;
    }
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    int *status = device_status_ptr();
    const dim3 blocks((unsigned)grid, count);
    auto run = [&](bool first) {
        const int ka = p[0].K, kb = p[count - 1].K;
        if (ka == 32) linear_token_kernel<T, 32, 32><<<blocks, kScanThreads, 0, st>>>(a, first, status);
        else if (ka == 64) linear_token_kernel<T, 64, 64><<<blocks, kScanThreads, 0, st>>>(a, first, status);
        else if (kb == 64) linear_token_kernel<T, 128, 64><<<blocks, kScanThreads, 0, st>>>(a, first, status);
        else linear_token_kernel<T, 128, 128><<<blocks, kScanThreads, 0, st>>>(a, first, status);
        return cudaGetLastError();
    };
    if (cut) {
        const cudaError_t e = run(true);
        if (e != cudaSuccess) return e;
    }
    return run(false);
}

// ------------------------------------------------------------------ step
//
// S <- a S + v k^T, o = scale S q, one read and one write of the state: 8 V K
// bytes a head, bound by memory.  K / 4 lanes own a row as float4 pieces; a
// lane's row loads are all issued before any arithmetic.
constexpr int kStepThreads = 128;
constexpr int kStepRows = 4;  // rows of a lane

__device__ __forceinline__ float4 load4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

template <typename T, int K>
__global__ void __launch_bounds__(kStepThreads)
    linear_step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                       const float *__restrict__ alpha, const float *S, float *S_out,
                       T *__restrict__ o, int H, int group, int V, int blocks, float scale) {
    constexpr int LPR = K / 4, RPW = 32 / LPR;
    const int bh = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cl = lane % LPR;
    const int row0 = (blk * (kStepThreads / 32) + warp) * RPW * kStepRows + lane / LPR;
    const size_t head = (size_t)bh * V;
    // the previous step's states are complete before the first read
    pdl_wait();
    float4 s[kStepRows];
    float w[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int row = row0 + r * RPW;
        if (row < V) {
            s[r] = load4(S + (head + row) * K + 4 * cl);
            w[r] = to_f32(v[head + row]);
        } else {
            s[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            w[r] = 0.f;
        }
    }
    const int hq = bh / group;  // [B, H] -> [B, Hq], H = group Hq
    const float4 kf = load4(k + (size_t)hq * K + 4 * cl), qf = load4(q + (size_t)hq * K + 4 * cl);
    const float a = alpha[bh % H];
    pdl_trigger();
#pragma unroll
    for (int r = 0; r < kStepRows; ++r) {
        const int row = row0 + r * RPW;
        float4 x = s[r];
        x.x = fmaf(w[r], kf.x, a * x.x);
        x.y = fmaf(w[r], kf.y, a * x.y);
        x.z = fmaf(w[r], kf.z, a * x.z);
        x.w = fmaf(w[r], kf.w, a * x.w);
        float d = x.x * qf.x + x.y * qf.y + x.z * qf.z + x.w * qf.w;
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if (row < V) {
            *reinterpret_cast<float4 *>(S_out + (head + row) * K + 4 * cl) = x;
            if (cl == 0) o[head + row] = from_f32<T>(scale * d);
        }
    }
}

template <typename T>
cudaError_t launch_step(const void *q, const void *k, const void *v, const float *alpha,
                        const float *S, float *S_out, void *o, int B, int Hq, int H, int K, int V,
                        float scale, cudaStream_t st) {
    const int rows = (kStepThreads / 32) * (32 / (K / 4)) * kStepRows;
    const int blocks = (V + rows - 1) / rows;
    const long long grid = (long long)B * H * blocks;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    auto go = [&](auto kern) {
        return launch_pdl(kern, (unsigned)grid, kStepThreads, 0, st, static_cast<const T *>(q),
                          static_cast<const T *>(k), static_cast<const T *>(v), alpha, S, S_out,
                          static_cast<T *>(o), H, H / Hq, V, blocks, scale);
    };
    switch (K) {
        case 32: return go(linear_step_kernel<T, 32>);
        case 64: return go(linear_step_kernel<T, 64>);
        case 128: return go(linear_step_kernel<T, 128>);
        default: return cudaErrorInvalidValue;
    }
}

// Sums over the heads of a group, in their order, of one tensor or two.
template <typename T>
__global__ void __launch_bounds__(256) group_sum_kernel(const float *x0, const float *x1, T *y0,
                                                        T *y1, long long pieces, int group, int D) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= pieces) return;
    const int per = D / 8;
    const long long row = i / per;
    const float *src = (blockIdx.y ? x1 : x0) + row * group * D + (i - row * per) * 8;
    float s[8] = {};
#pragma unroll 2
    for (int g = 0; g < group; ++g) {
        Vec8<float> v;
        v.load(src + (long long)g * D);
        float u[8];
        v.get(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += u[e];
    }
    Vec8<T>::store((blockIdx.y ? y1 : y0) + i * 8, s);
}

}  // namespace

// bf16 runs on the tensor cores where a tile fills them and there are more than
// eight tokens (in all, where packed).  The outputs of one or two tokens may be
// what is left of terms that cancel (one token's dq is one number for each head,
// summed over the heads that share it, times k): rounded scores then showed as
// up to a third of the result, where the token kernel is off by float32 steps.
// It is also the faster one there (16 heads, 128 x 128, device, prompt / gradients:
// 1 token 5 / 6 us against 21 / 37 on the tensor cores; 64 sequences of 8 tokens
// 65 / 248 against 152 / 261; of 16 tokens 91 / 322 against 153 / 265).
constexpr int kFewTokens = 8;
bool linear_on_tensor_cores(int T, int K, int V, gdn_dtype dt) {
    return dt == GDN_BF16 && K >= 64 && V >= 64 && T > kFewTokens;
}

size_t linear_scan_workspace(int B, int T, int H, int K, int V, bool packed, gdn_dtype dt) {
    const SegPlan plan = linear_on_tensor_cores(T, K, V, dt) ? linear_tc_plan(B, T, H, K, V, packed)
                                                          : token_plan(B, T, H, V, packed);
    return plan.items > B ? (size_t)plan.items * H * V * K * sizeof(float) : 0;
}

cudaError_t launch_linear_scan(const LinearScan *a, int count, gdn_dtype dt, void *workspace,
                               cudaStream_t stream) {
    float *slots = static_cast<float *>(workspace);
    if (linear_on_tensor_cores(a->T, a->K, a->V, dt)) return launch_linear_tc(*a, slots, stream);
    return dt == GDN_BF16 ? launch_token<__nv_bfloat16>(a, count, slots, stream)
                          : launch_token<float>(a, count, slots, stream);
}

cudaError_t launch_group_sum(const float *x0, const float *x1, void *y0, void *y1, long long rows,
                             int Hq, int group, int D, gdn_dtype dt, cudaStream_t stream) {
    const long long pieces = rows * Hq * (D / 8), grid = (pieces + 255) / 256;
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 blocks((unsigned)grid, x1 ? 2 : 1);
    if (dt == GDN_BF16)
        group_sum_kernel<<<blocks, 256, 0, stream>>>(x0, x1, static_cast<__nv_bfloat16 *>(y0),
                                                     static_cast<__nv_bfloat16 *>(y1), pieces, group, D);
    else
        group_sum_kernel<<<blocks, 256, 0, stream>>>(x0, x1, static_cast<float *>(y0),
                                                     static_cast<float *>(y1), pieces, group, D);
    return cudaGetLastError();
}

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *alpha,
                                 const float *S, float *S_out, void *o, int B, int Hq, int H,
                                 int K, int V, float scale, gdn_dtype dt, cudaStream_t stream) {
    return dt == GDN_BF16 ? launch_step<__nv_bfloat16>(q, k, v, alpha, S, S_out, o, B, Hq, H, K, V,
                                                       scale, stream)
                          : launch_step<float>(q, k, v, alpha, S, S_out, o, B, Hq, H, K, V, scale,
                                               stream);
}

}  // namespace gdn
