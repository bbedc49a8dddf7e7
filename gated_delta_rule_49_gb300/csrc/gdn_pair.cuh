// Packed float32 arithmetic: two values an instruction.
#pragma once

#include "gdn_vec8.cuh"

namespace gdn {

// Two float32 values in the registers that packed operations take.
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float x, float y) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }
__device__ __forceinline__ float2 split(Pair a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Pair either(bool first, Pair a, Pair b) { return {first ? a.v : b.v}; }

// Two bf16 values, the lower half first.
__device__ __forceinline__ Pair unpack(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// (As one register pair: put together from two, a load ahead of its use was waited
// for where it stood.)
__device__ __forceinline__ Pair load2(const float *p) {
    return {*reinterpret_cast<const unsigned long long *>(p)};
}
__device__ __forceinline__ void store2(float *p, Pair x) { *reinterpret_cast<float2 *>(p) = split(x); }
__device__ __forceinline__ Pair load2(const __nv_bfloat16 *p) {
    return unpack(*reinterpret_cast<const uint32_t *>(p));
}
__device__ __forceinline__ void store2(__nv_bfloat16 *p, Pair x) {
    const float2 f = split(x);
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(f.x, f.y);
}

// The eight values of a Vec8 as pairs, and back, rounded to its type.
__device__ __forceinline__ void get4(const Vec8<__nv_bfloat16> &v, Pair (&x)[4]) {
    x[0] = unpack(v.a.x);
    x[1] = unpack(v.a.y);
    x[2] = unpack(v.a.z);
    x[3] = unpack(v.a.w);
}
__device__ __forceinline__ void get4(const Vec8<float> &v, Pair (&x)[4]) {
    x[0] = pair(v.a.x, v.a.y);
    x[1] = pair(v.a.z, v.a.w);
    x[2] = pair(v.b.x, v.b.y);
    x[3] = pair(v.b.z, v.b.w);
}
__device__ __forceinline__ uint32_t round2(Pair x) {
    const float2 f = split(x);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ void set4(Vec8<__nv_bfloat16> &v, const Pair (&x)[4]) {
    v.a = make_uint4(round2(x[0]), round2(x[1]), round2(x[2]), round2(x[3]));
}
__device__ __forceinline__ void set4(Vec8<float> &v, const Pair (&x)[4]) {
    const float2 f[4] = {split(x[0]), split(x[1]), split(x[2]), split(x[3])};
    v.a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    v.b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
// From shared memory, and to global memory (both 16-byte aligned).
__device__ __forceinline__ void from_shared(Vec8<__nv_bfloat16> &v, const __nv_bfloat16 *p) {
    v.a = *reinterpret_cast<const uint4 *>(p);
}
__device__ __forceinline__ void from_shared(Vec8<float> &v, const float *p) {
    v.a = reinterpret_cast<const float4 *>(p)[0];
    v.b = reinterpret_cast<const float4 *>(p)[1];
}
__device__ __forceinline__ void put8(__nv_bfloat16 *p, const Vec8<__nv_bfloat16> &v) {
    *reinterpret_cast<uint4 *>(p) = v.a;
}
__device__ __forceinline__ void put8(float *p, const Vec8<float> &v) {
    reinterpret_cast<float4 *>(p)[0] = v.a;
    reinterpret_cast<float4 *>(p)[1] = v.b;
}

}  // namespace gdn
