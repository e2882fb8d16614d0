// fw_rows.cuh -- elements of rows as kernels bound by their bytes handle them: V of them a thread and load,
// as they are stored (Raw), or as fp32 two to an operation (Chan); copies into shared memory ahead of their use.
#pragma once

#include "fw_decay.cuh"

namespace fw {
namespace rows {

template <typename T, int V> struct Raw;
template <> struct Raw<float, 1> { float v; };
template <> struct Raw<float, 2> { float2 v; };
template <> struct Raw<float, 4> { float4 v; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 v; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t v; };
template <> struct Raw<__nv_bfloat16, 4> { uint2 v; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };

template <int V> struct Chan {
    static constexpr int N = (V + 1) / 2;
    uint64_t p[N];                            // (V = 1: the low half; the high one is zero)
};

__device__ __forceinline__ uint64_t bf16_pair(uint32_t x) {
    return pair(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pair_bf16(uint64_t x) {
    const float2 f = halves(x);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ Chan<1> widen(const Raw<float, 1> &r) { return {{pair(r.v, 0.f)}}; }
__device__ __forceinline__ Chan<2> widen(const Raw<float, 2> &r) { return {{pair(r.v.x, r.v.y)}}; }
__device__ __forceinline__ Chan<4> widen(const Raw<float, 4> &r) { return {{pair(r.v.x, r.v.y), pair(r.v.z, r.v.w)}}; }
__device__ __forceinline__ Chan<1> widen(const Raw<__nv_bfloat16, 1> &r) { return {{pair(__bfloat162float(r.v), 0.f)}}; }
__device__ __forceinline__ Chan<2> widen(const Raw<__nv_bfloat16, 2> &r) { return {{bf16_pair(r.v)}}; }
__device__ __forceinline__ Chan<4> widen(const Raw<__nv_bfloat16, 4> &r) { return {{bf16_pair(r.v.x), bf16_pair(r.v.y)}}; }
__device__ __forceinline__ Chan<8> widen(const Raw<__nv_bfloat16, 8> &r) {
    return {{bf16_pair(r.v.x), bf16_pair(r.v.y), bf16_pair(r.v.z), bf16_pair(r.v.w)}};
}

__device__ __forceinline__ void narrow(Raw<float, 1> &r, const Chan<1> &c) { r.v = halves(c.p[0]).x; }
__device__ __forceinline__ void narrow(Raw<float, 2> &r, const Chan<2> &c) { r.v = halves(c.p[0]); }
__device__ __forceinline__ void narrow(Raw<float, 4> &r, const Chan<4> &c) {
    const float2 a = halves(c.p[0]), b = halves(c.p[1]);
    r.v = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 1> &r, const Chan<1> &c) { r.v = __float2bfloat16_rn(halves(c.p[0]).x); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 2> &r, const Chan<2> &c) { r.v = pair_bf16(c.p[0]); }
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 4> &r, const Chan<4> &c) {
    r.v = make_uint2(pair_bf16(c.p[0]), pair_bf16(c.p[1]));
}
__device__ __forceinline__ void narrow(Raw<__nv_bfloat16, 8> &r, const Chan<8> &c) {
    r.v = make_uint4(pair_bf16(c.p[0]), pair_bf16(c.p[1]), pair_bf16(c.p[2]), pair_bf16(c.p[3]));
}

template <typename T, int V> __device__ __forceinline__ Raw<T, V> load(const T *p) {
    return *reinterpret_cast<const Raw<T, V> *>(p);
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const Chan<V> &c) {
    Raw<T, V> r;
    narrow(r, c);
    *reinterpret_cast<Raw<T, V> *>(p) = r;
}

template <int V> __device__ __forceinline__ Chan<V> all(float x) {
    Chan<V> c;
#pragma unroll
    for (int i = 0; i < Chan<V>::N; ++i) c.p[i] = pair(x, V > 1 ? x : 0.f);
    return c;
}
template <int V> __device__ __forceinline__ Chan<V> none() { return all<V>(0.f); }
template <int V> __device__ __forceinline__ Chan<V> fma_n(const Chan<V> &a, const Chan<V> &b, const Chan<V> &c) {
    Chan<V> r;
#pragma unroll
    for (int i = 0; i < Chan<V>::N; ++i) r.p[i] = fma2(a.p[i], b.p[i], c.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Chan<V> mul_n(const Chan<V> &a, const Chan<V> &b) {
    Chan<V> r;
#pragma unroll
    for (int i = 0; i < Chan<V>::N; ++i) r.p[i] = mul2(a.p[i], b.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Chan<V> add_n(const Chan<V> &a, const Chan<V> &b) {
    Chan<V> r;
#pragma unroll
    for (int i = 0; i < Chan<V>::N; ++i) r.p[i] = add2(a.p[i], b.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ float total(const Chan<V> &a) {
    uint64_t t = a.p[0];
#pragma unroll
    for (int i = 1; i < Chan<V>::N; ++i) t = add2(t, a.p[i]);
    const float2 f = halves(t);
    return f.x + f.y;
}

template <int V> __device__ __forceinline__ float element(const Chan<V> &a, int e) {
    const float2 f = halves(a.p[e / 2]);
    return e & 1 ? f.y : f.x;
}

// V floats of a parameter; `other` where it is not given.
template <int V> __device__ __forceinline__ Chan<V> param(const float *p, int64_t at, float other) {
    if (!p) return all<V>(other);
    Chan<V> c;
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + at + e);
            c.p[e / 2] = pair(q.x, q.y);
            c.p[e / 2 + 1] = pair(q.z, q.w);
        }
    } else if constexpr (V == 2) {
        c.p[0] = pair(p[at], p[at + 1]);
    } else {
        c.p[0] = pair(p[at], 0.f);
    }
    return c;
}

// 1 / (1 + exp(-a)) for rows of type T, from one fast power of two and one fast reciprocal (2^-22 each).  bf16 rows
// take the power's argument -a log2(e) as it is rounded, |a| 2^-24 relative (a thousandth of the rows' own
// rounding where it matters); fp32 rows put back what the rounding drops.
template <typename T> __device__ __forceinline__ float sigmoid(float a) {
    const float l = -1.44269504f, t = a * l;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    // 2^t' = 2^t (1 + ln2 (t' - t)), t' = -a log2(e) unrounded; log2(e) = 1.44269504.. + 1.926e-8
    if (sizeof(T) == 4 && fabsf(t) < 126.f) e = fmaf(e, fmaf(0.693147181f, fmaf(a, l, -t), -1.335e-8f * a), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename T, int V> __device__ __forceinline__ Chan<V> sigmoid_n(const Chan<V> &a) {
    Chan<V> s;
#pragma unroll
    for (int i = 0; i < Chan<V>::N; ++i) {
        const float2 f = halves(a.p[i]);
        s.p[i] = pair(sigmoid<T>(f.x), V > 1 ? sigmoid<T>(f.y) : 0.f);
    }
    return s;
}
// silu'(a) = s (1 + a (1 - s)), s = sigmoid(a)
template <int V> __device__ __forceinline__ Chan<V> silu_slope(const Chan<V> &a, const Chan<V> &s) {
    const Chan<V> rest = fma_n(s, all<V>(-1.f), all<V>(1.f));
    return mul_n(s, fma_n(a, rest, all<V>(1.f)));
}

// ---- copies into shared memory, each thread waiting for its own ----------------------------------

template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(BYTES) : "memory");
}
// `bytes` of 16, 16-byte aligned, and zeros behind them.
__device__ __forceinline__ void copy_async_part(void *dst, const void *src, int bytes) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of copies have landed.
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace rows
}  // namespace fw
