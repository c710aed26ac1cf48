// seq_common.cuh -- device helpers of the token-sequence operators (convolution, selective scan,
// norms around a block).
#pragma once

#include "gspn_common.cuh"
#include "gspn_internal.h"
#include "gspn_seq.h"

namespace gspn {
namespace seq {

// ------------------------------------------------------------------ vectors of 16 bytes
// V consecutive elements (8 bf16 or 4 fp32). `n` of them exist; the rest read as zero and are not
// written. `wide` (uniform) says that whole vectors are 16-byte aligned: otherwise, and at a ragged
// end, elements go one by one.
template <typename T> struct Vec { static constexpr int V = 16 / sizeof(T); };

template <typename T>
__device__ __forceinline__ uint4 ld_raw(const T* p, int n, bool wide) {
    constexpr int V = Vec<T>::V;
    if (wide && n >= V) return *(const uint4*)p;
    uint4 q = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 4) {
        const uint32_t* s = (const uint32_t*)p;
        if (n > 0) q.x = s[0];
        if (n > 1) q.y = s[1];
        if (n > 2) q.z = s[2];
        if (n > 3) q.w = s[3];
    } else {
        const uint16_t* s = (const uint16_t*)p;
        auto two = [&](int i) { return (n > i ? (uint32_t)s[i] : 0u) | (n > i + 1 ? (uint32_t)s[i + 1] << 16 : 0u); };
        q.x = two(0); q.y = two(2); q.z = two(4); q.w = two(6);
    }
    return q;
}

template <typename T>
__device__ __forceinline__ void unpack_raw(const uint4& q, float (&v)[Vec<T>::V]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
        v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);          // bf16 is the upper half of an fp32
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
}

// Four consecutive elements, as stored.
template <typename T> struct Quad;
template <> struct Quad<float> { typedef uint4 raw; };
template <> struct Quad<__nv_bfloat16> { typedef uint2 raw; };

__device__ __forceinline__ uint4 ld_quad(const float* p, int n, bool wide) { return ld_raw<float>(p, n, wide); }
__device__ __forceinline__ uint2 ld_quad(const __nv_bfloat16* p, int n, bool wide) {
    if (wide && n >= 4) return *(const uint2*)p;
    const uint16_t* s = (const uint16_t*)p;
    auto two = [&](int i) { return (n > i ? (uint32_t)s[i] : 0u) | (n > i + 1 ? (uint32_t)s[i + 1] << 16 : 0u); };
    return make_uint2(two(0), two(2));
}
__device__ __forceinline__ void unpack_quad(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack_quad(const uint2& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ void st_quad(T* p, const float (&v)[4], int n, bool wide) {
    if (wide && n >= 4) {
        st_lanes<T, 4>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) Io<T>::st(p + i, v[i]);
    }
}

// ------------------------------------------------------------------ functions
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Dynamic shared memory that kernels over 48 KB are allowed: the same for every call, since calls at once would
// set each other's limit.
constexpr int kMostSmem = 224 * 1024;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// exp(-v) may overflow to infinity, where the quotient is the right 0. The exponential's argument is
// rounded once, which puts an error of |v| / 2^24 into it.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(v * -kLog2e)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
// d/dv silu = s + v s (1 - s)
__device__ __forceinline__ float silu_slope(float v) {
    const float s = sigmoid(v);
    return fmaf(v * s, 1.f - s, s);
}

// ------------------------------------------------------------------ pairs
// Two fp32 values in one 64-bit register pair: one instruction does both, with the same roundings as
// two scalar ones. Where issue slots bound a kernel, this halves its multiplies and adds.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    const float2 s = unpack(v);
    return pack(ex2(s.x), ex2(s.y));
}
__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
// The larger of the two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 sigmoid2(f2 v) {
    const float2 e = unpack(add2(ex2_2(mul2(v, both(-kLog2e))), both(1.f)));
    return pack(rcp(e.x), rcp(e.y));
}
__device__ __forceinline__ f2 silu2(f2 v) { return mul2(v, sigmoid2(v)); }
__device__ __forceinline__ f2 silu_slope2(f2 v) {
    const f2 s = sigmoid2(v);
    return fma2(mul2(v, s), fma2(s, both(-1.f), both(1.f)), s);
}
// Four floats of shared memory (16-byte aligned) as two pairs.
__device__ __forceinline__ void ld_pairs(const float* p, f2& a, f2& b) {
    const ulonglong2 q = *(const ulonglong2*)p;
    a = q.x;
    b = q.y;
}

// V elements as stored (16 bytes), or four of them, as pairs.
template <int P>
__device__ __forceinline__ void to_pairs(const uint4& q, f2 (&v)[P]) {
    static_assert(P == 2 || P == 4, "four fp32 or eight bf16");
    if constexpr (P == 2) {
        v[0] = pack(__uint_as_float(q.x), __uint_as_float(q.y));
        v[1] = pack(__uint_as_float(q.z), __uint_as_float(q.w));
    } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    }
}
__device__ __forceinline__ void to_pairs(const uint2& q, f2 (&v)[2]) {
    v[0] = pack(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
    v[1] = pack(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
}
template <int P>
__device__ __forceinline__ void to_floats(const f2 (&v)[P], float (&o)[2 * P]) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
        const float2 f = unpack(v[k]);
        o[2 * k] = f.x;
        o[2 * k + 1] = f.y;
    }
}

// ------------------------------------------------------------------ sequences
// Where sequence q lies: its row, first token and length. Entries of cu are clamped to the row, so
// no value of them leads out of bounds.
struct Span {
    int row, first, len;
};
__device__ __forceinline__ Span span_of(const int* cu, int q, int L) {
    if (!cu) return Span{q, 0, L};
    const int a = min(max(cu[q], 0), L), b = min(max(cu[q + 1], a), L);
    return Span{0, a, b - a};
}

inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline size_t dtype_size(int dtype) { return dtype == GSPN_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == GSPN_F32 || dtype == GSPN_BF16; }
// True where every vector of an input with these strides is 16-byte aligned.
inline bool wide_ok(const void* p, long long row, long long tok, size_t es) {
    return aligned_to(p, 16) && (row * (long long)es) % 16 == 0 && (tok * (long long)es) % 16 == 0;
}
inline gspn_status last_status() { return cudaGetLastError() == cudaSuccess ? GSPN_OK : GSPN_ERR_CUDA; }

}  // namespace seq
}  // namespace gspn
