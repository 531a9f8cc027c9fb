// lq_act.cuh -- activations' types and functions shared by the recurrent
// layer's kernels: 1- and 8-element loads and stores of f32 / bf16 / f16 rows
// as floats, SiLU / sigmoid / softplus, and the walk over a batch's rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "lq_layer.h"

namespace lq {

using bf16 = __nv_bfloat16;
using f16 = __half;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<bf16>(bf16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f<f16>(f16 v) { return __half2float(v); }

// Round to nearest even: the one rounding an output takes.
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ f16 from_f<f16>(float v) { return __float2half_rn(v); }

// V consecutive elements as stored (V = 8 and 4: vector accesses, V = 1: one element).
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void store(T *p) const { *p = v; }
    __device__ __forceinline__ void zero() { v = from_f<T>(0.0f); }
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f<T>(v); }
    __device__ __forceinline__ void set(const float (&f)[1]) { v = from_f<T>(f[0]); }
};
template <>
struct Raw<float, 4> {
    float4 a;
    __device__ __forceinline__ void load(const float *p) { a = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; }
    __device__ __forceinline__ void set(const float (&f)[4]) { a = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Raw<bf16, 4> {
    uint2 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint2 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(a.x << 16);
        f[1] = __uint_as_float(a.x & 0xffff0000u);
        f[2] = __uint_as_float(a.y << 16);
        f[3] = __uint_as_float(a.y & 0xffff0000u);
    }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[0], f[1]), q = __floats2bfloat162_rn(f[2], f[3]);
        a = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
    }
};
template <>
struct Raw<f16, 4> {
    uint2 a;
    __device__ __forceinline__ void load(const f16 *p) { a = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void store(f16 *p) const { *reinterpret_cast<uint2 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[4]) const {
        const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&a.x));
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&a.y));
        f[0] = u.x; f[1] = u.y; f[2] = v.x; f[3] = v.y;
    }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        const __half2 p = __floats2half2_rn(f[0], f[1]), q = __floats2half2_rn(f[2], f[3]);
        a = make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
    }
};
template <>
struct Raw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Raw<bf16, 8> {
    uint4 a;
    __device__ __forceinline__ void load(const bf16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(bf16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Raw<f16, 8> {
    uint4 a;
    __device__ __forceinline__ void load(const f16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void store(f16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// sigmoid(x): EXACT takes the IEEE-accurate exponential and division (f32
// outputs); otherwise the hardware exponential and reciprocal, about 2^-21
// relative, far below a 16-bit output's half step.  At the ends: exp(-x) = inf
// gives 0, x = -inf gives 0, NaN stays NaN.
template <bool EXACT>
__device__ __forceinline__ float sigmoid_f(float x) {
    if constexpr (EXACT) return 1.0f / (1.0f + expf(-x));
    return __fdividef(1.0f, 1.0f + __expf(-x));
}

template <bool EXACT>
__device__ __forceinline__ float silu_f(float x) {
    if constexpr (EXACT) return x / (1.0f + expf(-x));
    return x * sigmoid_f<false>(x);
}

__device__ __forceinline__ float ex2_f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_f(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two at once, the products and the sum as packed instructions.
template <bool EXACT>
__device__ __forceinline__ float2 silu2_f(float2 x) {
    if constexpr (EXACT) return make_float2(silu_f<true>(x.x), silu_f<true>(x.y));
    const float l = -1.4426950408889634f;
    const float2 t = __fmul2_rn(x, make_float2(l, l));
    const float2 d = __fadd2_rn(make_float2(ex2_f(t.x), ex2_f(t.y)), make_float2(1.0f, 1.0f));
    return __fmul2_rn(x, make_float2(rcp_f(d.x), rcp_f(d.y)));
}

// log(1 + e^x) without overflow: max(x, 0) + log1p(e^-|x|).  A NaN passes
// through (fmaxf alone would drop it).
__device__ __forceinline__ float softplus_f(float x) {
    return x != x ? x : fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x)));
}

// Pieces of SEG tokens of a batch of ragged sequences, numbered without a host
// copy of the lengths: sequence b's pieces are floor(cu[b] / SEG) + b + j,
// j < max(1, ceil(len / SEG)).  The numbers are disjoint, since
// floor((c + l) / SEG) + 1 >= floor(c / SEG) + ceil(l / SEG), and below
// rows / SEG + B.  Offsets are clamped to [0, rows] and to a non-decreasing
// order with the one before, so that a bad array reads and writes inside the
// rows.  Returns false for a number no piece has.
struct Piece {
    int b;        // sequence
    int j;        // piece of the sequence
    int len;      // the sequence's tokens
    int n;        // pieces of the sequence
    int64_t row0, step;   // row of token t: row0 + t * step
    int64_t id;           // its number
};

__device__ __forceinline__ int cu_at(const Rows &r, int i) { return min(max(r.cu[i], 0), r.rows); }

// The last sequence b with floor(cu[b] / seg) + add b <= id (0 if none): each
// lane of the warp probes one of 32 places of what is left, so B sequences
// take log32(B) dependent loads.  All lanes call it with the same arguments.
__device__ __forceinline__ int last_sequence(const Rows &r, int seg, int add, int id) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = r.B;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool le = at < lo + n && cu_at(r, at) / seg + add * at <= id;
        const int k = 31 - __clz((int)(__ballot_sync(0xffffffffu, le) | 1u));
        const int end = lo + n;
        lo += k * step;
        n = min(step, end - lo);
    }
    return lo;
}

// Sequence b's pieces, and the first of them.
__device__ __forceinline__ int pieces_of(const Rows &r, int seg, int b) {
    const int len = r.cu ? cu_at(r, b + 1) - cu_at(r, b) : r.rows / r.B;
    return len > seg ? (len + seg - 1) / seg : 1;
}
__device__ __forceinline__ int64_t first_piece(const Rows &r, int seg, int b) {
    return r.cu ? cu_at(r, b) / seg + b : (int64_t)b * pieces_of(r, seg, b);
}

// (Called by whole warps, every lane with the same id.)
__device__ __forceinline__ bool find_piece(const Rows &r, int seg, int id, Piece &p) {
    p.id = id;
    if (!r.cu) {
        p.len = r.rows / r.B;
        p.n = max(1, (p.len + seg - 1) / seg);
        p.b = id / p.n;
        p.j = id - p.b * p.n;
        p.row0 = p.b;
        p.step = r.B;
        return p.b < r.B;
    }
    const int b = last_sequence(r, seg, 1, id);
    const int c0 = cu_at(r, b), c1 = max(cu_at(r, b + 1), c0);
    p.b = b;
    p.j = id - (c0 / seg + b);
    p.len = c1 - c0;
    p.n = max(1, (p.len + seg - 1) / seg);
    p.row0 = c0;
    p.step = 1;
    return p.j >= 0 && p.j < p.n;
}

// The k-th place where a sequence may be cut: piece j of a sequence whose piece
// j + 1 exists.  Sequence b's are floor(cu[b] / seg) + j, j < n - 1, disjoint as
// above, below rows / seg.
__device__ __forceinline__ bool find_cut(const Rows &r, int seg, int k, Piece &p) {
    if (!r.cu) {
        const int cuts = (r.rows / r.B - 1) / seg;
        const int b = k / cuts;
        return b < r.B && find_piece(r, seg, b * (cuts + 1) + k % cuts, p);
    }
    const int b = last_sequence(r, seg, 0, k);
    const int c0 = cu_at(r, b), c1 = max(cu_at(r, b + 1), c0);
    p.b = b;
    p.j = k - c0 / seg;
    p.id = k + b;
    p.len = c1 - c0;
    p.n = max(1, (p.len + seg - 1) / seg);
    p.row0 = c0;
    p.step = 1;
    return p.j >= 0 && p.j < p.n - 1;
}

__host__ __device__ inline int64_t piece_count(const Rows &r, int seg) {
    if (r.cu) return (int64_t)(r.rows / seg) + r.B;
    const int T = r.rows / r.B;
    return (int64_t)r.B * (T > 0 ? ((int64_t)T + seg - 1) / seg : 1);
}

inline int64_t cut_count(const Rows &r, int seg) {
    if (r.cu) return r.rows / seg;
    const int T = r.rows / r.B;
    return T > seg ? (int64_t)r.B * ((T - 1) / seg) : 0;
}

}  // namespace lq
