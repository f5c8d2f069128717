// sg_rows.h -- device helpers of the vocabulary operators: rows of logits
// read as 16-byte chunks, and the running maximum and sum of a softmax.
//
// A row is V elements of fp32 or bf16 that start anywhere (rows of an odd
// vocabulary are only element-aligned; gfx950 loads and stores 16 bytes at
// any address).  Chunk j holds elements [j*VEC, (j+1)*VEC); the V % VEC
// elements after the last whole chunk are handled one by one.
#pragma once
#include "sg_device.h"

namespace sg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Rows {
    const void* x; // [T] rows, ld elements apart
    uint64_t T, ld;
    uint32_t V;
    float c;   // exp(inv_temp * d) = exp2(c * d)
    double it; // inv_temp
};

// what one pass over (a part of) a row gives: maximum of the raw logits and
// sum of exp2(c * (x - m)); {-inf, 0} for nothing.  fp32: every thread adds
// at most a few thousand terms of at most 1, and the threads' sums are joined
// as a tree, so the relative error stays near 1e-7.
struct RowStat {
    float m, s;
};

template <typename E>
struct RowIO;

template <>
struct RowIO<float> {
    static constexpr int VEC = 4;
    static __device__ __forceinline__ void unpack(u32x4 w, float* v)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
    }
    static __device__ __forceinline__ u32x4 pack(const float* v)
    {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
        return w;
    }
    static __device__ __forceinline__ float get(const float* p) { return *p; }
    static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};

typedef uint16_t bf16_bits;

template <>
struct RowIO<bf16_bits> {
    static constexpr int VEC = 8;
    static __device__ __forceinline__ void unpack(u32x4 w, float* v)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // rounded to nearest even, once, from the fp32 value
    static __device__ __forceinline__ u32x4 pack(const float* v)
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x2 f = {v[2 * i], v[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
        }
        return w;
    }
    static __device__ __forceinline__ float get(const bf16_bits* p) { return bf16_to_f32(*p); }
    static __device__ __forceinline__ void put(bf16_bits* p, float v)
    {
        *p = __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};

template <typename E>
__device__ __forceinline__ u32x4 load_chunk(const E* p)
{
    u32x4 r;
    __builtin_memcpy(&r, p, 16);
    return r;
}

template <typename E>
__device__ __forceinline__ void store_chunk(E* p, u32x4 v)
{
    __builtin_memcpy(p, &v, 16);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// the maximum as it is subtracted: a row (or part) of nothing but -inf has
// exp(-inf - 0) = 0 terms, not exp(-inf + inf)
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// Adds N values to a running (maximum, sum).  A NaN among them, or a +inf,
// makes the sum NaN; -inf adds nothing.
template <int N>
__device__ __forceinline__ void stat_add(RowStat& r, const float* v, float c)
{
    float m = r.m;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
    const float sh = shift_of(m);
    float s = r.s * exp2_fast((r.m - sh) * c);
#pragma unroll
    for (int i = 0; i < N; ++i) s += exp2_fast((v[i] - sh) * c);
    r.m = m;
    r.s = s;
}

__device__ __forceinline__ RowStat stat_join(RowStat a, RowStat b, float c)
{
    const float m = fmaxf(a.m, b.m), sh = shift_of(m);
    return {m, a.s * exp2_fast((a.m - sh) * c) + b.s * exp2_fast((b.m - sh) * c)};
}

// the lanes' parts joined in a fixed order; every lane holds the result
__device__ __forceinline__ RowStat wave_stat(RowStat r, float c)
{
#pragma unroll
    for (int d = 1; d < SG_WAVE; d <<= 1) {
        RowStat o = {__shfl_xor(r.m, d, SG_WAVE), __shfl_xor(r.s, d, SG_WAVE)};
        // the lower lane's part first on both sides, so both hold the same bits
        r = (lane_id() & d) ? stat_join(o, r, c) : stat_join(r, o, c);
    }
    return r;
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int d = 1; d < SG_WAVE; d <<= 1) v += __shfl_xor(v, d, SG_WAVE);
    return v;
}

// 1/S with a row of nothing (S = 0) giving 0; a NaN stays
__device__ __forceinline__ double inverse_of(double S) { return S == 0.0 ? 0.0 : 1.0 / S; }

} // namespace sg
