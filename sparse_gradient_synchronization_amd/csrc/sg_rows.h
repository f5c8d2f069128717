// sg_rows.h -- device helpers of the vocabulary operators: rows of logits
// read as 16-byte chunks, and the running maximum and sum of a softmax.
//
// A row is V elements of fp32 or bf16 that start anywhere: rows of an odd
// vocabulary are only element-aligned.  gfx950 loads and stores 16 bytes at
// any address, but a wave's unaligned kilobyte touches one more cache line
// than it fills: reading 3000 rows of 100003 bf16 ran at 4.9 TB/s that way
// and at 6.2 TB/s with rows that start on 16 bytes.  So the chunks of a row
// start at its first 16-byte boundary, `head` elements in; the elements
// before it and after the last whole chunk are handled one by one.
#pragma once
#include "sg_device.h"

namespace sg {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2))); // anywhere an element may be

// log2(e) * inv_temp in fp32, and the rest of it.  With the first alone every
// log-probability of a batch is off by the same small share (1.3e-8 at
// temperature 1) of its distance from the row's mean.  That is lost in the
// rounding of a result per token, and there the row's scalars take the
// temperature that hi stands for; but the preference loss adds thousands of
// them and takes differences (an IPO loss of 12000 tokens was 3e-4 off), so
// its sums are FINE and use both parts, an fma more a term.
struct Scale {
    float hi, lo; // FINE: lo > 0, so that -inf times it stays -inf
};

struct Rows {
    const void* x; // [T] rows, ld elements apart
    uint64_t T, ld;
    uint64_t row0; // first row of this launch
    uint32_t V;
    Scale c;   // exp(inv_temp * d) = exp2(c * d)
    double it; // inv_temp; not FINE: that of c.hi
};

// the chunks of one row
struct RowSpan {
    uint32_t head, nc, V; // first element of chunk 0, whole chunks, elements
};

// BYTES: where the chunks start, 16 or a cache line's 128
template <int BYTES = 16, typename E>
__device__ __forceinline__ RowSpan span_of(const E* x, uint32_t V)
{
    constexpr uint32_t VEC = 16 / sizeof(E);
    RowSpan s;
    s.head = (uint32_t)(-(reinterpret_cast<uintptr_t>(x) / sizeof(E))) % (BYTES / sizeof(E));
    s.head = s.head < V ? s.head : V;
    s.nc = (V - s.head) / VEC;
    s.V = V;
    return s;
}

// the i-th element outside the chunks, V or more if there is none
__device__ __forceinline__ uint32_t loose_element(const RowSpan& s, uint32_t vec, uint32_t i)
{
    return i < s.head ? i : i + s.nc * vec;
}

// What one pass over (a part of) a row gives: maximum of the raw logits and
// sum of exp2(c * (x - m)); {-inf, 0} for nothing.  The exponentials of a chunk
// are added in fp32 as a tree, chunks and lanes in fp64: a preference loss adds
// the log-probabilities of thousands of tokens, and what fp32 sums lose in a
// row whose largest term dominates is of one sign (1.7e-7 a token).  It costs
// nothing measurable beside the loads.
struct RowStat {
    float m;
    double s;
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
    // the elements of set bits replaced by -inf
    static __device__ __forceinline__ u32x4 without(u32x4 w, uint32_t b)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = b >> i & 1u ? 0xff800000u : w[i];
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
    static __device__ __forceinline__ u32x4 without(u32x4 w, uint32_t b)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = b >> (2 * i) & 1u ? (w[i] & 0xffff0000u) | 0xff80u : w[i];
            w[i] = b >> (2 * i + 1) & 1u ? (w[i] & 0xffffu) | 0xff800000u : w[i];
        }
        return w;
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

// PAST: the store goes past the caches (a template, since the compiler makes
// one ordinary store of two in branches)
template <bool PAST, typename E>
__device__ __forceinline__ void store_chunk(E* p, u32x4 v)
{
    if (PAST) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_at2*>(p));
    else __builtin_memcpy(p, &v, 16);
}

// address of chunk j + j0: j is the same for all lanes, so it goes into a
// scalar base and one 32-bit lane offset serves every chunk of the row
template <typename E, typename P>
__device__ __forceinline__ P* chunk_at(P* x, uint32_t j, uint32_t j0)
{
    return x + (uint64_t)j * RowIO<E>::VEC + j0 * RowIO<E>::VEC;
}

// Chunks j0, j0 + NT, ... of a row with nc > 0 chunks.  Past the row's end the
// last chunk is loaded again: with every load issued on every path, the wait
// for one of them need not be a wait for all (a load in a branch may or may
// not be among those in flight, so the compiler waits until none is).
template <int J, int NT, typename E>
__device__ __forceinline__ void load_chunks(u32x4* w, const E* x, uint32_t j0, uint32_t nc)
{
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t c = j0 + j * NT < nc ? j0 + j * NT : nc - 1;
        w[j] = load_chunk(chunk_at<E>(x, 0, c));
    }
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// exp2(c * d), d <= 0; -inf gives 0.  The small product goes first: added to
// a rounded d * hi it would be rounded away.
template <bool FINE>
__device__ __forceinline__ float exp2_scaled(float d, Scale c)
{
    return exp2_fast(FINE ? fmaf(d, c.hi, d * c.lo) : d * c.hi);
}

// the maximum as it is subtracted: a row (or part) of nothing but -inf has
// exp(-inf - 0) = 0 terms, not exp(-inf + inf)
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.f : m; }

// Adds N values to a running (maximum, sum).  A NaN among them, or a +inf,
// makes the sum NaN; -inf adds nothing.
template <int N, bool FINE = false>
__device__ __forceinline__ void stat_add(RowStat& r, const float* v, Scale c)
{
    float m = r.m;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
    const float sh = shift_of(m);
    float e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) e[i] = exp2_scaled<FINE>(v[i] - sh, c);
#pragma unroll
    for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
        for (int i = 0; i < w; ++i) e[i] += e[i + w];
    r.s = r.s * (double)exp2_scaled<FINE>(r.m - sh, c) + (double)e[0];
    r.m = m;
}

// the parts of every N lanes joined in a fixed order; each of them holds the result
template <int N = SG_WAVE, bool FINE = false>
__device__ __forceinline__ RowStat wave_stat(RowStat r, Scale c)
{
    float m = r.m;
#pragma unroll
    for (int d = 1; d < N; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, SG_WAVE));
    double s = r.s * (double)exp2_scaled<FINE>(r.m - shift_of(m), c);
#pragma unroll
    for (int d = 1; d < N; d <<= 1) s += __shfl_xor(s, d, SG_WAVE);
    return {m, s};
}

constexpr int next_pow2(int n)
{
    int p = 1;
    while (p < n) p *= 2;
    return p;
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int d = 1; d < SG_WAVE; d <<= 1) v += __shfl_xor(v, d, SG_WAVE);
    return v;
}

// exp and log of the row scalars in fp64, from their series: 1e-12 relative
// is plenty for results of 24 bits.  Terms are added one at a time (the
// scheduling barrier): left alone, the compiler loads all constants first,
// into registers that the row held in them has no room for.
template <int N>
__device__ __forceinline__ double series_step(double a, double q, const double (&k)[N])
{
#pragma unroll
    for (int n = N - 1; n >= 0; --n) {
        a = a * q + k[n];
        __builtin_amdgcn_sched_barrier(0);
    }
    return a;
}

constexpr double kLn2 = 0.69314718055994530942, kLn2Lo = 2.3190468138462996e-17; // kLn2 + kLn2Lo = log 2

// exp(r) - 1 for |r| <= 0.35: r + r^2/2! + ... + r^11/11!
__device__ __forceinline__ double row_expm1_small(double r)
{
    constexpr double k[11] = {1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320,
                              1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800};
    return r * series_step(0.0, r, k);
}

__device__ __forceinline__ double row_exp(double x)
{
    const double k = rint(fmin(fmax(x, -1100.0), 1100.0) * (1.0 / kLn2));
    const double r = (x - k * kLn2) - k * kLn2Lo;
    const double y = ldexp(1.0 + row_expm1_small(r), (int)k);
    return x != x ? x : (x < -745.0 ? 0.0 : (x > 709.7 ? (double)INFINITY : y));
}

__device__ __forceinline__ double row_expm1(double x)
{
    return fabs(x) <= 0.34 ? row_expm1_small(x) : row_exp(x) - 1.0;
}

// log(m 2^e) = e log 2 + 2 (s + s^3/3 + s^5/5 + ...), s = (m - 1) / (m + 1), m in [1/sqrt 2, sqrt 2]
__device__ __forceinline__ double row_log(double x)
{
    constexpr double k[9] = {1.0, 1.0 / 3, 1.0 / 5, 1.0 / 7, 1.0 / 9, 1.0 / 11, 1.0 / 13, 1.0 / 15, 1.0 / 17};
    double m = __builtin_amdgcn_frexp_mant(x);
    int e = __builtin_amdgcn_frexp_exp(x);
    if (m < 0.70710678118654752440) {
        m *= 2.0;
        --e;
    }
    const double s = (m - 1.0) / (m + 1.0);
    const double y = e * kLn2 + 2.0 * s * series_step(0.0, s * s, k);
    return x > 0.0 && x < INFINITY ? y : (x == 0.0 ? -(double)INFINITY : x);
}

// log(1 + u) for u in [0, 1]: s = u / (2 + u) is at most 1/3
__device__ __forceinline__ double row_log1p(double u)
{
    constexpr double k[13] = {1.0, 1.0 / 3, 1.0 / 5, 1.0 / 7, 1.0 / 9, 1.0 / 11, 1.0 / 13, 1.0 / 15, 1.0 / 17,
                              1.0 / 19, 1.0 / 21, 1.0 / 23, 1.0 / 25};
    const double s = u / (2.0 + u);
    return 2.0 * s * series_step(0.0, s * s, k);
}

// 1/S with a row of nothing (S = 0) giving 0; a NaN stays
__device__ __forceinline__ double inverse_of(double S) { return S == 0.0 ? 0.0 : 1.0 / S; }

} // namespace sg
