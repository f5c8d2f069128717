// sg_linear_ce.hip -- softmax cross entropy of hidden states against a
// vocabulary head, with both gradients, without the logits in memory:
//   z_tv = x_t . w_v / temperature,  lse_t = log sum_v exp z_tv
//   loss_t = weight_t (lse_t - z_ty + zc lse_t^2)
//   g_tv = weight_t / temperature ((1 + 2 zc lse_t) exp(z_tv - lse_t) - 1[v = y_t])
//   dx = g w,  dw = g^T x
//
// Three products of 2 T V H operations bound it for more than a few hundred
// rows; below that the head is read and its gradient written.
//
// The rows that count are gathered first, so every product runs over them
// alone (their number stays on the device: a block past it ends at once).
// What goes from the first product to the other two:
//   - per row and tile of the vocabulary the maximum and the sum of the
//     exponentials, from the sums in registers; a row's are joined in fp64
//   - the exponentials themselves, relative to their tile's maximum, in 16
//     bits, while T x V of them fit in keep_bytes; a pass over them then makes
//     g in place.  Otherwise the vocabulary is taken in pieces that fit, each
//     with a second product of the logits that ends in g: 8 T V H operations
//     instead of 6.
// 16 bits for a number in [0, 1]: no sign, 6 bits of exponent (down to
// 2^-63) and 10 of mantissa, so that keeping them (2^-12) adds little to the
// one rounding of g to bf16 (2^-9) that the matrix instructions ask for.
//
// fp32: hidden states, head and g are two fp16 planes each under one power of
// two per tensor (sg_gemm.h), which loses 2^-22 of each element down to 2^-17
// of the tensor's largest and an absolute 2^-39 of it below.  The kept
// exponentials are whole fp32 there, in the two planes of g.
#include <type_traits>

#include "sg_gemm.h"
#include "sg_rows.h"

namespace sg {

// what the joined sums leave for a live row
struct CeRow {
    float m;    // maximum logit, before the temperature
    float ls;   // log2 of the sum of exp2(c (x - m))
    float a, b; // g = top (a p - b 1[v = y])
};

struct CeScal { // power-of-two scales of the fp32 planes and their inverses
    uint32_t max_x, max_w, max_g; // bits of the largest finite magnitudes
    uint32_t live;                // rows that count
    // largest finite |weight / temperature| of the live rows: g is kept relative to it,
    // so that with equal weights the label's -1 is a bf16 number and not 1 / N rounded
    double top;
};

// the power of two that brings a largest magnitude to [2^12, 2^13)
__device__ __forceinline__ int ce_exponent(uint32_t bits)
{
    const int e = (int)(bits >> 23 & 255) - 127;
    return 12 - (e < -126 ? -126 : e);
}

struct CeArgs {
    const int32_t* label;
    const float* weight;
    float *loss, *lse;
    uint64_t T;
    uint32_t V;
    double it, zc;
    float c; // log2(e) / temperature
};

// The rows that count, in order, by the NT threads of a block: list[j] (LDS, or
// NULL).  write: row[j], pos[t] = j or -1, the call's scalars, and 0 for the other
// rows' losses.  Returns how many there are.
template <int NT>
__device__ __forceinline__ uint32_t ce_gather(const CeArgs& p, bool write, uint32_t* list, uint32_t* row, int32_t* pos,
                                              CeScal* scal)
{
    __shared__ uint32_t count[NT / 64];
    __shared__ float most[NT / 64];
    uint32_t done = 0;
    float top = 0.f;
    const uint32_t w = threadIdx.x / 64;
    for (uint64_t t0 = 0; t0 < p.T; t0 += NT) {
        const uint64_t t = t0 + threadIdx.x;
        bool live = false;
        if (t < p.T) {
            const int32_t y = p.label[t];
            const float wt = p.weight ? p.weight[t] : 1.f;
            live = y >= 0 && (uint32_t)y < p.V && wt != 0.f;
            if (live && fabsf(wt) < INFINITY) top = fmaxf(top, fabsf(wt));
        }
        const uint64_t b = ballot(live);
        __syncthreads();
        if (threadIdx.x % 64 == 0) count[w] = popc64(b);
        __syncthreads();
        uint32_t before = done, all = 0;
        for (uint32_t i = 0; i < NT / 64; ++i) {
            before += i < w ? count[i] : 0;
            all += count[i];
        }
        done += all;
        const uint32_t j = before + count_below(b);
        if (live && list) list[j] = (uint32_t)t;
        if (live && write) row[j] = (uint32_t)t;
        if (t < p.T && write) {
            pos[t] = live ? (int32_t)j : -1;
            if (!live) {
                p.loss[t] = 0.f;
                if (p.lse) p.lse[t] = 0.f;
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x % 64 == 0) most[w] = top;
    __syncthreads(); // the list is whole, too
    if (threadIdx.x == 0 && write) {
        for (int i = 0; i < NT / 64; ++i) top = fmaxf(top, most[i]);
        *scal = {0u, 0u, 0u, done, (double)top * p.it};
    }
    return done;
}

// one block: T labels are little
__global__ __launch_bounds__(1024) void ce_rows_kernel(CeArgs p, uint32_t* row, int32_t* pos, CeScal* scal)
{
    ce_gather<1024>(p, true, nullptr, row, pos, scal);
}

// rows of a user's matrix
struct CeSrc {
    const void* x;
    uint64_t ld;
    uint32_t n; // elements of a row
};
template <typename E>
__device__ __forceinline__ void ce_load8(const CeSrc& s, uint64_t r, uint32_t c, float* v)
{
    const E* x = static_cast<const E*>(s.x) + r * s.ld + c;
    if (c + 8 <= s.n) { // gfx950 loads 16 bytes at any element's address
        constexpr int VEC = RowIO<E>::VEC;
#pragma unroll
        for (int i = 0; i < 8; i += VEC) RowIO<E>::unpack(load_chunk(x + i), v + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < s.n ? RowIO<E>::get(x + i) : 0.f;
}

// items of `per` a row; most are few enough for a 32-bit division
struct CeItems {
    uint64_t n;
    uint32_t per;
    __device__ __forceinline__ CeItems(uint64_t n_, uint32_t per_) : n(n_), per(per_) {}
    __device__ __forceinline__ void split(uint64_t i, uint64_t* row, uint32_t* at) const
    {
        if (n <= 0xffffffffull) {
            *row = (uint32_t)i / per;
            *at = (uint32_t)i - (uint32_t)*row * per;
        } else {
            *row = i / per;
            *at = (uint32_t)(i - *row * per);
        }
    }
};

// One of the two matrices that a kernel takes in one launch, and its blocks
struct CeSide {
    CeSrc s;
    uint64_t rows;
    const uint32_t* row; // the live ones, NULL: all
    uint32_t* max_bits;
    uint16_t *hi, *lo;
    uint32_t blocks;
};

// the largest finite magnitudes of the rows; one row's infinity or NaN leaves the
// others their precision
__global__ __launch_bounds__(256) void ce_max_kernel(CeSide x, CeSide w, const CeScal* scal)
{
    const bool first = blockIdx.x < x.blocks;
    const CeSide& side = first ? x : w;
    const CeSrc s = side.s;
    const uint32_t* const row = side.row;
    uint32_t* const out = side.max_bits;
    const uint32_t block = first ? blockIdx.x : blockIdx.x - x.blocks, blocks = side.blocks;
    const uint64_t n = row ? scal->live : side.rows;
    const uint32_t per = (s.n + 7) / 8;
    const CeItems items(n * per, per);
    uint32_t m = 0;
    for (uint64_t i0 = block * 256ull + threadIdx.x; i0 < items.n; i0 += blocks * 1024ull) {
        float v[4][8]; // four loads of 32 bytes under way
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint64_t i = i0 + u * blocks * 256ull, r;
            uint32_t c;
            items.split(i < items.n ? i : i0, &r, &c);
            ce_load8<float>(s, row ? row[r] : r, c * 8, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t b = __float_as_uint(v[u][k]) & 0x7fffffffu;
                m = b > m && b < 0x7f800000u ? b : m;
            }
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_xor(m, d);
        m = o > m ? o : m;
    }
    // a maximum of whole numbers: the order of the blocks does not matter
    if (threadIdx.x % 64 == 0 && m > *(volatile uint32_t*)out) atomicMax(out, m);
}

// Rows as planes: gathered (row != NULL; rows up to the next multiple of 64 are
// zeros), columns padded with zeros to np.  GATHER (up to CE_GATHER rows): every
// block of the hidden states finds the live rows itself, the first one writes them.
constexpr uint32_t CE_GATHER = 1024;
template <typename E, bool GATHER>
__global__ __launch_bounds__(256) void ce_pack_kernel(CeSide x, CeSide w, CeScal* scal, uint32_t np, CeArgs p,
                                                      uint32_t* rows_out, int32_t* pos)
{
    __shared__ uint32_t list[GATHER ? CE_GATHER : 1];
    const bool first = blockIdx.x < x.blocks;
    const CeSide& side = first ? x : w;
    const CeSrc s = side.s;
    const uint32_t* const row = side.row;
    uint16_t *const hi = side.hi, *const lo = side.lo;
    const uint32_t block = first ? blockIdx.x : blockIdx.x - x.blocks, blocks = side.blocks;
    uint64_t n = side.rows;
    if (GATHER && first) n = ce_gather<256>(p, blockIdx.x == 0, list, rows_out, pos, scal);
    else if (row) n = scal->live;
    const uint64_t padded = row ? (n + 63) / 64 * 64 : n;
    const uint32_t per = np / 8;
    const int e = lo ? ce_exponent(*side.max_bits) : 0;
    const CeItems items(padded * per, per);
    for (uint64_t i = block * 256ull + threadIdx.x; i < items.n; i += blocks * 256ull) {
        uint64_t r;
        uint32_t c;
        items.split(i, &r, &c);
        c *= 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < n && c < s.n) ce_load8<E>(s, !row ? r : GATHER ? list[r] : row[r], c, v);
        if (lo) {
            s16x8 h, l;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint16_t x, y;
                split_f16(ldexpf(v[k], e), &x, &y);
                h[k] = (short)x;
                l[k] = (short)y;
            }
            *reinterpret_cast<s16x8*>(hi + r * np + c) = h;
            *reinterpret_cast<s16x8*>(lo + r * np + c) = l;
        } else {
            *reinterpret_cast<u32x4*>(hi + r * np + c) = RowIO<bf16_bits>::pack(v);
        }
    }
}

// a number in [0, 1] in 16 bits, and back; below 2^-63 it is 0
__device__ __forceinline__ uint16_t ce_code(float e)
{
    const int b = (int)__float_as_uint(e) - (0x20000000 - 0x1000);
    return (uint16_t)((b > 0 ? b : 0) >> 13);
}
__device__ __forceinline__ float ce_decode(uint32_t code)
{
    return code ? __uint_as_float((code << 13) + 0x20000000u) : 0.f;
}

// g and the exponentials it comes from: panels of 256 tokens, in each the rows' 256
// one after another.  As rows of a vocabulary, a tile's rows lay on as many pages:
// 8192 x 131072 x 4096, 10% masked, took 6.38 + 6.25 + 6.07 ms for the three products and
// takes 6.22 + 6.22 + 5.97 with panels.
struct CeG {
    uint16_t *hi, *lo;
    uint64_t rows; // of a panel
    __device__ __forceinline__ uint64_t at(uint32_t m, uint32_t n) const { return (n / 256 * rows + m) * 256 + n % 256; }
};

// Where the logits' products end the first time: the rows' statistics over the
// block's columns, the labels' logits, and (g.hi) the exponentials.
template <bool PLANES>
struct CeLogitsEpi {
    const uint32_t* row;
    const int32_t* label;
    const CeScal* scal;
    float2* stat; // [rows][groups]
    float* zy;    // [rows] the label's logit
    CeG g;        // hi NULL: keep nothing
    uint32_t groups, Vp; // Vp: columns of g
    float c;

    template <class Cfg>
    __device__ __forceinline__ void run(f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        const int unit = PLANES ? -ce_exponent(scal->max_x) - ce_exponent(scal->max_w) : 0;
        float mx[Cfg::MT], sum[Cfg::MT];
        uint32_t y[Cfg::MT]; // the row's label as a column of the wave's part
        float* const lm = reinterpret_cast<float*>(at.lds); // [WN][BM]
        float* const ls = lm + Cfg::WN * Cfg::BM;
        const uint32_t last = at.M - 1;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t m = at.m0 + i * 16 + l % 16;
            y[i] = row[m < at.M ? m : last];
        }
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) y[i] = (uint32_t)label[y[i]] - at.n0;
        if (PLANES) {
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[i][j][k] = ldexpf(acc[i][j][k], unit);
        }
        if (at.n0 + Cfg::NTT * 16 > at.N) { // columns past the vocabulary's end
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (at.n0 + j * 16 + l / 16 * 4 + k >= at.N) acc[i][j][k] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            // few tiles hold a label of their rows
            const uint32_t mine = y[i] - l / 16 * 4; // 16 j + k where this lane holds it
            if (__any(y[i] < Cfg::NTT * 16)) {
                float z = 0.f;
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) z = mine == j * 16u + k ? acc[i][j][k] : z;
                if (mine < Cfg::NTT * 16u && mine % 16 < 4 && at.m0 + i * 16 + l % 16 < at.M)
                    zy[at.m0 + i * 16 + l % 16] = z;
            }
            mx[i] = -INFINITY;
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j)
                mx[i] = fmaxf(mx[i], fmaxf(fmaxf(acc[i][j][0], acc[i][j][1]), fmaxf(acc[i][j][2], acc[i][j][3])));
            mx[i] = fmaxf(mx[i], __shfl_xor(mx[i], 16));
            mx[i] = fmaxf(mx[i], __shfl_xor(mx[i], 32));
            if (l < 16) lm[at.wn * Cfg::BM + at.m0 - at.bm0 + i * 16 + l] = mx[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t q = at.m0 - at.bm0 + i * 16 + l % 16;
#pragma unroll
            for (int w = 0; w < Cfg::WN; ++w) mx[i] = fmaxf(mx[i], lm[w * Cfg::BM + q]);
            const float shift = shift_of(mx[i]);
            sum[i] = 0.f;
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[i][j][k] = exp2_fast(c * (acc[i][j][k] - shift));
                sum[i] += (acc[i][j][0] + acc[i][j][1]) + (acc[i][j][2] + acc[i][j][3]);
            }
            sum[i] += __shfl_xor(sum[i], 16);
            sum[i] += __shfl_xor(sum[i], 32);
            if (l < 16) ls[at.wn * Cfg::BM + q] = sum[i];
        }
        __syncthreads();
        if (at.wn == 0 && l < 16) {
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i) {
                const uint32_t q = at.m0 - at.bm0 + i * 16 + l;
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < Cfg::WN; ++w) s += ls[w * Cfg::BM + q];
                if (at.bm0 + q < at.M)
                    stat[(uint64_t)(at.bm0 + q) * groups + at.bn0 / Cfg::BN] = make_float2(mx[i], s);
            }
        }
        if (g.hi) keep<Cfg>(acc, at);
    }
    // the exponentials, a plane after another through LDS (the statistics lie there until they are written)
    template <class Cfg>
    __device__ __forceinline__ void keep(const f32x4 (&e)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        typedef TileRows<Cfg> Rows;
        const auto put = [&](uint16_t* out, auto low) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    s16x4 w;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t bits = __float_as_uint(e[i][j][k]);
                        w[k] = (short)(!PLANES ? ce_code(e[i][j][k]) : decltype(low)::value ? bits : bits >> 16);
                    }
                    Rows::put(at.lds, at.m0 - at.bm0 + i * 16 + l % 16, at.n0 - at.bn0 + j * 16 + l / 16 * 4, w);
                }
            __syncthreads();
            Rows::each(at.lds, [&](uint32_t m, uint32_t n, s16x8 v) {
                if (at.bm0 + m < at.M && at.bn0 + n < Vp)
                    *reinterpret_cast<s16x8*>(out + g.at(at.bm0 + m, at.bn0 + n)) = v;
            });
        };
        put(g.hi, std::false_type());
        if (PLANES) put(g.lo, std::true_type());
    }
};

// The second time, for a piece of the vocabulary: g from the joined sums.
template <bool PLANES>
struct CePieceEpi {
    const uint32_t* row;
    const int32_t* label;
    const CeScal* scal;
    const CeRow* info;
    CeG g;
    uint32_t v0, Vp; // first token of the piece; columns of g
    float c;

    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64, last = at.M - 1;
        const int unit = PLANES ? -ce_exponent(scal->max_x) - ce_exponent(scal->max_w) : 0;
        const int gexp = PLANES ? ce_exponent(scal->max_g) : 0;
        uint32_t y[Cfg::MT];
        CeRow r[Cfg::MT];
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t m = at.m0 + i * 16 + l % 16;
            y[i] = row[m < at.M ? m : last];
            r[i] = info[m < at.M ? m : last];
        }
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) y[i] = (uint32_t)label[y[i]] - v0;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
                const uint32_t m = at.m0 + i * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
                s16x4 h, q;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float z = PLANES ? ldexpf(acc[i][j][k], unit) : acc[i][j][k];
                    const float e = n + k < at.N ? r[i].a * exp2_fast(c * (z - r[i].m) - r[i].ls) : 0.f;
                    const float v = e - (n + k == y[i] ? r[i].b : 0.f);
                    if (PLANES) {
                        uint16_t a, b;
                        split_f16(ldexpf(v, gexp), &a, &b);
                        h[k] = (short)a;
                        q[k] = (short)b;
                    } else {
                        h[k] = __builtin_bit_cast(short, (__bf16)v);
                    }
                }
                if (m >= at.M || n >= Vp) continue;
                *reinterpret_cast<s16x4*>(g.hi + g.at(m, n)) = h;
                if (PLANES) *reinterpret_cast<s16x4*>(g.lo + g.at(m, n)) = q;
            }
    }
};

// loss, lse (write) and what g needs of live row t from its joined sums
__device__ __forceinline__ CeRow ce_finish(const CeArgs& p, uint32_t t, float shift, double s, float zy, double top,
                                           bool write)
{
    const double w = p.weight ? (double)p.weight[t] : 1.0, lse = p.it * (double)shift + log(s);
    if (write) {
        p.loss[t] = (float)(w * (lse - p.it * (double)zy + p.zc * lse * lse));
        if (p.lse) p.lse[t] = (float)lse;
    }
    const double b = w * p.it / top;
    return {shift, (float)log2(s), (float)(b * (1.0 + 2.0 * p.zc * lse)), (float)b};
}

// A live row's statistics joined.  A block a row.
__global__ __launch_bounds__(256) void ce_join_kernel(CeArgs p, const uint32_t* row, const float2* stat,
                                                      uint32_t groups, const float* zy, CeRow* info, CeScal* scal,
                                                      bool planes)
{
    const uint32_t j = blockIdx.x;
    if (j >= scal->live) return;
    __shared__ float sm[4];
    __shared__ double ss[4];
    float m = -INFINITY;
    for (uint32_t i = threadIdx.x; i < groups; i += 256) m = fmaxf(m, stat[(uint64_t)j * groups + i].x);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    if (threadIdx.x % 64 == 0) sm[threadIdx.x / 64] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float shift = shift_of(m);
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < groups; i += 256) {
        const float2 q = stat[(uint64_t)j * groups + i];
        s += (double)q.y * exp2_fast(p.c * (q.x - shift)); // q.x = -inf: its sum is 0, its factor 0
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (threadIdx.x % 64 == 0) ss[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = ss[0] + ss[1] + ss[2] + ss[3];
    const CeRow r = ce_finish(p, row[j], shift, s, zy[j], scal->top, true);
    if (!info) return;
    info[j] = r;
    // A maximum of whole numbers: the order of the rows does not matter.  Looked at first: with equal weights
    // most rows have nothing to add, and as many atomics on one word took 12 ns each (4088 rows: 50 us).
    const uint32_t big = __float_as_uint(fmaxf(fabsf(r.a), fabsf(r.b)));
    if (planes && big < 0x7f800000u && big > *(volatile uint32_t*)&scal->max_g) atomicMax(&scal->max_g, big);
}

// kept exponentials -> g, in place; rows up to the next multiple of 64 are
// zeros.  A block takes 8 rows of a panel.  JOIN: it joins its rows' statistics
// itself, the first panel's blocks write loss and lse.
template <bool JOIN>
__global__ __launch_bounds__(256) void ce_grad_kernel(CeArgs p, const uint32_t* row, const float2* stat,
                                                      uint32_t groups, uint32_t group_cols, const float* zy,
                                                      const CeRow* info, const CeScal* scal, CeG g)
{
    const uint32_t per = (uint32_t)(g.rows / 8), v0 = blockIdx.x / per * 256 + threadIdx.x % 32 * 8;
    const uint32_t j = blockIdx.x % per * 8 + threadIdx.x / 32, live = scal->live;
    if (j >= (live + 63) / 64 * 64) return;
    u32x4* const hi = reinterpret_cast<u32x4*>(g.hi + g.at(j, v0));
    u32x4* const lo = g.lo ? reinterpret_cast<u32x4*>(g.lo + g.at(j, v0)) : nullptr;
    if (j >= live) {
        *hi = u32x4{0, 0, 0, 0};
        if (lo) *lo = u32x4{0, 0, 0, 0};
        return;
    }
    const uint32_t t = row[j], y = (uint32_t)p.label[t];
    CeRow r;
    if constexpr (JOIN) { // 32 lanes have the row
        const float2* const q = stat + (uint64_t)j * groups;
        const float z = zy[j];
        float m = -INFINITY;
        for (uint32_t i = threadIdx.x % 32; i < groups; i += 32) m = fmaxf(m, q[i].x);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
        const float shift = shift_of(m);
        double s = 0.0;
        for (uint32_t i = threadIdx.x % 32; i < groups; i += 32) s += (double)q[i].y * exp2_fast(p.c * (q[i].x - shift));
#pragma unroll
        for (int d = 1; d < 32; d *= 2) s += __shfl_xor(s, d);
        r = ce_finish(p, t, shift, s, z, scal->top, blockIdx.x < per && threadIdx.x % 32 == 0);
    } else {
        r = info[j];
    }
    // a group past the vocabulary's end (padding columns): its exponentials are 0
    const uint32_t grp = v0 / group_cols;
    const float scale = grp < groups ? r.a * exp2_fast(p.c * (stat[(uint64_t)j * groups + grp].x - r.m) - r.ls) : 0.f;
    const u32x4 h = grp < groups ? *hi : u32x4{0, 0, 0, 0};
    float v[8];
    if (lo) {
        const u32x4 q = grp < groups ? *lo : u32x4{0, 0, 0, 0};
        const int gexp = ce_exponent(scal->max_g);
        s16x8 oh, ol;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t bits = (h[i / 2] >> (i % 2 * 16) << 16) | (q[i / 2] >> (i % 2 * 16) & 0xffffu);
            v[i] = scale * __uint_as_float(bits) - (v0 + i == y ? r.b : 0.f);
            uint16_t a, b;
            split_f16(ldexpf(v[i], gexp), &a, &b);
            oh[i] = (short)a;
            ol[i] = (short)b;
        }
        *hi = __builtin_bit_cast(u32x4, oh);
        *lo = __builtin_bit_cast(u32x4, ol);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = scale * ce_decode(h[i / 2] >> (i % 2 * 16) & 0xffffu) - (v0 + i == y ? r.b : 0.f);
    *hi = RowIO<bf16_bits>::pack(v);
}

// rows live .. next multiple of 64 of g as zeros (pieces: their product left them)
__global__ __launch_bounds__(256) void ce_zero_kernel(const CeScal* scal, CeG g, uint32_t Vp)
{
    const uint32_t live = scal->live, end = (live + 63) / 64 * 64;
    const uint32_t per = Vp / 8;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < (uint64_t)(end - live) * per; i += gridDim.x * 256ull) {
        const uint64_t at = g.at(live + (uint32_t)(i / per), (uint32_t)(i % per) * 8);
        *reinterpret_cast<u32x4*>(g.hi + at) = u32x4{0, 0, 0, 0};
        if (g.lo) *reinterpret_cast<u32x4*>(g.lo + at) = u32x4{0, 0, 0, 0};
    }
}

// sums of dx, one set per part of the vocabulary (later pieces add to them), or
// of dw, one set per part of the rows
struct CePartEpi {
    float* part; // [splits][rows][ld]
    uint64_t ld, rows;
    bool add;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
                const uint32_t m = at.m0 + i * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
                if (m >= at.M || n >= ld) continue; // ld: H rounded up
                f32x4* q = reinterpret_cast<f32x4*>(part + (at.split * rows + m) * ld + n);
                *q = add ? *q + acc[i][j] : acc[i][j];
            }
    }
};

// The rows of dx (pos: their places, or -1) or dw (pos NULL) from the sums, four
// columns to S threads, each with every S-th part.  other: what the planes of g were
// multiplied with.
template <typename E, int S>
__global__ __launch_bounds__(256) void ce_sum_kernel(const int32_t* pos, uint64_t n, const CeScal* scal,
                                                     const uint32_t* other, const float* part, uint64_t ldp,
                                                     uint64_t rows, uint32_t splits, bool planes, E* out, uint64_t ld,
                                                     uint32_t H)
{
    constexpr uint32_t W = 256 / S;
    const uint32_t sl = threadIdx.x / W, per = (H + 3) / 4;
    const uint64_t i0 = blockIdx.x * (uint64_t)W + threadIdx.x % W;
    const CeItems items(n * per, per);
    const bool in = i0 < items.n;
    uint64_t t = 0;
    uint32_t h = 0;
    if (in) items.split(i0, &t, &h);
    h *= 4;
    const int64_t j = !in ? -1 : pos ? pos[t] : (int64_t)t;
    const int unit = planes ? -ce_exponent(scal->max_g) - ce_exponent(*other) : 0;
    const float top = (float)scal->top;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (j >= 0) {
        const float* q = part + (uint64_t)j * ldp + h;
#pragma unroll 8
        for (uint32_t k = sl; k < splits; k += S) s += *reinterpret_cast<const f32x4*>(q + k * rows * ldp);
    }
    if constexpr (S > 1) {
        __shared__ f32x4 lds[S - 1][W];
        if (sl > 0) lds[sl - 1][threadIdx.x % W] = s;
        __syncthreads();
        if (sl > 0) return;
#pragma unroll
        for (int k = 0; k < S - 1; ++k) s += lds[k][threadIdx.x];
    }
    if (!in) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (h + i < H) RowIO<E>::put(out + t * ld + h + i, j < 0 ? 0.f : ldexpf(s[i], unit) * top);
}

// dw, rounded once to the caller's type
template <bool PLANES>
struct CeHeadEpi {
    const CeScal* scal;
    void* out;
    uint64_t ld;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        const int unit = PLANES ? -ce_exponent(scal->max_g) - ce_exponent(scal->max_x) : 0;
        const float top = (float)scal->top;
        if constexpr (!PLANES) {
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    s16x4 w;
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = __builtin_bit_cast(short, (__bf16)(acc[i][j][k] * top));
                    TileRows<Cfg>::put(at.lds, at.m0 - at.bm0 + i * 16 + l % 16, at.n0 - at.bn0 + j * 16 + l / 16 * 4, w);
                }
            __syncthreads();
            TileRows<Cfg>::each(at.lds, [&](uint32_t m, uint32_t n, s16x8 v) {
                m += at.bm0;
                n += at.bn0;
                if (m < at.M && n < at.N) store_tail(static_cast<uint16_t*>(out) + m * ld + n, v, at.N - n);
            });
            return;
        }
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
                const uint32_t m = at.m0 + i * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
                if (m >= at.M || n >= at.N) continue;
                f32x4 v = acc[i][j];
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = ldexpf(v[k], unit) * top;
                store_tail(static_cast<float*>(out) + m * ld + n, v, at.N - n);
            }
    }
};

// dw of up to 64 rows: a write of the whole head and little else.  A block takes
// 64 tokens; their g stays in registers (a wave 16 tokens, all 64 k) while the
// hidden states come by, 64 columns at a time, the next ones' fetch under way (two
// fetches and fewer blocks to a compute unit: 29 us for 27).
// The products' B fragments take the columns 32 p + 8 q + 4 (j % 2) .., q = 0 .. 3,
// so that a lane's results of two fragments are eight neighbours.
// 24 x 32000 x 2048 bf16: 28 us, which is 131 MB at 4.7 TB/s; as tiles of the products 42.
template <bool PLANES>
__global__ __launch_bounds__(256, PLANES ? 3 : 4) void ce_head_few_kernel(Mat g, Mat x, const CeScal* scal, void* out,
                                                                          uint64_t ld, uint32_t V, uint32_t H,
                                                                          uint32_t cols)
{
    constexpr int P = PLANES ? 2 : 1, TILE = 64 * GEMM_BK * 2;
    __shared__ __align__(1024) char lds[3 * P * TILE];
    // this block's columns
    const uint32_t first = blockIdx.y * cols, end = first + cols < H ? first + cols : H;
    typedef TileLoader<KS, 64, 256> Loader;
    const uint32_t l = threadIdx.x % 64, w = threadIdx.x / 64, v0 = blockIdx.x * 64;
    const bool any = scal->live > 0; // otherwise g was not written
    const int unit = PLANES ? -ce_exponent(scal->max_g) - ce_exponent(scal->max_x) : 0;
    const float top = (float)scal->top;
    const auto fetch = [&](const Mat& m, uint32_t first, bool on, char* to) {
        const Loader ld_(m, first, 0, GEMM_BK);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const typename Loader::Step s = ld_.step(0, p, on, to + p * TILE);
#pragma unroll
            for (int i = 0; i < Loader::U; ++i) s.issue(i);
        }
    };
    char* const xs = lds + P * TILE;
    fetch(g, v0, any, lds);
    fetch(x, first, any, xs);
    // the lane's place in a fragment of columns; the pair's swizzle as in FragReader
    const uint32_t sw = ((l >> 2 & 3) | (l >> 4 & 1) << 2) & 3, kr = (l / 16 * 8 + l % 16 / 4) * 128;
    const auto column = [&](int j) { // of fragment j
        const uint32_t c = j / 2 * 32 + l % 4 * 8 + j % 2 * 4;
        return kr + ((c / 16) ^ sw) * 32 + c % 16 * 2;
    };
    const FragReader<KS, 64, 1> fa(w * 16);
    s16x8 a[P][2];
    wait_loads<P * Loader::U>(); // g is here
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[p][h] = fa.read(lds + p * TILE, 0, h);
    const uint32_t v = v0 + w * 16 + l % 16;
    uint32_t stage = 0;
    for (uint32_t n0 = first; n0 < end; n0 += 64, stage ^= 1) {
        const char* const cur = xs + stage * P * TILE;
        fetch(x, n0 + 64, any && n0 + 64 < end, xs + (stage ^ 1) * P * TILE);
        wait_loads<P * Loader::U>(); // all but the next columns (and, as stores count too, the stores before them)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        f32x4 acc[4] = {};
        const auto multiply = [&](int pa, int pb) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const char* const q = cur + pb * TILE + column(j) + h * 32 * 128;
                    const s16x4 lo = read_transposed((LdsS16x4*)q), hi = read_transposed((LdsS16x4*)(q + 4 * 128));
                    acc[j] = mfma16<PLANES>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), a[pa][h], acc[j]);
                }
        };
        multiply(0, 0);
        if constexpr (PLANES) {
            multiply(0, 1);
            multiply(1, 0);
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t n = n0 + p * 32 + l / 16 * 8;
            float r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = ldexpf(acc[2 * p + i / 4][i % 4], unit) * top;
            if (v < V && n < H) {
                if (PLANES) {
                    float* const q = static_cast<float*>(out) + v * ld + n;
                    store_tail(q, f32x4{r[0], r[1], r[2], r[3]}, H - n);
                    if (n + 4 < H) store_tail(q + 4, f32x4{r[4], r[5], r[6], r[7]}, H - n - 4);
                } else {
                    store_tail(static_cast<uint16_t*>(out) + v * ld + n,
                               __builtin_bit_cast(s16x8, RowIO<bf16_bits>::pack(r)), H - n);
                }
            }
        }
        // this wave's reads are done before the place is fetched into again
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); // the last fetch's zeros
}

// zeros where there is no row at all
template <typename E>
__global__ __launch_bounds__(256) void ce_no_rows_kernel(E* out, uint64_t ld, uint64_t V, uint32_t H)
{
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < V * H; i += gridDim.x * 256ull)
        RowIO<E>::put(out + i / H * ld + i % H, 0.f);
}

// sizes and buffers of a call
struct CePlan {
    uint32_t H, Hp, Tp, piece; // Hp, Tp: rounded up to 64; piece: columns of g
    uint32_t groups, splits, splits_w; // parts of the sums of dx and dw
    bool two, pack, kept, grads, hidden;
    int tile, tile_w, tile_x; // of the logits' product, dw and dx: 0 large, 1 middle, 2 few rows
    CeScal* scal;
    uint32_t* row;
    int32_t* pos;
    float *zy, *part, *part_w;
    float2* stat;
    CeRow* info;
    uint16_t *x[2], *w[2], *g[2];
};

static int ce_tile_cols(int tile) { return tile == 0 ? 256 : 128; }

static CePlan ce_plan(Carver& cv, uint64_t T, uint64_t V, uint32_t H, sg_dtype dt, const void* head, uint64_t ld_head,
                      bool hidden, bool dhead, uint64_t keep)
{
    CePlan p = {};
    p.H = H;
    p.Hp = (uint32_t)align_up(H, 64);
    p.Tp = (uint32_t)align_up(T, 64);
    p.two = dt == SG_F32;
    p.hidden = hidden;
    p.grads = hidden || dhead;
    // the head as it lies: bf16 rows that start on 16 bytes, near enough to one another
    p.pack = p.two || H % 8 || ld_head % 8 || reinterpret_cast<uintptr_t>(head) % 16 || ld_head > GEMM_MAX_LD;
    // By what the tiles take (tile_time).  Up to 32 rows the product is a read of the head, and a tile of 32 rows
    // leaves room for more blocks to a compute unit.  us a call, tiles of 32 rows and of 128, bf16: 32 x 32000 x 2048
    // 100, 105, 32 x 4000 x 1024 46, 50, 32 x 131072 x 4096 826 both; 64 x 131072 x 4096 833, 807
    const uint64_t nseg = p.two ? 3 : 1, kh = ceil_div(H, 64) * nseg, kt = ceil_div(T, 64) * nseg;
    const auto tiles = [](uint64_t m, uint64_t n, uint64_t side) { return ceil_div(m, side) * ceil_div(n, side); };
    const auto pick = [&](uint64_t m, uint64_t n, uint64_t steps) {
        return tile_time(TILE_L, tiles(m, n, 256), steps) <= tile_time(TILE_M, tiles(m, n, 128), steps) ? 0 : 1;
    };
    p.tile = T <= 32 ? 2 : pick(T, V, kh);
    p.groups = (uint32_t)ceil_div(V, ce_tile_cols(p.tile));
    const uint64_t Vp = align_up(V, 256), es = p.two ? 4 : 2;
    // 8 elements of g to a thread of ce_grad_kernel.  All kept where they fit: a second product instead costs more than
    // the pass over them from some hundreds of H on.  us a call, kept and again, 4096 x 32768 x H bf16: 128 424, 370; 256
    // 476, 468; 512 620, 643; 1024 886, 998; fp32: 128 887, 939; 512 1477, 1715
    p.kept = Vp <= (1u << 20) && p.Tp * Vp * es <= keep && p.Tp * Vp < (1ull << 35);
    if (p.kept) {
        p.piece = (uint32_t)Vp;
    } else {
        uint64_t c = keep / (p.Tp * es) / 256 * 256;
        c = c < 256 ? 256 : c > (1u << 20) ? (1u << 20) : c;
        p.piece = (uint32_t)(c < Vp ? c : Vp);
    }
    // dx has few tiles and a long sum, dw where the vocabulary is small: in parts, whose sums are written and read once more
    const auto parts = [&](uint64_t m, uint64_t n, uint64_t steps, bool alone, int* tile, uint32_t* splits) {
        double least = 1e300;
        for (int t = 0; t < 2; ++t)
            for (uint64_t s = 1; s <= 64 && s <= steps; ++s) {
                const uint64_t per = ceil_div(steps, s);
                if (ceil_div(steps, per) != s) continue; // a part without a step
                if (s > 1 && m * ceil_div(n, 1024) >= (1u << 24)) continue; // ce_sum_kernel's grid
                double us = tile_time(t == 0 ? TILE_L : TILE_M, tiles(m, n, t == 0 ? 256 : 128) * s, per * nseg);
                if (s > 1 || !alone) us += 5.0 + 8.0 * s * m * n / 4.5e6;
                if (us < least) {
                    least = us;
                    *tile = t;
                    *splits = (uint32_t)s;
                }
            }
    };
    const uint64_t kv = ceil_div(p.piece, 64);
    if (T <= 32) { // as many parts as there are compute units for 4 blocks each
        p.tile_x = 2;
        const uint64_t want = ceil_div(1024, ceil_div(H, 128)), per = ceil_div(kv, want < kv ? want : kv);
        p.splits = (uint32_t)ceil_div(kv, per);
    } else {
        parts(T, H, kv, false, &p.tile_x, &p.splits);
    }
    // Up to 64 rows dw is one step of 64 k.  us a call, its own kernel and the products' tiles, bf16: 24 x 32000 x 2048 105, 117;
    // 6 x 96832 x 4096 614, 625; 1 x 7972 x 3584 78, 84
    p.tile_w = 2;
    p.splits_w = 1;
    if (kt / nseg > 1) parts(p.piece, H, kt / nseg, true, &p.tile_w, &p.splits_w);

    p.scal = cv.take<CeScal>(1);
    p.row = cv.take<uint32_t>(p.Tp);
    p.pos = cv.take<int32_t>(p.Tp);
    p.zy = cv.take<float>(p.Tp);
    p.stat = cv.take<float2>((uint64_t)p.Tp * p.groups);
    p.info = p.grads ? cv.take<CeRow>(p.Tp) : nullptr;
    for (int i = 0; i < (p.two ? 2 : 1); ++i) {
        p.x[i] = cv.take<uint16_t>((uint64_t)p.Tp * p.Hp);
        p.w[i] = p.pack ? cv.take<uint16_t>(V * p.Hp) : nullptr;
        p.g[i] = p.grads ? cv.take<uint16_t>((uint64_t)p.Tp * p.piece) : nullptr;
    }
    p.part = hidden ? cv.take<float>((uint64_t)p.splits * p.Tp * p.Hp) : nullptr;
    p.part_w = dhead && p.splits_w > 1 ? cv.take<float>((uint64_t)p.splits_w * p.piece * p.Hp) : nullptr;
    return p;
}

template <int AL, int BL, bool F16, class Epi>
static int ce_product(int tile, const Gemm& g, const Epi& e, hipStream_t st)
{
    if (tile == 0) return launch_gemm<TileL, AL, BL, F16>(g, 1, e, st);
    if (AL == KS || tile == 1) return launch_gemm<TileM, AL, BL, F16>(g, 1, e, st);
    if constexpr (AL == KC) return launch_gemm<TileRow, AL, BL, F16>(g, 1, e, st);
    return SG_EUNSUPPORTED;
}

static bool ce_sizes(uint64_t T, uint64_t V, uint64_t H, sg_dtype dt)
{
    return T < (1ull << 31) && V > 0 && V < (1ull << 31) && H > 0 && (dt == SG_F32 || dt == SG_BF16);
}
static bool ce_supported(uint64_t T, uint64_t V, uint64_t H)
{
    // grids of 2^32 threads: 256 to a tile of 128 x 128 and to a row, one to 4 columns of a row
    return H <= (1u << 20) && T * ceil_div(H, 1024) < (1u << 24) && ceil_div(T, 128) * ceil_div(V, 128) < (1u << 24);
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_linear_ce_workspace_bytes(uint64_t T, uint64_t V, uint64_t H, sg_dtype dt, const void* d_head,
                                               uint64_t ld_head, int want_hidden, int want_head, uint64_t keep_bytes)
{
    if (T == 0 || !ce_sizes(T, V, H, dt) || !ce_supported(T, V, H)) return 0;
    Carver cv(nullptr);
    ce_plan(cv, T, V, (uint32_t)H, dt, d_head, ld_head, want_hidden != 0, want_head != 0, keep_bytes);
    return cv.bytes();
}

extern "C" int sg_linear_ce_loss(const void* d_hidden, uint64_t ld_hidden, const void* d_head, uint64_t ld_head,
                                 sg_dtype dt, uint64_t T, uint64_t V, uint64_t H, double inv_temp,
                                 const int32_t* d_label, const float* d_weight, double z_coef, float* d_loss,
                                 float* d_lse, void* d_grad_hidden, uint64_t ld_grad_hidden, void* d_grad_head,
                                 uint64_t ld_grad_head, uint64_t keep_bytes, void* d_ws, size_t ws_bytes, void* stream)
{
    if (!ce_sizes(T, V, H, dt)) return SG_EINVAL;
    if (!(inv_temp >= 1e-37) || !(inv_temp <= 1e6) || !(z_coef >= 0.0) || !(z_coef <= 1e6)) return SG_EINVAL;
    const uint64_t es = dt == SG_F32 ? 4 : 2, far = 1ull << 40;
    if (ld_hidden < H || ld_hidden >= far || ld_head < H || ld_head >= far) return SG_EINVAL;
    if (d_grad_hidden && (ld_grad_hidden < H || ld_grad_hidden >= far)) return SG_EINVAL;
    if (d_grad_head && (ld_grad_head < H || ld_grad_head >= far)) return SG_EINVAL;
    for (const void* q : {d_hidden, d_head, (const void*)d_grad_hidden, (const void*)d_grad_head})
        if (reinterpret_cast<uintptr_t>(q) % es) return SG_EINVAL;
    if (!d_head || (T > 0 && (!d_hidden || !d_label || !d_loss))) return SG_EINVAL;
    if (d_grad_head && d_grad_head == d_head) return SG_EINVAL; // the head is read to the end
    if (!ce_supported(T, V, H)) return SG_EUNSUPPORTED;
    hipStream_t st = as_stream(stream);
    if (T == 0) {
        if (!d_grad_head) return SG_OK;
        if (dt == SG_F32) ce_no_rows_kernel<float><<<2048, 256, 0, st>>>((float*)d_grad_head, ld_grad_head, V, (uint32_t)H);
        else ce_no_rows_kernel<bf16_bits><<<2048, 256, 0, st>>>((bf16_bits*)d_grad_head, ld_grad_head, V, (uint32_t)H);
        SG_TRY_LAUNCH();
        return SG_OK;
    }
    if (!d_ws) return SG_EINVAL;
    if (ws_bytes < sg_linear_ce_workspace_bytes(T, V, H, dt, d_head, ld_head, d_grad_hidden != nullptr, d_grad_head != nullptr, keep_bytes))
        return SG_ECAPACITY;
    Carver cv(d_ws);
    const CePlan p = ce_plan(cv, T, V, (uint32_t)H, dt, d_head, ld_head, d_grad_hidden != nullptr, d_grad_head != nullptr, keep_bytes);
    const float c = (float)(inv_temp * 1.4426950408889634);
    const CeArgs a = {d_label, d_weight, d_loss, d_lse, T, (uint32_t)V, inv_temp, z_coef, c};
    // One launch less while every block can find the live rows itself (fp32: their largest magnitude comes first).
    // us a call, two launches and one, bf16: 56 x 1856 x 79 40.5, 36.3; 24 x 32000 x 2048 96.1, 93.4; 1024 x 1000 x 4096 58.7, 58.4
    const bool gather = !p.two && T <= CE_GATHER;
    if (!gather) {
        ce_rows_kernel<<<1, 1024, 0, st>>>(a, p.row, p.pos, p.scal);
        SG_TRY_LAUNCH();
    }
    // the hidden states' and (head copied) the head's blocks
    const auto blocks = [](uint64_t items, unsigned most) { const uint64_t b = ceil_div(items, 256); return (unsigned)(b < most ? b : most); };
    CeSide sx = {{d_hidden, ld_hidden, p.H}, T, p.row, &p.scal->max_x, p.x[0], p.x[1], blocks((uint64_t)p.Tp * p.Hp / 8, 1024)};
    CeSide sw = {{d_head, ld_head, p.H}, V, nullptr, &p.scal->max_w, p.w[0], p.w[1], blocks(V * p.Hp / 8, 2048)};
    if (p.two) {
        ce_max_kernel<<<sx.blocks + sw.blocks, 256, 0, st>>>(sx, sw, p.scal);
        SG_TRY_LAUNCH();
    }
    sx.blocks = blocks((uint64_t)p.Tp * p.Hp / 8, 8192);
    sw.blocks = p.pack ? blocks(V * p.Hp / 8, 8192) : 0;
    const auto pack = [&](auto zero, auto own) {
        ce_pack_kernel<decltype(zero), decltype(own)::value><<<sx.blocks + sw.blocks, 256, 0, st>>>(sx, sw, p.scal, p.Hp, a, p.row, p.pos);
    };
    if (p.two) pack(float(), std::false_type());
    else if (gather) pack(bf16_bits(), std::true_type());
    else pack(bf16_bits(), std::false_type());
    SG_TRY_LAUNCH();
    const uint32_t nseg = p.two ? 3 : 1;
    const uint64_t ldw = p.pack ? p.Hp : ld_head;
    const uint16_t* const w0 = p.pack ? p.w[0] : static_cast<const uint16_t*>(d_head);
    // rows v0 .. v0 + n of the head
    const auto head = [&](uint64_t v0, uint64_t n) {
        return Mat{{w0 + v0 * ldw, p.w[1] ? p.w[1] + v0 * ldw : nullptr}, ldw, (n - 1) * ldw + (p.pack ? p.Hp : H), 0, 0};
    };
    const Mat mx = {{p.x[0], p.x[1]}, p.Hp, (uint64_t)p.Tp * p.Hp, 0, 0};
    const CeG none = {nullptr, nullptr, 0}, g = {p.g[0], p.g[1], p.Tp};
    const uint32_t* live = &p.scal->live;
    const uint32_t k1 = p.pack ? p.Hp : p.H;
    int rc;

    const bool keep = p.kept && p.grads;
    const Gemm g1 = {mx, head(0, V), (uint32_t)T, (uint32_t)V, k1, nseg, 1, 0, live, nullptr};
    const auto first = [&](auto planes) {
        const CeLogitsEpi<decltype(planes)::value> e = {p.row, d_label, p.scal, p.stat, p.zy, keep ? g : none, p.groups, p.piece, c};
        return ce_product<KC, KC, decltype(planes)::value>(p.tile, g1, e, st);
    };
    if ((rc = p.two ? first(std::true_type()) : first(std::false_type()))) return rc;
    // One launch less where a row's statistics are one load a lane (and g needs no scale of its largest element, as fp32
    // does).  us a call, two launches and one, bf16: 56 x 1856 x 79 44, 40, 8192 x 512 x 512 81, 73; 24 x 32000 x 2048 97,
    // 98, 2048 x 8000 x 256 96, 100
    const bool join = !p.two && keep && p.groups <= 32;
    if (!join) {
        ce_join_kernel<<<(unsigned)T, 256, 0, st>>>(a, p.row, p.stat, p.groups, p.zy, p.info, p.scal, p.two);
        SG_TRY_LAUNCH();
    }
    if (!p.grads) return SG_OK;

    for (uint64_t v0 = 0; v0 < V; v0 += p.piece) {
        const uint64_t n = V - v0 < p.piece ? V - v0 : p.piece, np = align_up(n, 64);
        if (p.kept) {
            const unsigned blocks = (unsigned)(p.Tp / 8 * (p.piece / 256));
            if (join) ce_grad_kernel<true><<<blocks, 256, 0, st>>>(a, p.row, p.stat, p.groups, ce_tile_cols(p.tile), p.zy, p.info, p.scal, g);
            else ce_grad_kernel<false><<<blocks, 256, 0, st>>>(a, p.row, p.stat, p.groups, ce_tile_cols(p.tile), p.zy, p.info, p.scal, g);
            SG_TRY_LAUNCH();
        } else {
            const Gemm g2 = {mx, head(v0, n), (uint32_t)T, (uint32_t)n, k1, nseg, 1, 0, live, nullptr};
            const auto second = [&](auto planes) {
                const CePieceEpi<decltype(planes)::value> e = {p.row, d_label, p.scal, p.info, g, (uint32_t)v0, p.piece, c};
                return ce_product<KC, KC, decltype(planes)::value>(p.tile, g2, e, st);
            };
            if ((rc = p.two ? second(std::true_type()) : second(std::false_type()))) return rc;
            ce_zero_kernel<<<256, 256, 0, st>>>(p.scal, g, p.piece);
            SG_TRY_LAUNCH();
        }
        const Mat mg = {{p.g[0], p.g[1]}, 256, (uint64_t)p.Tp * p.piece, 0, (uint64_t)p.Tp * 256};
        if (d_grad_head) {
            char* const out = static_cast<char*>(d_grad_head) + v0 * ld_grad_head * es;
            const Gemm g3 = {mg, mx, (uint32_t)n, p.H, (uint32_t)T, nseg, p.splits_w, 0, nullptr, live};
            if (p.tile_w == 2) {
                // columns to a block: enough blocks, and 256 columns to pay for g
                const uint64_t want = ceil_div(1024, ceil_div(n, 64)), most = ceil_div(H, 256);
                const uint32_t cols = (uint32_t)align_up(ceil_div(H, want < most ? want : most), 64);
                const dim3 blocks((unsigned)ceil_div(n, 64), (unsigned)ceil_div(H, cols));
                if (p.two) ce_head_few_kernel<true><<<blocks, 256, 0, st>>>(mg, mx, p.scal, out, ld_grad_head, (uint32_t)n, p.H, cols);
                else ce_head_few_kernel<false><<<blocks, 256, 0, st>>>(mg, mx, p.scal, out, ld_grad_head, (uint32_t)n, p.H, cols);
                SG_TRY_LAUNCH();
            } else if (p.splits_w > 1) {
                const CePartEpi e = {p.part_w, p.Hp, p.piece, false};
                rc = p.two ? ce_product<KS, KS, true>(p.tile_w, g3, e, st) : ce_product<KS, KS, false>(p.tile_w, g3, e, st);
                if (rc) return rc;
                const unsigned blocks = (unsigned)ceil_div(n * ceil_div(H, 4), 256);
                if (p.two)
                    ce_sum_kernel<float, 1><<<blocks, 256, 0, st>>>(nullptr, n, p.scal, &p.scal->max_x, p.part_w, p.Hp, p.piece,
                                                                    p.splits_w, true, (float*)out, ld_grad_head, p.H);
                else
                    ce_sum_kernel<bf16_bits, 1><<<blocks, 256, 0, st>>>(nullptr, n, p.scal, nullptr, p.part_w, p.Hp, p.piece,
                                                                        p.splits_w, false, (bf16_bits*)out, ld_grad_head, p.H);
                SG_TRY_LAUNCH();
            } else {
                if (p.two) rc = ce_product<KS, KS, true>(p.tile_w, g3, CeHeadEpi<true>{p.scal, out, ld_grad_head}, st);
                else rc = ce_product<KS, KS, false>(p.tile_w, g3, CeHeadEpi<false>{p.scal, out, ld_grad_head}, st);
                if (rc) return rc;
            }
        }
        if (d_grad_hidden) {
            const CePartEpi e = {p.part, p.Hp, p.Tp, v0 > 0};
            const Gemm g4 = {mg, head(v0, n), (uint32_t)T, p.H, (uint32_t)np, nseg, p.splits, 0, live, nullptr};
            rc = p.two ? ce_product<KC, KS, true>(p.tile_x, g4, e, st) : ce_product<KC, KS, false>(p.tile_x, g4, e, st);
            if (rc) return rc;
        }
    }
    if (d_grad_hidden) {
        // few rows have many parts: four threads to a sum.  us a call, 24 x 32000 x 2048 bf16: 96 for 98
        const auto sum = [&](auto zero, auto slices) {
            typedef decltype(zero) E;
            constexpr int S = decltype(slices)::value;
            ce_sum_kernel<E, S><<<(unsigned)ceil_div(T * ceil_div(H, 4), 256 / S), 256, 0, st>>>(
                p.pos, T, p.scal, &p.scal->max_w, p.part, p.Hp, p.Tp, p.splits, p.two, (E*)d_grad_hidden, ld_grad_hidden, p.H);
        };
        const auto by_rows = [&](auto zero) {
            if (T <= 32) sum(zero, std::integral_constant<int, 4>());
            else sum(zero, std::integral_constant<int, 1>());
        };
        if (p.two) by_rows(float());
        else by_rows(bf16_bits());
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}
