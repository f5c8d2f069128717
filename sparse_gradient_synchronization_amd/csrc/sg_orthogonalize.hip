// sg_orthogonalize.hip -- a matrix's singular values driven towards 1 by
// Newton-Schulz products (the update of the Muon optimiser):
//   X0 = U / (|U|_F + eps),  X <- a X + (b G + c G^2) X,  G = X X^T
// or, for a matrix taller than wide, X <- a X + X (b G + c G^2), G = X^T X:
// G always has the shorter side, and no matrix is transposed (a KS operand
// of the product takes X^T).
//
// Everything between input and output is fp16 in the workspace, under powers
// of two that keep it clear of the type's ends (below).  fp16 and not bf16: the
// iterates' range is known and the 11 bits are not.  A bf16 update takes one
// plane (2^-12 a rounding, 16 times finer than the output's), an fp32 one two
// (22 bits, three products instead of one; fp32 itself has 24).
//
// The division by the norm: U is scaled by the power of two 2^-e that brings
// |U|_F to [1/2, 1), which rounds nothing; (|U|_F + eps) 2^-e = f 2^q with f in
// [1/2, 1), and the first step takes a / f, b / f^3, c / f^5.  q is 0 unless eps
// outweighs the norm.  Then X itself would leave fp16 at its lower end, so the planes
// hold X 2^q; a step multiplies X by at most 4, so q falls by 2 a step.
#include <cmath>
#include <type_traits>

#include "sg_gemm.h"
#include "sg_rows.h"

namespace sg {

// exponents of the planes' scales.  Singular values of the iterates stay
// below 4 and |b| s^2 + |c| s^4 below 128 (checked by the host), so the
// largest stored values are 4 * 2^10, 16 * 2^10 and 128 * 2^8; the smallest
// step of fp16 (2^-24) is 2^-34, 2^-34 and 2^-32 of the true values.
constexpr int NS_EX = 10, NS_EG = 10, NS_EB = 8;
constexpr uint32_t NS_NORM_BLOCKS = 512; // of a matrix; 2048 of a batch are enough for the card

struct NsCoef {
    float a, b, c;
};
struct NsScale {
    NsCoef first; // the first step's coefficients
    int q;        // the planes hold X 2^q at first
};
// q before step s
__device__ __forceinline__ int ns_q(const NsScale& n, uint32_t s)
{
    return n.q > 2 * (int)s ? n.q - 2 * (int)s : 0;
}

// the matrices of the call
struct NsIn {
    const void* x;
    uint64_t ld, stride;
    uint32_t m, n;
};

// 8 elements of a row from column c; what is past the end is 0
template <typename E>
__device__ __forceinline__ void ns_load8(const NsIn& in, uint32_t b, uint32_t r, uint32_t c, float* v)
{
    const E* x = static_cast<const E*>(in.x) + b * in.stride + r * in.ld + c;
    if (c + 8 <= in.n) { // gfx950 loads 16 bytes at any element's address
        constexpr int VEC = RowIO<E>::VEC;
#pragma unroll
        for (int i = 0; i < 8; i += VEC) RowIO<E>::unpack(load_chunk(x + i), v + i);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < in.n ? RowIO<E>::get(x + i) : 0.f;
}

__device__ __forceinline__ double wave_sum64(double s)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    return s;
}

// sums of squares of a share of the matrix, in fp64: an fp32 element's square
// may be out of fp32's range
template <typename E>
__global__ __launch_bounds__(256) void ns_norm_kernel(NsIn in, double* part)
{
    const uint32_t per = (in.n + 7) / 8; // 8 columns at a time
    const uint64_t items = (uint64_t)in.m * per;
    double s = 0.0;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < items; i += gridDim.x * 256ull) {
        float v[8];
        ns_load8<E>(in, blockIdx.y, (uint32_t)(i / per), (uint32_t)(i % per) * 8, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += (double)v[k] * v[k];
    }
    s = wave_sum64(s);
    __shared__ double w[4];
    if (threadIdx.x % 64 == 0) w[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = w[0] + w[1] + w[2] + w[3];
}

// The first planes (rows and columns padded with zeros to 64) and the first
// step's coefficients.
template <typename E>
__global__ __launch_bounds__(256) void ns_pack_kernel(NsIn in, const double* part, uint32_t parts, double eps,
                                                      double a, double b, double c, uint16_t* hi, uint16_t* lo,
                                                      uint32_t mp, uint32_t np, NsScale* scale)
{
    double sum = 0.0;
    for (uint32_t i = threadIdx.x % 64; i < parts; i += 64) sum += part[blockIdx.y * parts + i];
    const double norm = sqrt(wave_sum64(sum));
    int e = 0, q = 0;
    double f = NAN; // an infinity or NaN, or 0 / 0: its whole matrix is NaN
    if (isfinite(norm) && norm > 0.0) {
        (void)frexp(norm, &e);
        f = frexp(ldexp(norm + eps, -e), &q);
    } else if (norm == 0.0 && eps > 0.0) {
        f = 1.0;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        scale[blockIdx.y] = {{(float)(a / f), (float)(b / (f * f * f)), (float)(c / (f * f * f * f * f))}, q};
    const uint32_t per = np / 8;
    const uint64_t items = (uint64_t)mp * per, plane = blockIdx.y * (uint64_t)mp * np;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < items; i += gridDim.x * 256ull) {
        const uint32_t r = (uint32_t)(i / per), col = (uint32_t)(i % per) * 8;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < in.m && col < in.n) ns_load8<E>(in, blockIdx.y, r, col, v);
        s16x8 h, l;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint16_t x, y;
            split_f16(ldexpf(v[k], NS_EX - e), &x, &y);
            h[k] = (short)x;
            l[k] = (short)y;
        }
        const uint64_t o = plane + (uint64_t)r * np + col;
        *reinterpret_cast<s16x8*>(hi + o) = h;
        if (lo) *reinterpret_cast<s16x8*>(lo + o) = l;
    }
}

// fp16 planes as a product's result: rows of ld, matrices of a batch apart.
// diag: of a symmetric result in one plane, what the rounding took from the
// diagonal.  Near the end G and its polynomial are close to multiples of the
// identity, so most of what one plane loses is lost there (a 1000 x 1000 bf16
// update is 1.84e-3 off with it and 1.99e-3 without; the output's rounding alone
// is 1.66e-3).
struct NsPlanes {
    uint16_t *hi, *lo;
    uint64_t ld, batch;
    float* diag; // [B][ld], NULL: none
};

// four neighbours
__device__ __forceinline__ f32x4 ns_get(const NsPlanes& p, uint64_t at)
{
    const s16x4 h = *reinterpret_cast<const s16x4*>(p.hi + at);
    f32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f16_value((uint16_t)h[i]);
    if (p.lo) {
        const s16x4 l = *reinterpret_cast<const s16x4*>(p.lo + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += f16_value((uint16_t)l[i]);
    }
    return v;
}
__device__ __forceinline__ void ns_put(const NsPlanes& p, uint64_t at, f32x4 v)
{
    s16x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t x, y;
        split_f16(v[i], &x, &y);
        h[i] = (short)x;
        l[i] = (short)y;
    }
    *reinterpret_cast<s16x4*>(p.hi + at) = h;
    if (p.lo) *reinterpret_cast<s16x4*>(p.lo + at) = l;
}
// what rounding takes from the diagonal, where the four neighbours from (m, n) meet it
__device__ __forceinline__ void ns_put_diag(const NsPlanes& p, uint32_t batch, uint32_t m, uint32_t n, f32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m == n + i) p.diag[batch * p.ld + m] = v[i] - (float)(_Float16)v[i];
}

// A tile's values as planes, through LDS (TileRows), and with `mirror` in the
// transposed place too: there ds_read_b64_tr_b16 hands a lane eight rows of a
// column.  M and N are multiples of 64.
template <class Cfg, bool TWO>
__device__ __forceinline__ void ns_put_tile(const NsPlanes& p, const TileAt& at, f32x4 (&v)[Cfg::MT][Cfg::NTT],
                                            bool mirror)
{
    static_assert(Cfg::BM == Cfg::BN, "a mirrored tile is a tile");
    const uint32_t l = threadIdx.x % 64, mr = at.m0 - at.bm0, nr = at.n0 - at.bn0;
    const uint64_t base = at.batch * p.batch;
    typedef TileRows<Cfg> Rows;
    const auto put = [&](uint16_t* out, auto low) {
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
                s16x4 w;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint16_t x, y;
                    split_f16(v[i][j][k], &x, &y);
                    w[k] = (short)(decltype(low)::value ? y : x);
                }
                Rows::put(at.lds, mr + i * 16 + l % 16, nr + j * 16 + l / 16 * 4, w);
            }
        __syncthreads();
        Rows::each(at.lds, [&](uint32_t m, uint32_t n, s16x8 w) {
            if (at.bm0 + m < at.M && at.bn0 + n < at.N)
                *reinterpret_cast<s16x8*>(out + base + (at.bm0 + m) * p.ld + at.bn0 + n) = w;
        });
        if (!mirror) return;
        // a wave: 16 columns, 32 rows at a time
        constexpr uint32_t WAVES = Cfg::NT / 64, PARTS = Cfg::BM / 32;
        for (uint32_t i = threadIdx.x / 64; i < Cfg::BN / 16 * PARTS; i += WAVES) {
            const uint32_t n0 = i / PARTS * 16, m0 = i % PARTS * 32 + l / 16 * 8;
            // the lane's share of a group's four rows: row l % 16 / 4, columns l % 4 * 4
            const uint32_t r = m0 + l % 16 / 4, c = n0 + l % 4 * 4;
            const s16x4 lo = read_transposed((LdsS16x4*)(at.lds + Rows::place(r, c))),
                        hi = read_transposed((LdsS16x4*)(at.lds + Rows::place(r + 4, c)));
            const uint32_t n = at.bn0 + n0 + l % 16, m = at.bm0 + m0;
            if (n < at.N && m < at.M)
                *reinterpret_cast<s16x8*>(out + base + n * p.ld + m) = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    // Both planes are taken from the same fp32 numbers: not rounded to fp16 from a product and a sum that were never
    // rounded to fp32 (the first plane alone, in one instruction), and not both halves kept from the first pass (they spill).
    const auto settle = [&]() {
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) asm volatile("" : "+v"(v[i][j]));
    };
    if (TWO) settle();
    put(p.hi, std::false_type());
    if (!TWO) return;
    settle();
    __syncthreads(); // the first plane is out
    put(p.lo, std::true_type());
}

// what rounding takes from the diagonal of a tile on it
template <class Cfg>
__device__ __forceinline__ void ns_put_tile_diag(const NsPlanes& p, const TileAt& at,
                                                 const f32x4 (&v)[Cfg::MT][Cfg::NTT])
{
    if (at.bm0 != at.bn0) return;
    const uint32_t l = threadIdx.x % 64;
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j)
            if (at.m0 + i * 16 == at.n0 + j * 16 && at.m0 + i * 16 < at.M)
                ns_put_diag(p, at.batch, at.m0 + i * 16 + l % 16, at.n0 + j * 16 + l / 16 * 4, v[i][j]);
}

// G = X X^T: the tiles on and above the diagonal, and their mirror images
template <bool TWO>
struct NsGramEpi {
    NsPlanes out;
    template <class Cfg>
    __device__ __forceinline__ void run(f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) acc[i][j] *= 1.f / (1 << (2 * NS_EX - NS_EG));
        if (!TWO) ns_put_tile_diag<Cfg>(out, at, acc);
        ns_put_tile<Cfg, TWO>(out, at, acc, at.bm0 != at.bn0);
    }
};

// Four neighbours of planes for the blocks of rows i0 .. i0 + R of a wave's
// part, all loaded before the first is used (what lies outside from the tile's first).
template <class Cfg, bool TWO, int R>
__device__ __forceinline__ void ns_get_rows(const NsPlanes& p, const TileAt& at, int i0, f32x4 (&v)[R][Cfg::NTT])
{
    const uint32_t l = threadIdx.x % 64;
    s16x4 h[R][Cfg::NTT], q[R][Cfg::NTT];
    const uint64_t tile = at.batch * p.batch + at.bm0 * p.ld + at.bn0;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t m = at.m0 + (i0 + i) * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
            // 256 rows of GEMM_MAX_LD: 32 bits
            const uint32_t o = m < at.M && n < at.N ? (m - at.bm0) * (uint32_t)p.ld + (n - at.bn0) : 0;
            h[i][j] = *reinterpret_cast<const s16x4*>(p.hi + tile + o);
            if (TWO) q[i][j] = *reinterpret_cast<const s16x4*>(p.lo + tile + o);
        }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[i][j][k] = f16_value((uint16_t)h[i][j][k]);
                if (TWO) v[i][j][k] += f16_value((uint16_t)q[i][j][k]);
            }
}

// b G + c G^2 from the sums of G^2
template <bool TWO>
struct NsPolyEpi {
    NsPlanes gram, out;
    const NsScale* scale; // one per matrix
    uint32_t step;
    NsCoef coef;
    template <class Cfg>
    __device__ __forceinline__ void run(f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        const NsScale sc = scale[at.batch];
        const NsCoef k = step == 0 ? sc.first : coef;
        const int q0 = ns_q(sc, step);
        const float kb = ldexpf(k.b, NS_EB - NS_EG - 2 * q0), kc = ldexpf(k.c, NS_EB - 2 * NS_EG - 4 * q0);
        // G = q + diag(d): G^2 = q^2 + d_m q + q d_n (+ d^2, below fp32's last bit)
        float dm[Cfg::MT];
        f32x4 dn[Cfg::NTT];
        const float* const d = TWO ? nullptr : gram.diag + at.batch * gram.ld;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t m = at.m0 + i * 16 + l % 16;
            dm[i] = TWO ? 0.f : d[m < at.M ? m : 0];
        }
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t n = at.n0 + j * 16 + l / 16 * 4;
            dn[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (!TWO) dn[j] = *reinterpret_cast<const f32x4*>(d + (n < at.N ? n : 0));
        }
        constexpr int R = Cfg::MT * Cfg::NTT > 16 ? (TWO ? 1 : 2) : Cfg::MT; // what fits beside the sums
#pragma unroll
        for (int i0 = 0; i0 < Cfg::MT; i0 += R) {
            f32x4 q[R][Cfg::NTT];
            ns_get_rows<Cfg, TWO>(gram, at, i0, q);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    const f32x4 v = acc[i0 + i][j] + (dm[i0 + i] + dn[j]) * q[i][j];
                    const uint32_t m = at.m0 + (i0 + i) * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
                    if (!TWO) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) q[i][j][x] += m == n + x ? dm[i0 + i] : 0.f;
                    }
                    acc[i0 + i][j] = kc * v + kb * q[i][j];
                }
            __builtin_amdgcn_sched_barrier(0); // the next rows' loads stay behind: all at once they spill
        }
        if (!TWO) ns_put_tile_diag<Cfg>(out, at, acc);
        ns_put_tile<Cfg, TWO>(out, at, acc, at.bm0 != at.bn0);
    }
};

// Sums over a part of k of a symmetric product, as they are
struct NsPartEpi {
    float* part; // [splits][B][sp][sp]
    uint32_t sp, B;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        float* const p = part + ((uint64_t)at.split * B + at.batch) * sp * sp;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) {
                const uint32_t m = at.m0 + i * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
                if (m < at.M && n < at.N) *reinterpret_cast<f32x4*>(p + (uint64_t)m * sp + n) = acc[i][j];
            }
    }
};

// The parts added in their order: G (gram.hi NULL) or b G + c G^2, both halves.
// A block takes 64 x 64 on or above the diagonal.
__global__ __launch_bounds__(1024) void ns_join_kernel(const float* part, uint32_t splits, uint32_t sp, uint32_t B,
                                                       NsPlanes gram, NsPlanes out, const NsScale* scale,
                                                       uint32_t step, NsCoef coef)
{
    __shared__ float tile[64][65];
    const uint32_t side = sp / 64;
    uint32_t bm = 0, in = blockIdx.x;
    while (in >= side - bm) in -= side - bm++;
    const uint32_t bn = bm + in, r = threadIdx.x / 16, c = threadIdx.x % 16 * 4, b = blockIdx.y;
    const uint32_t m = bm * 64 + r, n = bn * 64 + c;
    const uint64_t mat = (uint64_t)sp * sp, at = (uint64_t)m * sp + n;
    f32x4 v = {0.f, 0.f, 0.f, 0.f}, q = v, d = v;
    float dm = 0.f, kb = 0.f, kc = 0.f;
    if (gram.hi) { // loaded beside the parts
        const NsScale sc = scale[b];
        const NsCoef k = step == 0 ? sc.first : coef;
        const int q0 = ns_q(sc, step);
        kb = ldexpf(k.b, NS_EB - NS_EG - 2 * q0);
        kc = ldexpf(k.c, NS_EB - 2 * NS_EG - 4 * q0);
        q = ns_get(gram, b * mat + at);
        if (gram.diag) {
            dm = gram.diag[(uint64_t)b * sp + m];
            d = *reinterpret_cast<const f32x4*>(gram.diag + (uint64_t)b * sp + n);
        }
    }
#pragma unroll 8
    for (uint32_t s = 0; s < splits; ++s)
        v += *reinterpret_cast<const f32x4*>(part + ((uint64_t)s * B + b) * mat + at);
    if (gram.hi) {
        v += (dm + d) * q;
#pragma unroll
        for (int x = 0; x < 4; ++x) q[x] += m == n + x ? dm : 0.f;
        v = kc * v + kb * q;
    } else {
        v *= 1.f / (1 << (2 * NS_EX - NS_EG));
    }
    ns_put(out, b * mat + at, v);
    if (bm == bn) { // the whole block: its other half is in it
        if (out.diag) ns_put_diag(out, b, m, n, v);
        return;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) tile[r][c + x] = v[x];
    __syncthreads();
    f32x4 w;
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = tile[c + x][r];
    ns_put(out, b * mat + (uint64_t)(bn * 64 + r) * sp + bm * 64 + c, w);
}

// a X + (the polynomial) X, as the next planes or, after the last step, as
// the result in the caller's type
template <bool TWO>
struct NsStepEpi {
    NsPlanes x, out;
    const float* diag; // the polynomial's, [B][sp], or NULL
    uint32_t sp;
    bool tall;
    void* last; // NULL: planes
    uint64_t ld, stride;
    uint32_t m, n;
    const NsScale* scale;
    uint32_t step;
    NsCoef coef;
    template <class Cfg>
    __device__ __forceinline__ void run(f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const NsScale sc = scale[at.batch];
        const int q0 = ns_q(sc, step), q1 = ns_q(sc, step + 1);
        // the next planes' scale, or none
        const float up = ldexpf(1.f, last ? -NS_EX - q0 : q1 - q0);
        const float a = step == 0 ? sc.first.a : coef.a;
        const uint32_t l = threadIdx.x % 64;
        const float* const d = TWO ? nullptr : diag + at.batch * (uint64_t)sp;
        // a and the polynomial's diagonal, by rows, or by columns for a tall matrix
        float dm[Cfg::MT];
        f32x4 dn[Cfg::NTT];
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t r = at.m0 + i * 16 + l % 16;
            dm[i] = a + (!TWO && !tall ? d[r < at.M ? r : 0] * (1.f / (1 << NS_EB)) : 0.f);
        }
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t c = at.n0 + j * 16 + l / 16 * 4;
            dn[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (!TWO && tall) dn[j] = *reinterpret_cast<const f32x4*>(d + (c < at.N ? c : 0)) * (1.f / (1 << NS_EB));
        }
        constexpr int R = Cfg::MT * Cfg::NTT > 16 ? (TWO ? 1 : 2) : Cfg::MT; // what fits beside the sums
#pragma unroll
        for (int i0 = 0; i0 < Cfg::MT; i0 += R) {
            f32x4 have[R][Cfg::NTT];
            ns_get_rows<Cfg, TWO>(x, at, i0, have);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    acc[i0 + i][j] = ((dm[i0 + i] + dn[j]) * have[i][j] + acc[i0 + i][j] * (1.f / (1 << NS_EB))) * up;
                }
            __builtin_amdgcn_sched_barrier(0); // as in NsPolyEpi
        }
        if (!last) {
            ns_put_tile<Cfg, TWO>(out, at, acc, false);
        } else if constexpr (!TWO) { // an update of one plane is bf16
            typedef TileRows<Cfg> Rows;
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    s16x4 w;
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = __builtin_bit_cast(short, (__bf16)acc[i][j][x]);
                    Rows::put(at.lds, at.m0 - at.bm0 + i * 16 + l % 16, at.n0 - at.bn0 + j * 16 + l / 16 * 4, w);
                }
            __syncthreads();
            Rows::each(at.lds, [&](uint32_t r, uint32_t c, s16x8 w) {
                r += at.bm0;
                c += at.bn0;
                if (r < m && c < n) store_tail(static_cast<uint16_t*>(last) + at.batch * stride + r * ld + c, w, n - c);
            });
        } else {
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    const uint32_t r = at.m0 + i * 16 + l % 16, c = at.n0 + j * 16 + l / 16 * 4;
                    if (r < m && c < n) store_tail(static_cast<float*>(last) + at.batch * stride + r * ld + c, acc[i][j], n - c);
                }
        }
    }
};

// The tile and the parts of k that take least (tile_time).  A symmetric
// product may be split: its parts' sums are written and read once more, at
// 4.5 TB/s, by a kernel of 6 us.
struct NsPlan {
    TileKind tile;
    uint32_t splits;
};
static NsPlan ns_plan(uint32_t M, uint32_t N, uint32_t K, uint32_t nseg, uint32_t B, bool symmetric)
{
    NsPlan best = {TILE_L, 1};
    double least = 1e300;
    const uint64_t ks = ceil_div(K, GEMM_BK);
    for (TileKind t : {TILE_L, TILE_M, TILE_S, TILE_K}) {
        const uint64_t side = tile_side(t), tm = ceil_div(M, side), tn = ceil_div(N, side);
        const uint64_t tiles = (symmetric ? tm * (tm + 1) / 2 : tm * tn) * B;
        for (uint32_t s = 1; s <= (symmetric && t != TILE_K ? 16u : 1u) && s <= ks; ++s) {
            const uint64_t per = ceil_div(ks, s);
            if (ceil_div(ks, per) != s) continue; // a part without a step
            double us = tile_time(t, tiles * s, per * nseg);
            if (s > 1) us += 6.0 + 8.0 * s * tiles * side * side / 4.5e6;
            if (us < least) {
                least = us;
                best = {t, s};
            }
        }
    }
    return best;
}

struct NsWs {
    double* part;
    NsScale* scale;
    uint16_t *x[2][2], *gram[2], *poly[2]; // [which][plane]
    float *dgram, *dpoly;                  // diagonals, one plane only
    uint32_t sp, mp, np;                   // shorter side, rows and columns, padded to 64
    NsPlan pg, pp, ps;                     // how each product is taken
    float* parts;                          // sums of the split ones
};
static NsWs ns_carve(Carver& cv, uint32_t B, uint32_t m, uint32_t n, bool two)
{
    NsWs w;
    w.mp = (uint32_t)align_up(m, 64);
    w.np = (uint32_t)align_up(n, 64);
    w.sp = w.mp < w.np ? w.mp : w.np;
    const uint32_t nseg = two ? 3 : 1;
    w.pg = ns_plan(w.sp, w.sp, w.mp < w.np ? w.np : w.mp, nseg, B, true);
    w.pp = ns_plan(w.sp, w.sp, w.sp, nseg, B, true);
    w.ps = ns_plan(w.mp, w.np, w.sp, nseg, B, false);
    const uint32_t most = w.pg.splits > w.pp.splits ? w.pg.splits : w.pp.splits;
    w.parts = most > 1 ? cv.take<float>((uint64_t)most * B * w.sp * w.sp) : nullptr;
    w.part = cv.take<double>((uint64_t)B * NS_NORM_BLOCKS);
    w.scale = cv.take<NsScale>(B);
    w.dgram = two ? nullptr : cv.take<float>((uint64_t)B * w.sp);
    w.dpoly = two ? nullptr : cv.take<float>((uint64_t)B * w.sp);
    const uint64_t xs = (uint64_t)B * w.mp * w.np, gs = (uint64_t)B * w.sp * w.sp;
    for (int p = 0; p < 2; ++p) {
        const bool none = p == 1 && !two;
        for (int i = 0; i < 2; ++i) w.x[i][p] = none ? nullptr : cv.take<uint16_t>(xs);
        w.gram[p] = none ? nullptr : cv.take<uint16_t>(gs);
        w.poly[p] = none ? nullptr : cv.take<uint16_t>(gs);
    }
    return w;
}

template <int AL, int BL, class Epi>
static int ns_product(TileKind t, const Gemm& g, uint32_t B, const Epi& e, hipStream_t st)
{
    if (t == TILE_L) return launch_gemm<TileL, AL, BL, true>(g, B, e, st);
    if (t == TILE_M) return launch_gemm<TileM, AL, BL, true>(g, B, e, st);
    if (t == TILE_S) return launch_gemm<TileS, AL, BL, true>(g, B, e, st);
    return launch_gemm<TileK, AL, BL, true>(g, B, e, st);
}

static Mat ns_mat(uint16_t* const p[2], uint32_t rows, uint32_t ld)
{
    return {{p[0], p[1]}, ld, (uint64_t)rows * ld, (uint64_t)rows * ld, 0};
}

// Whether the iterates' singular values stay where the scales were made for.
// The first step starts from singular values of at most 1.
static bool ns_in_range(uint32_t steps, double a, double b, double c)
{
    double top = 1.0;
    if (!(fabs(a) <= 4.0)) return false;
    for (uint32_t s = 0; s < steps; ++s) {
        if (!(fabs(b) * top * top + fabs(c) * top * top * top * top <= 128.0)) return false;
        double next = 0.0;
        for (int i = 1; i <= 128; ++i) {
            const double x = top * i / 128, grow = fabs(a + x * x * (b + c * x * x));
            if (!(grow <= 4.0)) return false;
            next = x * grow > next ? x * grow : next;
        }
        if (!(next <= 3.9)) return false;
        top = next * 1.001;
    }
    return true;
}

static bool ns_sizes(uint32_t m, uint32_t n) { return m <= GEMM_MAX_LD - 64 && n <= GEMM_MAX_LD - 64; }

} // namespace sg

using namespace sg;

extern "C" size_t sg_orthogonalize_workspace_bytes(uint32_t B, uint32_t m, uint32_t n, sg_dtype dt)
{
    if (B == 0 || m == 0 || n == 0 || !ns_sizes(m, n) || (dt != SG_F32 && dt != SG_BF16)) return 0;
    Carver cv(nullptr);
    ns_carve(cv, B, m, n, dt == SG_F32);
    return cv.bytes();
}

extern "C" int sg_orthogonalize(const void* d_update, sg_dtype dt, uint32_t B, uint32_t m, uint32_t n, uint64_t ld,
                                uint64_t stride, uint32_t steps, double a, double b, double c, double eps,
                                void* d_out, uint64_t ld_out, uint64_t stride_out, void* d_ws, size_t ws_bytes,
                                void* stream)
{
    if ((dt != SG_F32 && dt != SG_BF16) || steps == 0 || steps > 64 || !(eps >= 0.0) || !(eps <= 1e6)) return SG_EINVAL;
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return SG_EINVAL;
    if (B == 0 || m == 0 || n == 0) return SG_OK;
    if (ld < n || ld_out < n || ld >= (1ull << 40) || ld_out >= (1ull << 40)) return SG_EINVAL;
    if (B > 1 && (stride < (m - 1) * ld + n || stride_out < (m - 1) * ld_out + n || stride >= (1ull << 60) || stride_out >= (1ull << 60))) return SG_EINVAL;
    if (!d_update || !d_out || !d_ws) return SG_EINVAL;
    for (const void* q : {d_update, (const void*)d_out})
        if (reinterpret_cast<uintptr_t>(q) % (dt == SG_F32 ? 4 : 2)) return SG_EINVAL;
    if (d_out == d_update && (ld != ld_out || (B > 1 && stride != stride_out))) return SG_EINVAL;
    if (!ns_sizes(m, n) || B > 65535 || !ns_in_range(steps, a, b, c)) return SG_EUNSUPPORTED;
    if (ws_bytes < sg_orthogonalize_workspace_bytes(B, m, n, dt)) return SG_ECAPACITY;
    const bool two = dt == SG_F32, tall = m > n;
    const size_t es = two ? 4 : 2;
    Carver cv(d_ws);
    NsWs w = ns_carve(cv, B, m, n, two);
    hipStream_t st = as_stream(stream);

    const NsIn in = {d_update, ld, stride, m, n};
    const uint64_t items = ceil_div((uint64_t)m * ceil_div(n, 8), 256);
    uint32_t parts = (uint32_t)ceil_div(2048, B);
    if (parts > NS_NORM_BLOCKS) parts = NS_NORM_BLOCKS;
    if (parts > items) parts = (uint32_t)items;
    const uint64_t pitems = ceil_div((uint64_t)w.mp * w.np / 8, 256);
    const dim3 ngrid(parts, B), pgrid((unsigned)(pitems < 4096 ? pitems : 4096), B);
    if (two) ns_norm_kernel<float><<<ngrid, 256, 0, st>>>(in, w.part);
    else ns_norm_kernel<bf16_bits><<<ngrid, 256, 0, st>>>(in, w.part);
    SG_TRY_LAUNCH();
    if (two) ns_pack_kernel<float><<<pgrid, 256, 0, st>>>(in, w.part, parts, eps, a, b, c, w.x[0][0], w.x[0][1], w.mp, w.np, w.scale);
    else ns_pack_kernel<bf16_bits><<<pgrid, 256, 0, st>>>(in, w.part, parts, eps, a, b, c, w.x[0][0], w.x[0][1], w.mp, w.np, w.scale);
    SG_TRY_LAUNCH();

    const uint32_t nseg = two ? 3 : 1;
    const uint64_t gb = (uint64_t)w.sp * w.sp, xb = (uint64_t)w.mp * w.np;
    const NsPlanes gram = {w.gram[0], w.gram[1], w.sp, gb, w.dgram},
                   poly = {w.poly[0], w.poly[1], w.sp, gb, w.dpoly};
    const Mat mg = ns_mat(w.gram, w.sp, w.sp), mb = ns_mat(w.poly, w.sp, w.sp);
    const NsCoef coef = {(float)a, (float)b, (float)c};
    const auto run = [&](auto planes) -> int {
        constexpr bool TWO = decltype(planes)::value;
        for (uint32_t s = 0; s < steps; ++s) {
            uint16_t *const *x = w.x[s & 1], *const *y = w.x[~s & 1];
            const Mat mx = ns_mat(x, w.mp, w.np);
            const NsPlanes px = {x[0], x[1], w.np, xb, nullptr}, py = {y[0], y[1], w.np, xb, nullptr};
            int rc;
            const Gemm gg = {mx, mx, w.sp, w.sp, tall ? w.mp : w.np, nseg, w.pg.splits, 1, nullptr, nullptr};
            const Gemm gp = {mg, mg, w.sp, w.sp, w.sp, nseg, w.pp.splits, 1, nullptr, nullptr};
            const dim3 jgrid(w.sp / 64 * (w.sp / 64 + 1) / 2, B);
            const NsPartEpi parts = {w.parts, w.sp, B};
            if (w.pg.splits > 1) {
                rc = tall ? ns_product<KS, KS>(w.pg.tile, gg, B, parts, st) : ns_product<KC, KC>(w.pg.tile, gg, B, parts, st);
                if (rc) return rc;
                ns_join_kernel<<<jgrid, 1024, 0, st>>>(w.parts, w.pg.splits, w.sp, B, NsPlanes{}, gram, w.scale, s, coef);
                SG_TRY_LAUNCH();
            } else {
                const NsGramEpi<TWO> e = {gram};
                rc = tall ? ns_product<KS, KS>(w.pg.tile, gg, B, e, st) : ns_product<KC, KC>(w.pg.tile, gg, B, e, st);
                if (rc) return rc;
            }
            if (w.pp.splits > 1) {
                if ((rc = ns_product<KC, KC>(w.pp.tile, gp, B, parts, st))) return rc;
                ns_join_kernel<<<jgrid, 1024, 0, st>>>(w.parts, w.pp.splits, w.sp, B, gram, poly, w.scale, s, coef);
                SG_TRY_LAUNCH();
            } else if ((rc = ns_product<KC, KC>(w.pp.tile, gp, B, NsPolyEpi<TWO>{gram, poly, w.scale, s, coef}, st))) {
                return rc;
            }
            const bool end = s + 1 == steps;
            const NsStepEpi<TWO> e = {px, py, w.dpoly, w.sp, tall, end ? d_out : nullptr, ld_out, stride_out, m, n, w.scale, s, coef};
            const Gemm gx = {tall ? mx : mb, tall ? mb : mx, w.mp, w.np, w.sp, nseg, 1, 0, nullptr, nullptr};
            rc = tall ? ns_product<KC, KC>(w.ps.tile, gx, B, e, st) : ns_product<KC, KS>(w.ps.tile, gx, B, e, st);
            if (rc) return rc;
        }
        return SG_OK;
    };
    return two ? run(std::true_type()) : run(std::false_type());
}
