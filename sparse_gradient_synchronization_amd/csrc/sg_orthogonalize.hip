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
// update is 1.7e-3 off with it and 2.0e-3 without; the output's rounding alone
// is 1.66e-3).
struct NsPlanes {
    uint16_t *hi, *lo;
    uint64_t ld, batch;
    float* diag; // [B][ld], NULL: none
};

// four neighbours
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
// The mirrored place of a wave's 16 x 16 block of a symmetric result: through
// 512 bytes of LDS of the wave's own a plane, read back transposed, so that
// a lane again has four neighbours.  A wave's LDS operations run in order.
__device__ __forceinline__ void ns_put_mirrored(const NsPlanes& p, uint64_t base, uint32_t m0, uint32_t n0, f32x4 v,
                                                char* lds)
{
    const uint32_t l = threadIdx.x % 64;
    s16x4 h, q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t x, y;
        split_f16(v[i], &x, &y);
        h[i] = (short)x;
        q[i] = (short)y;
    }
    char* const w = lds + l % 16 * 32 + l / 16 * 8;                     // row m, columns n
    char* const r = lds + (l / 16 * 4 + l % 16 / 4) * 32 + l % 4 * 8;   // four rows of one column
    const uint64_t at = base + (n0 + l % 16) * p.ld + m0 + l / 16 * 4;
    *reinterpret_cast<s16x4*>(w) = h;
    if (p.lo) *reinterpret_cast<s16x4*>(w + 512) = q;
    asm volatile("" ::: "memory");
    *reinterpret_cast<s16x4*>(p.hi + at) = read_transposed((LdsS16x4*)r);
    if (p.lo) *reinterpret_cast<s16x4*>(p.lo + at) = read_transposed((LdsS16x4*)(r + 512));
    asm volatile("" ::: "memory");
}

// what rounding takes from the diagonal, where the four neighbours from (m, n) meet it
__device__ __forceinline__ void ns_put_diag(const NsPlanes& p, uint32_t batch, uint32_t m, uint32_t n, f32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m == n + i) p.diag[batch * p.ld + m] = v[i] - (float)(_Float16)v[i];
}

// A block of a symmetric result, and its mirror image; M and N are multiples of 64,
// so a 16 x 16 block lies inside or outside.
template <class Cfg>
__device__ __forceinline__ void ns_put_symmetric(const NsPlanes& p, const TileAt& at, int i, int j, f32x4 v)
{
    const uint32_t l = threadIdx.x % 64, m0 = at.m0 + i * 16, n0 = at.n0 + j * 16;
    if (m0 >= at.M || n0 >= at.N) return;
    const uint64_t base = at.batch * p.batch;
    const uint32_t m = m0 + l % 16, n = n0 + l / 16 * 4;
    ns_put(p, base + m * p.ld + n, v);
    if (p.diag && m0 == n0) ns_put_diag(p, at.batch, m, n, v);
    // the mirrored block's own tile, if it is taken, writes it itself
    const uint32_t tm = n0 / Cfg::BM, tn = m0 / Cfg::BN;
    if (m0 < n0 && tn < tri_first<Cfg::BM, Cfg::BN>(tm)) ns_put_mirrored(p, base, m0, n0, v, at.lds + (at.wm * Cfg::WN + at.wn) * 1024);
}

// G = X X^T: the tiles on and above the diagonal, and their mirror images
struct NsGramEpi {
    NsPlanes out;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j)
                ns_put_symmetric<Cfg>(out, at, i, j, acc[i][j] * (1.f / (1 << (2 * NS_EX - NS_EG))));
    }
};

// Four neighbours of planes for the blocks of rows i0 .. i0 + R of a wave's
// part, all loaded before the first is used (what lies outside from element 0).
template <class Cfg, int R>
__device__ __forceinline__ void ns_get_rows(const NsPlanes& p, const TileAt& at, int i0, f32x4 (&v)[R][Cfg::NTT])
{
    const uint32_t l = threadIdx.x % 64;
    s16x4 h[R][Cfg::NTT], q[R][Cfg::NTT];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t m = at.m0 + (i0 + i) * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
            const uint64_t o = at.batch * p.batch + (m < at.M && n < at.N ? m * p.ld + n : 0);
            h[i][j] = *reinterpret_cast<const s16x4*>(p.hi + o);
            if (p.lo) q[i][j] = *reinterpret_cast<const s16x4*>(p.lo + o);
        }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[i][j][k] = f16_value((uint16_t)h[i][j][k]);
                if (p.lo) v[i][j][k] += f16_value((uint16_t)q[i][j][k]);
            }
}

// b G + c G^2 from the sums of G^2
struct NsPolyEpi {
    NsPlanes gram, out;
    const NsScale* scale; // one per matrix
    uint32_t step;
    NsCoef coef;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const uint32_t l = threadIdx.x % 64;
        const NsScale sc = scale[at.batch];
        const NsCoef k = step == 0 ? sc.first : coef;
        const int q0 = ns_q(sc, step);
        const float kb = ldexpf(k.b, NS_EB - NS_EG - 2 * q0), kc = ldexpf(k.c, NS_EB - 2 * NS_EG - 4 * q0);
        // G = q + diag(d): G^2 = q^2 + d_m q + q d_n (+ d^2, below fp32's last bit)
        float dm[Cfg::MT];
        f32x4 dn[Cfg::NTT];
        const float* const d = gram.diag ? gram.diag + at.batch * gram.ld : nullptr;
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t m = at.m0 + i * 16 + l % 16;
            dm[i] = d ? d[m < at.M ? m : 0] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t n = at.n0 + j * 16 + l / 16 * 4;
            dn[j] = d ? *reinterpret_cast<const f32x4*>(d + (n < at.N ? n : 0)) : f32x4{0.f, 0.f, 0.f, 0.f};
        }
        constexpr int R = Cfg::MT % 4 == 0 ? 4 : Cfg::MT;
#pragma unroll
        for (int i0 = 0; i0 < Cfg::MT; i0 += R) {
            f32x4 q[R][Cfg::NTT];
            ns_get_rows<Cfg>(gram, at, i0, q);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    f32x4 v = acc[i0 + i][j] + (dm[i0 + i] + dn[j]) * q[i][j];
                    const uint32_t m = at.m0 + (i0 + i) * 16 + l % 16, n = at.n0 + j * 16 + l / 16 * 4;
#pragma unroll
                    for (int x = 0; x < 4; ++x) q[i][j][x] += m == n + x ? dm[i0 + i] : 0.f;
                    v = kc * v + kb * q[i][j];
                    ns_put_symmetric<Cfg>(out, at, i0 + i, j, v);
                }
        }
    }
};

// a X + (the polynomial) X, as the next planes or, after the last step, as
// the result in the caller's type
struct NsStepEpi {
    NsPlanes x, out;
    const float* diag; // the polynomial's, [B][sp], or NULL
    uint32_t sp;
    bool tall;
    void* last; // NULL: planes
    uint64_t ld, stride;
    uint32_t m, n;
    bool bf16, wide;
    const NsScale* scale;
    uint32_t step;
    NsCoef coef;
    template <class Cfg>
    __device__ __forceinline__ void run(const f32x4 (&acc)[Cfg::MT][Cfg::NTT], const TileAt& at) const
    {
        const NsScale sc = scale[at.batch];
        const int q0 = ns_q(sc, step), q1 = ns_q(sc, step + 1);
        // the next planes' scale, or none
        const float up = ldexpf(1.f, last ? -NS_EX - q0 : q1 - q0);
        const float a = step == 0 ? sc.first.a : coef.a;
        const uint32_t l = threadIdx.x % 64;
        const float* const d = diag ? diag + at.batch * (uint64_t)sp : nullptr;
        // a and the polynomial's diagonal, by rows, or by columns for a tall matrix
        float dm[Cfg::MT];
        f32x4 dn[Cfg::NTT];
#pragma unroll
        for (int i = 0; i < Cfg::MT; ++i) {
            const uint32_t r = at.m0 + i * 16 + l % 16;
            dm[i] = a + (d && !tall ? d[r < at.M ? r : 0] * (1.f / (1 << NS_EB)) : 0.f);
        }
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) {
            const uint32_t c = at.n0 + j * 16 + l / 16 * 4;
            dn[j] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (d && tall) dn[j] = *reinterpret_cast<const f32x4*>(d + (c < at.N ? c : 0)) * (1.f / (1 << NS_EB));
        }
        constexpr int R = Cfg::MT % 4 == 0 ? 4 : Cfg::MT;
#pragma unroll
        for (int i0 = 0; i0 < Cfg::MT; i0 += R) {
            f32x4 have[R][Cfg::NTT];
            ns_get_rows<Cfg>(x, at, i0, have);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) {
                    const uint32_t r = at.m0 + (i0 + i) * 16 + l % 16, c = at.n0 + j * 16 + l / 16 * 4;
                    const f32x4 v = ((dm[i0 + i] + dn[j]) * have[i][j] + acc[i0 + i][j] * (1.f / (1 << NS_EB))) * up;
                    if (last) {
                        if (r < m && c < n) put_result(r, c, v, at.batch);
                    } else if (r < at.M && c < at.N) {
                        ns_put(out, at.batch * out.batch + r * out.ld + c, v);
                    }
                }
        }
    }
    __device__ __forceinline__ void put_result(uint32_t r, uint32_t c, f32x4 v, uint32_t batch) const
    {
        const uint64_t o = batch * stride + r * ld + c;
        if (bf16) {
            uint16_t* q = static_cast<uint16_t*>(last) + o;
            s16x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(short, (__bf16)v[i]);
            if (wide && c + 4 <= n) *reinterpret_cast<s16x4*>(q) = w;
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < n) q[i] = (uint16_t)w[i];
        } else {
            float* q = static_cast<float*>(last) + o;
            if (wide && c + 4 <= n) *reinterpret_cast<f32x4*>(q) = v;
            else
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < n) q[i] = v[i];
        }
    }
};

struct NsWs {
    double* part;
    NsScale* scale;
    uint16_t *x[2][2], *gram[2], *poly[2]; // [which][plane]
    float *dgram, *dpoly;                  // diagonals, one plane only
    uint32_t sp, mp, np;                   // shorter side, rows and columns, padded to 64
};
static NsWs ns_carve(Carver& cv, uint32_t B, uint32_t m, uint32_t n, bool two)
{
    NsWs w;
    w.mp = (uint32_t)align_up(m, 64);
    w.np = (uint32_t)align_up(n, 64);
    w.sp = w.mp < w.np ? w.mp : w.np;
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
static int ns_product(const Gemm& g, uint32_t B, const Epi& e, hipStream_t st)
{
    const uint64_t large = ceil_div(g.M, 256) * ceil_div(g.N, 256) * B, mid = ceil_div(g.M, 128) * ceil_div(g.N, 128) * B;
    if (large >= 256) return launch_gemm<TileL, AL, BL, true>(g, B, e, st);
    if (mid >= 256) return launch_gemm<TileM, AL, BL, true>(g, B, e, st);
    return launch_gemm<TileS, AL, BL, true>(g, B, e, st);
}

static Mat ns_mat(uint16_t* const p[2], uint32_t rows, uint32_t ld)
{
    return {{p[0], p[1]}, ld, (uint64_t)rows * ld, (uint64_t)rows * ld};
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
    for (uint32_t s = 0; s < steps; ++s) {
        uint16_t *const *x = w.x[s & 1], *const *y = w.x[~s & 1];
        const Mat mx = ns_mat(x, w.mp, w.np);
        const NsPlanes px = {x[0], x[1], w.np, xb, nullptr}, py = {y[0], y[1], w.np, xb, nullptr};
        int rc;
        const Gemm gg = {mx, mx, w.sp, w.sp, tall ? w.mp : w.np, nseg, 1, 1, nullptr, nullptr};
        rc = tall ? ns_product<KS, KS>(gg, B, NsGramEpi{gram}, st) : ns_product<KC, KC>(gg, B, NsGramEpi{gram}, st);
        if (rc) return rc;
        const Gemm gp = {mg, mg, w.sp, w.sp, w.sp, nseg, 1, 1, nullptr, nullptr};
        if ((rc = ns_product<KC, KC>(gp, B, NsPolyEpi{gram, poly, w.scale, s, coef}, st))) return rc;
        const bool end = s + 1 == steps;
        const bool owide = reinterpret_cast<uintptr_t>(d_out) % 16 == 0 && ld_out % 4 == 0 && (B == 1 || stride_out % 4 == 0);
        const NsStepEpi e = {px, py, w.dpoly, w.sp, tall, end ? d_out : nullptr, ld_out, stride_out, m, n, dt == SG_BF16, owide, w.scale, s, coef};
        const Gemm gx = {tall ? mx : mb, tall ? mb : mx, w.mp, w.np, w.sp, nseg, 1, 0, nullptr, nullptr};
        rc = tall ? ns_product<KC, KC>(gx, B, e, st) : ns_product<KC, KS>(gx, B, e, st);
        if (rc) return rc;
    }
    return SG_OK;
}
