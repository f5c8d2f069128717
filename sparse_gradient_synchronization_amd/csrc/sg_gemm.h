// sg_gemm.h -- matrix products of 16-bit operands with fp32 sums, the core of
// the operators that are products: C[m][n] = sum_k A(m, k) B(n, k).
//
// An operand lies in memory either with k contiguous (KC: one row per m or n)
// or with m or n contiguous (KS: one row per k), so no operand is transposed
// in memory: a KS tile is read from LDS by ds_read_b64_tr_b16, which hands
// each lane four k of one column.
//
// A block computes a BM x BN tile.  64 k of both operands at a time go
// straight from memory into LDS (buffer_load ... lds, 16 bytes a lane; what
// lies past an operand's end reads as zero).  Every 16 bytes land at a
// permuted place, so that the reads of a wave touch every bank once:
//   KC  row r of 128 bytes, chunk c at c ^ (r & 7)
//   KS  row k of 2 * tile bytes, 32-byte pair p at p ^ g(k), g from k's bits
//       0, 1 and 3 (the rows that one transposing read takes together)
//
// The products are taken as B-fragment times A-fragment, so a lane's four
// results of one instruction are neighbours in n:
//   m = 16 i + lane % 16, n = 16 j + 4 (lane / 16) + {0, 1, 2, 3}.
//
// fp32 operands are two fp16 planes, hi + lo = 22 bits of each element under
// a power-of-two scale; their product is the three plane products
// hi hi + hi lo + lo hi, one after another into the same sums ("segments").
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sg_host.h"

namespace sg {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

enum Layout { KC = 0, KS = 1 };

struct Mat {
    const uint16_t* p[2]; // planes; p[1] only with three segments
    uint64_t ld;          // elements between rows, a multiple of 8
    uint64_t elems;       // from the start to the end of the last row
    uint64_t batch;       // elements between the matrices of a batch
};

struct Gemm {
    Mat a, b;
    uint32_t M, N, K;
    uint32_t nseg;       // 1, or 3 for two planes
    uint32_t splits;     // k in so many parts, one per blockIdx.y
    uint32_t tri;        // 1: symmetric result, no tiles below the diagonal
    const uint32_t* d_m; // M, and K (rounded up to 64), from device memory instead
    const uint32_t* d_k;
};

constexpr int GEMM_BK = 64;
constexpr uint64_t GEMM_MAX_LD = 1u << 21; // 256 rows of it stay below 2^31 bytes

#define SG_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// where the chunk that thread-unit u of a tile fetches lies, in bytes from
// the tile's first element
template <int LAY, int R>
__device__ __forceinline__ uint32_t tile_source(uint32_t u, uint32_t ld, uint32_t* k_of)
{
    if (LAY == KC) {
        const uint32_t r = u / 8, c = (u % 8) ^ (r & 7);
        *k_of = c * 8;
        return (r * ld + c * 8) * 2;
    }
    constexpr uint32_t PER = R / 8;
    const uint32_t k = u / PER, g = ((k & 3) | ((k >> 3) & 1) << 2) & (R / 16 - 1);
    *k_of = 0; // rows past the end lie past the buffer's end
    return (k * ld + ((u % PER) ^ (2 * g)) * 8) * 2;
}

// One operand's tiles: R rows (KC) or columns (KS) from first, NT threads.
template <int LAY, int R, int NT>
struct TileLoader {
    static constexpr int U = R * 8 / NT; // chunks a thread fetches per step
    static_assert(R * 8 % NT == 0, "the tile is a whole number of chunks a thread");
    const uint16_t* p[2];
    uint64_t ld, left; // elements from the tile's start to the operand's end
    uint32_t src[U], kk[U], K;

    __device__ __forceinline__ TileLoader(const Mat& m, uint64_t first, uint32_t batch, uint32_t K_) : ld(m.ld), K(K_)
    {
        const uint64_t at = LAY == KC ? first * m.ld : first;
        left = m.elems > at ? m.elems - at : 0;
        p[0] = m.p[0] + batch * m.batch + at;
        p[1] = m.p[1] ? m.p[1] + batch * m.batch + at : p[0];
#pragma unroll
        for (int i = 0; i < U; ++i) src[i] = tile_source<LAY, R>(i * NT + threadIdx.x, (uint32_t)m.ld, &kk[i]);
    }
    __device__ __forceinline__ void load(uint32_t k0, int plane, char* lds) const
    {
        const uint64_t at = LAY == KC ? (uint64_t)k0 : (uint64_t)k0 * ld;
        uint64_t bytes = left > at ? (left - at) * 2 : 0;
        if (bytes > 0x7ffffff0ull) bytes = 0x7ffffff0ull;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint16_t*>(p[plane] + at), 0, (uint32_t)bytes, 0x00020000);
        char* to = lds + (threadIdx.x / 64) * 1024;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            // past the row's end: an offset past the buffer's end
            const uint32_t off = LAY == KS || k0 + kk[i] < K ? src[i] : 0xfffffff0u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, SG_LDS(to + i * NT * 16), 16, off, 0, 0, 0);
        }
    }
};

// A wave's fragments of 16 rows or columns from LDS, T side by side.
template <int LAY, int R, int T>
struct FragReader {
    uint32_t at[LAY == KC ? 1 : T];
    __device__ __forceinline__ explicit FragReader(uint32_t first)
    {
        const uint32_t l = threadIdx.x % 64;
        if (LAY == KC) {
            at[0] = (first + l % 16) * 128 + ((l / 16) ^ (l & 7)) * 16;
        } else {
            const uint32_t g = ((l >> 2 & 3) | (l >> 4 & 1) << 2) & (R / 16 - 1);
#pragma unroll
            for (int t = 0; t < T; ++t)
                at[LAY == KC ? 0 : t] =
                    ((l / 16) * 8 + (l % 16) / 4) * (R * 2) + ((first / 16 + t) ^ g) * 32 + l % 4 * 8;
        }
    }
    // 16 x 32 (k = 32 h ..): the lane's row or column is lane % 16, its k are 8 (lane / 16) ..
    __device__ __forceinline__ s16x8 read(const char* lds, int t, int h) const
    {
        if (LAY == KC) return *reinterpret_cast<const s16x8*>(lds + (at[0] ^ h * 64) + t * 2048);
        typedef __attribute__((address_space(3))) s16x4* P;
        const char* q = lds + at[LAY == KC ? 0 : t] + h * 32 * R * 2;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(q));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(q + 4 * R * 2));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

template <bool F16>
__device__ __forceinline__ f32x4 mfma16(s16x8 x, s16x8 y, f32x4 c)
{
    if (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c,
                                                      0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Consecutive blocks go to the 8 XCDs in turn; each XCD gets a contiguous run
// of tiles, in groups of 8 tile rows, so that its L2 holds what they share.
__device__ __forceinline__ void tile_of(uint32_t tm, uint32_t tn, uint32_t* m, uint32_t* n)
{
    const uint32_t id = blockIdx.x, total = tm * tn, x = id % 8, q = total / 8, r = total % 8;
    const uint32_t pid = x * q + (x < r ? x : r) + id / 8;
    const uint32_t group = pid / (8 * tn), first = group * 8, rows = tm - first < 8 ? tm - first : 8,
                   in = pid % (8 * tn);
    *m = first + in % rows;
    *n = in / rows;
}

template <int BM_, int BN_, int WM_, int WN_>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NT = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NTT = BN / WN / 16; // fragments of a wave
    static constexpr int STAGE = (BM + BN) * GEMM_BK * 2;
    static constexpr int LDS = 2 * STAGE;
    // waves per SIMD that the LDS leaves room for (160 KB)
    static constexpr int BLOCKS = 163840 / LDS, WAVES = BLOCKS * WM * WN / 4;
    static constexpr int PER_SIMD = WAVES < 1 ? 1 : WAVES > 4 ? 4 : WAVES;
};
typedef TileCfg<256, 256, 2, 4> TileL;
typedef TileCfg<128, 128, 2, 2> TileM;
typedef TileCfg<64, 64, 2, 2> TileS;   // few tiles: more blocks
typedef TileCfg<32, 128, 1, 4> TileRow; // few rows

// what an epilogue gets beside the sums
struct TileAt {
    uint32_t m0, n0;   // first element of the wave's part
    uint32_t bm0, bn0; // of the block's tile
    uint32_t M, N;
    uint32_t split, batch;
    uint32_t wm, wn; // the wave's place in the block
    char* lds;
};

template <class Cfg, int AL, int BL, bool F16, class Epi>
__global__ __launch_bounds__(Cfg::NT, Cfg::PER_SIMD) void gemm_kernel(Gemm g, Epi epi)
{
    __shared__ __align__(1024) char lds[Cfg::LDS];
    if (g.d_m) g.M = *g.d_m;
    if (g.d_k) g.K = (*g.d_k + GEMM_BK - 1) / GEMM_BK * GEMM_BK;
    const uint32_t tiles_n = (g.N + Cfg::BN - 1) / Cfg::BN;
    uint32_t tm, tn;
    tile_of(gridDim.x / tiles_n, tiles_n, &tm, &tn);
    if (tm * Cfg::BM >= g.M) return;                   // fewer rows than the launch was made for
    if (g.tri && tm * Cfg::BM >= (tn + 1) * Cfg::BN) return; // wholly below the diagonal
    const uint32_t w = threadIdx.x / 64, wm = w / Cfg::WN, wn = w % Cfg::WN;

    const TileLoader<AL, Cfg::BM, Cfg::NT> la(g.a, (uint64_t)tm * Cfg::BM, blockIdx.z, g.K);
    const TileLoader<BL, Cfg::BN, Cfg::NT> lb(g.b, (uint64_t)tn * Cfg::BN, blockIdx.z, g.K);
    const FragReader<AL, Cfg::BM, Cfg::MT> fa(wm * (Cfg::BM / Cfg::WM));
    const FragReader<BL, Cfg::BN, Cfg::NTT> fb(wn * (Cfg::BN / Cfg::WN));
    constexpr int UA = Cfg::BM * GEMM_BK * 2, LOADS = la.U + lb.U;

    // this part's steps of 64 k, then all of them again for the next segment
    const uint32_t ks = (g.K + GEMM_BK - 1) / GEMM_BK, per = (ks + g.splits - 1) / g.splits;
    const uint32_t first = blockIdx.y * per < ks ? blockIdx.y * per : ks, last = first + per < ks ? first + per : ks;
    const uint32_t steps = (last - first) * g.nseg;

    f32x4 acc[Cfg::MT][Cfg::NTT];
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint32_t k = first, seg = 0; // of the next step to fetch
    const auto fetch = [&](char* to) {
        la.load(k * GEMM_BK, seg == 2, to);
        lb.load(k * GEMM_BK, seg == 1, to + UA);
        if (++k == last) {
            k = first;
            ++seg;
        }
    };
    if (steps > 0) fetch(lds);
    for (uint32_t s = 0; s < steps; ++s) {
        char* const cur = lds + (s & 1) * Cfg::STAGE;
        if (s + 1 < steps) {
            fetch(lds + (~s & 1) * Cfg::STAGE);
            wait_loads<LOADS>();
        } else {
            wait_loads<0>();
        }
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s16x8 b[Cfg::NTT];
#pragma unroll
            for (int j = 0; j < Cfg::NTT; ++j) b[j] = fb.read(cur + UA, j, h);
#pragma unroll
            for (int i = 0; i < Cfg::MT; ++i) {
                const s16x8 a = fa.read(cur, i, h);
#pragma unroll
                for (int j = 0; j < Cfg::NTT; ++j) acc[i][j] = mfma16<F16>(b[j], a, acc[i][j]);
            }
        }
        // this wave's reads are done before another wave fetches into the same place
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    TileAt at;
    at.bm0 = tm * Cfg::BM;
    at.bn0 = tn * Cfg::BN;
    at.m0 = at.bm0 + wm * (Cfg::BM / Cfg::WM);
    at.n0 = at.bn0 + wn * (Cfg::BN / Cfg::WN);
    at.M = g.M;
    at.N = g.N;
    at.split = blockIdx.y;
    at.batch = blockIdx.z;
    at.wm = wm;
    at.wn = wn;
    at.lds = lds;
    epi.template run<Cfg>(acc, at);
}

template <class Cfg, int AL, int BL, bool F16, class Epi>
static int launch_gemm(const Gemm& g, uint32_t batch, const Epi& epi, hipStream_t st)
{
    const uint64_t tiles = ceil_div(g.M, Cfg::BM) * ceil_div(g.N, Cfg::BN);
    if (tiles == 0 || batch == 0) return SG_OK;
    if (tiles >= (1ull << 31) || g.splits == 0 || g.splits > 65535 || batch > 65535) return SG_EUNSUPPORTED;
    if (g.a.ld > GEMM_MAX_LD || g.b.ld > GEMM_MAX_LD) return SG_EUNSUPPORTED;
    gemm_kernel<Cfg, AL, BL, F16, Epi><<<dim3((unsigned)tiles, g.splits, batch), Cfg::NT, 0, st>>>(g, epi);
    SG_TRY_LAUNCH();
    return SG_OK;
}

// fp16 planes of an fp32 value: 22 bits of it
__device__ __forceinline__ void split_f16(float v, uint16_t* hi, uint16_t* lo)
{
    const _Float16 h = (_Float16)v;
    *hi = __builtin_bit_cast(uint16_t, h);
    *lo = __builtin_bit_cast(uint16_t, (_Float16)(v - (float)h));
}
__device__ __forceinline__ float f16_value(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }

} // namespace sg
