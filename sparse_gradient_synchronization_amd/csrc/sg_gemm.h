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
    // not 0: columns in panels of 256, so many elements apart, ld between the rows of one.
    // A tile of a wide matrix then lies close together and not over a page a row
    uint64_t panel;
};

struct Gemm {
    Mat a, b;
    uint32_t M, N, K;
    uint32_t nseg;       // 1, or 3 for two planes
    uint32_t splits;     // k in so many parts, each with sums of its own
    uint32_t tri;        // 1: symmetric result, no tiles below the diagonal
    const uint32_t* d_m; // M, and K (rounded up to 64), from device memory instead
    const uint32_t* d_k;
};

constexpr int GEMM_BK = 64;
constexpr uint64_t GEMM_MAX_LD = 1u << 21; // 256 rows of it stay below 2^31 bytes

#define SG_LDS(p) ((__attribute__((address_space(3))) void*)(p))

// One operand's tiles: R rows (KC) or columns (KS) from first, NT threads.
template <int LAY, int R, int NT>
struct TileLoader {
    static constexpr int U = R * 8 / NT; // chunks a thread fetches per step
    static_assert(R * 8 % NT == 0, "the tile is a whole number of chunks a thread");
    static constexpr int PER = LAY == KC ? 8 : R / 8; // chunks of a row (of 64 k, or of R columns)
    // A thread's chunks lie multiples of 8 rows apart.  The places repeat after
    // 8 (KC) or 16 (KS), so its odd chunks may have a place of their own.
    static_assert(U == 1 || NT / PER % 8 == 0, "at most two places for a thread's chunks");
    static constexpr bool TWO = LAY == KS && U > 1 && NT / PER % 16 != 0;
    const uint16_t* p[2];
    uint64_t ld, left;   // elements from the tile's start to the operand's end
    uint64_t panel;
    uint32_t src[2], kk, K; // the thread's first chunk, in bytes (for even and odd ones), and its k
    uint32_t apart;      // bytes between its chunks

    __device__ __forceinline__ TileLoader(const Mat& m, uint64_t first, uint32_t batch, uint32_t K_)
        : ld(m.ld), panel(m.panel), K(K_)
    {
        const uint32_t tid = threadIdx.x % NT;
        const uint64_t at = LAY == KC ? first * m.ld : panel ? first / 256 * panel + first % 256 : first;
        left = m.elems > at ? m.elems - at : 0;
        p[0] = m.p[0] + batch * m.batch + at;
        p[1] = m.p[1] ? m.p[1] + batch * m.batch + at : p[0];
        const uint32_t r = tid / PER, q = tid % PER;
        const uint32_t c = LAY == KC ? q ^ (r & 7) : q ^ (2 * (((r & 3) | ((r >> 3) & 1) << 2) & (R / 16 - 1)));
        src[0] = (r * (uint32_t)m.ld + c * 8) * 2;
        src[1] = (r * (uint32_t)m.ld + (c ^ (2 * (4 & (R / 16 - 1)))) * 8) * 2;
        kk = c * 8;
        apart = NT / PER * (uint32_t)m.ld * 2;
    }
    // One step's fetch, set up at once and issued chunk by chunk: 64 k from k0; nothing (zeros) if !on
    struct Step {
        __amdgpu_buffer_rsrc_t r;
        uint32_t off[2], apart;
        char* to;
        __device__ __forceinline__ void issue(int i) const
        {
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, SG_LDS(to + i * NT * 16), 16, off[TWO ? i % 2 : 0] + i * apart, 0,
                                                     0, 0);
        }
    };
    __device__ __forceinline__ Step step(uint32_t k0, int plane, bool on, char* lds) const
    {
        const uint64_t at = LAY == KS ? (uint64_t)k0 * ld : panel ? k0 / 256 * panel + k0 % 256 : (uint64_t)k0;
        uint64_t bytes = on && left > at ? (left - at) * 2 : 0;
        if (bytes > 0x7ffffff0ull) bytes = 0x7ffffff0ull;
        Step s;
        s.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p[plane] + at), 0, (uint32_t)bytes, 0x00020000);
        // KC, past the row's end: an offset past the buffer's end.  KS: rows past the end lie there
        s.off[0] = LAY == KS || k0 + kk < K ? src[0] : 0x80000000u;
        s.off[1] = src[1];
        s.apart = apart;
        s.to = lds + (threadIdx.x % NT / 64) * 1024;
        return s;
    }
};

typedef __attribute__((address_space(3))) s16x4 LdsS16x4;
// __restrict__ gives the read an alias scope.  Without one the compiler takes
// every fetch into LDS for one that this read may depend on and waits for all of
// them (the waits that are needed stand in the kernel).
__device__ __forceinline__ s16x4 read_transposed(LdsS16x4* __restrict__ p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
}

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
        const char* q = lds + at[LAY == KC ? 0 : t] + h * 32 * R * 2;
        const s16x4 lo = read_transposed((LdsS16x4*)q), hi = read_transposed((LdsS16x4*)(q + 4 * R * 2));
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

// The tiles of a launch, in their order: tiles, parts of k, matrices of a
// batch.  Consecutive blocks go to the 8 XCDs in turn; each XCD gets a contiguous
// run of what there is to do, so that its L2 holds what the tiles share and
// all have as much: groups of 8 tile rows, or, of a symmetric result, the rows of
// the tiles that are not wholly below the diagonal.
template <int BM, int BN>
__host__ __device__ __forceinline__ uint32_t tri_first(uint32_t m) // of tile row m
{
    return m * BM / BN;
}
template <int BM, int BN>
__host__ __device__ __forceinline__ uint32_t tile_count(uint32_t tm, uint32_t tn, uint32_t tri)
{
    if (!tri) return tm * tn;
    uint32_t c = 0;
    for (uint32_t m = 0; m < tm && tri_first<BM, BN>(m) < tn; ++m) c += tn - tri_first<BM, BN>(m);
    return c;
}
struct TilePlace {
    uint32_t m, n, split, batch;
};
template <int BM, int BN>
__device__ __forceinline__ bool tile_of(uint32_t tm, uint32_t tn, uint32_t tri, uint32_t splits, uint32_t batch,
                                        TilePlace* p)
{
    const uint32_t tiles = tile_count<BM, BN>(tm, tn, tri), total = tiles * splits * batch;
    const uint32_t id = blockIdx.x, x = id % 8, q = total / 8, r = total % 8;
    if (id >= total) return false; // fewer rows than the launch was made for
    const uint32_t at = x * q + (x < r ? x : r) + id / 8, pid = at % tiles, rest = at / tiles;
    p->split = rest % splits;
    p->batch = rest / splits;
    if (tri) {
        uint32_t m = 0, in = pid;
        while (in >= tn - tri_first<BM, BN>(m)) in -= tn - tri_first<BM, BN>(m++);
        p->m = m;
        p->n = tri_first<BM, BN>(m) + in;
        return true;
    }
    const uint32_t group = pid / (8 * tn), first = group * 8, rows = tm - first < 8 ? tm - first : 8,
                   in = pid % (8 * tn);
    p->m = first + in % rows;
    p->n = in / rows;
    return true;
}

// GR_: groups of WM x WN waves in a block, each with stages of its own and every
// GR-th step; their sums are added at the end
template <int BM_, int BN_, int WM_, int WN_, int GR_ = 1>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, GR = GR_, NT = 64 * WM * WN;
    static constexpr int MT = BM / WM / 16, NTT = BN / WN / 16; // fragments of a wave
    static constexpr int STAGE = (BM + BN) * GEMM_BK * 2;
    static constexpr int LDS = 2 * STAGE * GR;
    static_assert(GR == 1 || (GR - 1) * BM * BN * 4 + 1024 * WM * WN <= LDS, "the other groups' sums, and a kilobyte a wave");
    // waves per SIMD that the LDS leaves room for (160 KB)
    static constexpr int BLOCKS = 163840 / LDS, WAVES = BLOCKS * GR * WM * WN / 4;
    static constexpr int PER_SIMD = WAVES < 1 ? 1 : WAVES > 4 ? 4 : WAVES;
};
typedef TileCfg<256, 256, 2, 4> TileL;
typedef TileCfg<128, 128, 2, 2> TileM;
typedef TileCfg<64, 64, 2, 2> TileS;      // few tiles: more blocks
typedef TileCfg<64, 64, 2, 2, 4> TileK;   // fewer than compute units: more waves to a tile
typedef TileCfg<32, 128, 1, 4> TileRow;   // few rows

// what an epilogue gets beside the sums
struct TileAt {
    uint32_t m0, n0;   // first element of the wave's part
    uint32_t bm0, bn0; // of the block's tile
    uint32_t M, N;
    uint32_t split, batch;
    uint32_t wm, wn; // the wave's place in the block
    char* lds;
};

// Two stages of LDS, two halves of 32 k to a stage.  While one half is
// multiplied the next one is read into registers; the block meets once a step,
// between the halves, with the second half in registers: there are products to do
// on both sides of the barrier, behind which the stage just read is fetched into
// again.  Fetches are issued one at a time among the products: issued together
// they hold up the wave for as long as the memory pipeline takes them in (8192^3
// bf16: 870 us together, 790 apart; 670 without any fetch and 650 with neither
// fetch nor barrier, what the products alone take at the clock they leave the card).
// Tiles one after another in a block, the next one's fetches under the epilogue, took
// as long: a wait for fetches is one for the stores before them.
template <class Cfg, int AL, int BL, bool F16, class Epi>
__global__ __launch_bounds__(Cfg::NT * Cfg::GR, Cfg::PER_SIMD) void gemm_kernel(Gemm g, uint32_t batch, Epi epi)
{
    __shared__ __align__(1024) char lds_all[Cfg::LDS];
    if (g.d_m) g.M = *g.d_m;
    if (g.d_k) g.K = (*g.d_k + GEMM_BK - 1) / GEMM_BK * GEMM_BK;
    TilePlace t;
    if (!tile_of<Cfg::BM, Cfg::BN>((g.M + Cfg::BM - 1) / Cfg::BM, (g.N + Cfg::BN - 1) / Cfg::BN, g.tri, g.splits, batch,
                                   &t))
        return;
    const uint32_t w = threadIdx.x % Cfg::NT / 64, wm = w / Cfg::WN, wn = w % Cfg::WN;
    const uint32_t group = uniform(threadIdx.x / Cfg::NT);
    char* const lds = lds_all + group * 2 * Cfg::STAGE;

    typedef TileLoader<AL, Cfg::BM, Cfg::NT> LoadA;
    typedef TileLoader<BL, Cfg::BN, Cfg::NT> LoadB;
    const LoadA la(g.a, (uint64_t)t.m * Cfg::BM, t.batch, g.K);
    const LoadB lb(g.b, (uint64_t)t.n * Cfg::BN, t.batch, g.K);
    const FragReader<AL, Cfg::BM, Cfg::MT> fa(wm * (Cfg::BM / Cfg::WM));
    const FragReader<BL, Cfg::BN, Cfg::NTT> fb(wn * (Cfg::BN / Cfg::WN));
    constexpr int UA = Cfg::BM * GEMM_BK * 2, LOADS = LoadA::U + LoadB::U;
    constexpr int READS = Cfg::MT + Cfg::NTT, PRODUCTS = Cfg::MT * Cfg::NTT;
    // groups of a half's work: a fetch each, and reads in the first three quarters
    constexpr int G = LOADS < PRODUCTS ? LOADS : PRODUCTS, RG = G * 3 / 4;

    // this part's steps of 64 k, then all of them again for the next segment
    const uint32_t ks = (g.K + GEMM_BK - 1) / GEMM_BK, per = (ks + g.splits - 1) / g.splits;
    const uint32_t first = t.split * per < ks ? t.split * per : ks, last = first + per < ks ? first + per : ks;
    // a group's first k of a segment, and the steps of all (a group without a k of its own multiplies zeros)
    const uint32_t steps = (last - first + Cfg::GR - 1) / Cfg::GR * g.nseg;

    f32x4 acc[Cfg::MT][Cfg::NTT];
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::NTT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint32_t k = first, seg = 0; // of the block's next step to fetch; past the last one it fetches nothing
    struct Fetch {
        typename LoadA::Step a;
        typename LoadB::Step b;
        __device__ __forceinline__ void issue(int i) const
        {
            if (i < LoadA::U) a.issue(i);
            else b.issue(i - LoadA::U);
        }
    };
    const auto fetch = [&](char* to) {
        const bool on = seg < g.nseg && k + group < last;
        const uint32_t k0 = (k + group) * GEMM_BK;
        const Fetch f = {la.step(k0, seg == 2, on, to), lb.step(k0, seg == 1, on, to + UA)};
        const bool wrap = k + Cfg::GR >= last;
        k = wrap ? first : k + Cfg::GR;
        seg += wrap ? 1 : 0;
        return f;
    };
    struct Half { // a wave's fragments of 32 k
        s16x8 a[Cfg::MT], b[Cfg::NTT];
    } h0, h1;
    const auto read_one = [&](const char* from, int h, Half& to, int i) {
        if (i < Cfg::NTT) to.b[i] = fb.read(from + UA, i, h);
        else to.a[i - Cfg::NTT] = fa.read(from, i - Cfg::NTT, h);
    };
    // the products of one half, with the next half's reads and (f) a step's fetches among them
    const auto work = [&](const Half& have, const char* from, int h, Half& next, const Fetch* f) {
#pragma unroll
        for (int q = 0; q < G; ++q) {
#pragma unroll
            for (int i = q * LOADS / G; i < (q + 1) * LOADS / G; ++i)
                if (f) f->issue(i);
#pragma unroll
            for (int i = q * READS / RG; i < (q + 1) * READS / RG && i < READS; ++i) read_one(from, h, next, i);
#pragma unroll
            for (int i = q * PRODUCTS / G; i < (q + 1) * PRODUCTS / G; ++i) {
                f32x4& c = acc[i / Cfg::NTT][i % Cfg::NTT];
                c = mfma16<F16>(have.b[i % Cfg::NTT], have.a[i / Cfg::NTT], c);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    if (steps > 0) {
        const Fetch f0 = fetch(lds);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) f0.issue(i);
        const Fetch f1 = fetch(lds + Cfg::STAGE);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) f1.issue(i);
        wait_loads<LOADS>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < READS; ++i) read_one(lds, 0, h0, i);
        for (uint32_t s = 0; s < steps; ++s) {
            char *const cur = lds + (s & 1) * Cfg::STAGE, *const next = lds + (~s & 1) * Cfg::STAGE;
            const Fetch f = fetch(cur);
            work(h0, cur, 1, h1, nullptr);
            // every wave's reads of this stage and fetches of the next are done
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            work(h1, next, 0, h0, &f);
        }
        // the fetches past the end wrote zeros to LDS, which the epilogue may use
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    if (Cfg::GR > 1) { // the groups' sums, added in their order by the first
        f32x4* const sums = reinterpret_cast<f32x4*>(lds_all);
        constexpr int EACH = Cfg::MT * Cfg::NTT;
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                sums[((group - 1) * EACH + i) * Cfg::NT + threadIdx.x % Cfg::NT] = acc[i / Cfg::NTT][i % Cfg::NTT];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int q = 0; q < Cfg::GR - 1; ++q)
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                acc[i / Cfg::NTT][i % Cfg::NTT] += sums[(q * EACH + i) * Cfg::NT + threadIdx.x];
        // the epilogue's own LDS lies behind what another wave may still be reading
    }
    TileAt at;
    at.bm0 = t.m * Cfg::BM;
    at.bn0 = t.n * Cfg::BN;
    at.m0 = at.bm0 + wm * (Cfg::BM / Cfg::WM);
    at.n0 = at.bn0 + wn * (Cfg::BN / Cfg::WN);
    at.M = g.M;
    at.N = g.N;
    at.split = t.split;
    at.batch = t.batch;
    at.wm = wm;
    at.wn = wn;
    at.lds = Cfg::GR > 1 ? lds_all + (Cfg::GR - 1) * Cfg::BM * Cfg::BN * 4 : lds_all;
    epi.template run<Cfg>(acc, at);
}

// Which tile, by what each was measured to take: us for a step of 64 k of a
// round of blocks, and beside the steps (launch, first fetches, epilogue), where the
// card is full and where there is at most one block to a compute unit (L: a quarter of
// them).  From products of 2048 and 4096 k, bf16, every layout within a tenth; K's from
// short ones (orthogonalised 98 x 521 fp32: 160 us a call with 6.5 beside the steps, 122 with 8).
enum TileKind { TILE_L, TILE_M, TILE_S, TILE_K };
static double tile_time(TileKind kind, uint64_t tiles, uint64_t steps)
{
    static const struct {
        double slots, step, beside, few, few_step, few_beside;
    } t[] = {{256, 1.42, 20.0, 64, 1.07, 12.0}, {512, 0.90, 9.5, 256, 0.62, 7.0}, {1024, 0.70, 6.5, 512, 0.50, 5.0},
             {256, 0.225, 8.0, 256, 0.225, 8.0}};
    const auto& k = t[kind];
    const uint64_t full = tiles / (uint64_t)k.slots, rest = tiles % (uint64_t)k.slots;
    double us = full * (steps * k.step + k.beside);
    if (rest > 0) us += rest <= (uint64_t)k.few ? steps * k.few_step + k.few_beside : steps * k.step + k.beside;
    return us;
}
static uint64_t tile_side(TileKind kind) { return kind == TILE_L ? 256 : kind == TILE_M ? 128 : 64; }

template <class Cfg, int AL, int BL, bool F16, class Epi>
static int launch_gemm(const Gemm& g, uint32_t batch, const Epi& epi, hipStream_t st)
{
    const uint64_t tm = ceil_div(g.M, Cfg::BM), tn = ceil_div(g.N, Cfg::BN);
    if (tm == 0 || tn == 0 || batch == 0) return SG_OK;
    if (g.splits == 0 || tm * tn * g.splits * batch >= (1ull << 32) / (Cfg::NT * Cfg::GR)) return SG_EUNSUPPORTED;
    if (g.a.ld > GEMM_MAX_LD || g.b.ld > GEMM_MAX_LD) return SG_EUNSUPPORTED;
    const uint32_t blocks = tile_count<Cfg::BM, Cfg::BN>((uint32_t)tm, (uint32_t)tn, g.tri) * g.splits * batch;
    gemm_kernel<Cfg, AL, BL, F16, Epi><<<blocks, Cfg::NT * Cfg::GR, 0, st>>>(g, batch, epi);
    SG_TRY_LAUNCH();
    return SG_OK;
}

// A tile of 16-bit results, through LDS to rows of 16 bytes a lane: as the sums
// lie, a store is 32 bytes of each of 16 rows.  Rows and columns inside; the
// rows start on 16 bytes, n is the first column past the matrix.
template <class Cfg>
struct TileRows {
    static constexpr int CH = Cfg::BN / 8; // 16-byte chunks of a row
    static_assert(Cfg::BM * Cfg::BN * 2 <= Cfg::LDS, "the tile fits where the operands were");
    // where column n of the tile's row m lies; the chunk depends on the row, so that 16 rows' stores touch every bank
    static __device__ __forceinline__ uint32_t place(uint32_t m, uint32_t n)
    {
        return m * (Cfg::BN * 2) + ((n / 8) ^ (m % 16 & (CH - 1))) * 16 + n % 8 * 2;
    }
    static __device__ __forceinline__ void put(char* lds, uint32_t m, uint32_t n, s16x4 v) // four neighbours
    {
        *reinterpret_cast<s16x4*>(lds + place(m, n)) = v;
    }
    // all of the block's threads, after a barrier; f(row, column, chunk) stores one
    template <class F>
    static __device__ __forceinline__ void each(const char* lds, const F& f)
    {
        static_assert(Cfg::BM * CH % Cfg::NT == 0, "whole rounds");
#pragma unroll 4
        for (int q = 0; q < Cfg::BM * CH / Cfg::NT; ++q) {
            const uint32_t i = q * Cfg::NT + threadIdx.x, m = i / CH, c = i % CH;
            f(m, c * 8, *reinterpret_cast<const s16x8*>(lds + m * (Cfg::BN * 2) + (c ^ (m % 16 & (CH - 1))) * 16));
        }
    }
};

// eight results, of which `left` lie inside
// up to 8 elements or 4 of a row that may start anywhere: gfx950 stores 16 bytes at any element's address
__device__ __forceinline__ void store_tail(uint16_t* q, s16x8 v, uint32_t left)
{
    if (left >= 8) {
        __builtin_memcpy(q, &v, 16);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if ((uint32_t)k < left) q[k] = (uint16_t)v[k];
    }
}
__device__ __forceinline__ void store_tail(float* q, f32x4 v, uint32_t left)
{
    if (left >= 4) {
        __builtin_memcpy(q, &v, 16);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((uint32_t)k < left) q[k] = v[k];
    }
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
