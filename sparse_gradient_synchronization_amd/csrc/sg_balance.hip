// sg_balance.hip -- balance loss of a router over its experts.  With p_t the
// softmax of a row of E logits, N rows that count, c_e how often expert e was
// chosen, f_e = c_e / (k N) and P_e the mean of p_te:
//   loss = alpha E sum_e f_e P_e + zc mean lse^2
//   d loss / d logit_te = p_te (h_e - sum_i h_i p_ti + 2 zc lse_t / N),  h_e = alpha E f_e / N
// The gradient needs the counts and not P, so the logits are read once:
// balance_count_kernel counts; balance_rows_kernel does softmax, column sums
// and gradient in registers; balance_loss_kernel adds the column sums up.  (The
// last block of the rows could, but the fence before it counts itself done
// writes the whole gradient back from the caches: 114 us instead of 40.)  Few
// elements: one block does it all.
//
// A row is a group of L lanes, VEC neighbouring columns to each, C times; a
// thread has U rows under way, or the loads of a compute unit's one block
// would not cover the memory's latency (65536 x 256 fp32: 46 us with one row).
// Counts are whole numbers; column sums are fp32 over a lane's own rows,
// joined in a fixed order.
#include "sg_rows.h"

namespace sg {

constexpr uint32_t BL_MAX_E = 1024;
constexpr int BL_NT = 1024, BL_WAVES = BL_NT / 64;
constexpr uint32_t BL_COUNT_BLOCKS = 64; // their counts are added up by every block of the next kernel
constexpr uint32_t BL_FEW = 32768;       // elements that one block takes alone
constexpr uint32_t BL_BLOCKS = 256;

struct BalArgs {
    const void* x;
    uint64_t T, ld;
    uint32_t E, k, L; // L: lanes of a row, a power of two
    const int32_t* idx;
    const uint8_t* live;
    float* loss;
    int32_t* counts;
    float* prob;
    void* grad;
    uint64_t ld_grad;
    double alpha, zc;
    uint32_t* count_part; // [count blocks][E + 1], the last one: rows that count
    float* prob_part;     // [blocks][E]
    double* z_part;       // [blocks]
    uint32_t* hist;       // [E + 1] the counts, from the first block of the rows
};

// the block's share of the counts, in LDS: hist[E] and the rows that count in hist[E]
__device__ __forceinline__ void bal_count(const BalArgs& a, uint32_t block, uint32_t blocks, uint32_t* hist)
{
    for (uint32_t e = threadIdx.x; e <= a.E; e += BL_NT) hist[e] = 0;
    __syncthreads();
    const uint32_t n = (uint32_t)(a.T * a.k), step = blocks * BL_NT; // n < 2^31
    for (uint32_t i = block * BL_NT + threadIdx.x; i < n; i += step) {
        const uint32_t t = i / a.k;
        if (a.live && !a.live[t]) continue;
        const uint32_t e = (uint32_t)a.idx[i];
        if (e < a.E) atomicAdd(&hist[e], 1u);
        if (i == t * a.k) atomicAdd(&hist[a.E], 1u);
    }
    __syncthreads();
}

__global__ __launch_bounds__(BL_NT) void balance_count_kernel(BalArgs a)
{
    __shared__ uint32_t hist[BL_MAX_E + 1];
    bal_count(a, blockIdx.x, gridDim.x, hist);
    for (uint32_t e = threadIdx.x; e <= a.E; e += BL_NT) a.count_part[blockIdx.x * (a.E + 1) + e] = hist[e];
}

template <typename T, int VEC, int C>
struct BalRow {
    float v[C][VEC];
    // columns (i L + lane) VEC ..; what is past the row's end is -inf
    __device__ __forceinline__ void load(const BalArgs& a, const T* x, uint32_t lane)
    {
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const uint32_t c = (i * a.L + lane) * VEC;
            const bool in = c < a.E; // whole: E is a multiple of VEC
            T w[VEC];
            if (in) __builtin_memcpy(w, __builtin_assume_aligned(x + c, VEC * sizeof(T)), VEC * sizeof(T));
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[i][j] = in ? RowIO<T>::get(&w[j]) : -INFINITY;
        }
    }
};

__device__ __forceinline__ float group_max(float v, uint32_t L)
{
    for (uint32_t d = 1; d < L; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float group_sum(float v, uint32_t L)
{
    for (uint32_t d = 1; d < L; d *= 2) v += __shfl_xor(v, d);
    return v;
}

// All rows of this block.  h: [E] of the gradient, in LDS; n: rows that count.
// Leaves the column sums in sums[E] and the sum of lse^2 in *z (thread 0).
template <typename T, int VEC, int C, int U>
__device__ __forceinline__ void bal_rows(const BalArgs& a, uint32_t block, uint32_t blocks, const float* h, double n,
                                         float (*wave_sums)[BL_MAX_E], float* sums, double* z)
{
    const uint32_t per = BL_NT / a.L, lane = threadIdx.x % a.L, mine = threadIdx.x / a.L;
    float hl[C][VEC], cs[C][VEC];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const uint32_t c = (i * a.L + lane) * VEC + j;
            hl[i][j] = c < a.E ? h[c] : 0.f;
            cs[i][j] = 0.f;
        }
    const float zs = n > 0.0 ? (float)(2.0 * a.zc / n) : 0.f;
    double zsum = 0.0;
    const T* const x = static_cast<const T*>(a.x);
    for (uint64_t t0 = (uint64_t)block * per + mine; t0 < a.T; t0 += (uint64_t)blocks * per * U) {
        BalRow<T, VEC, C> rows[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint64_t t = t0 + (uint64_t)u * blocks * per;
            live[u] = t < a.T && (!a.live || a.live[t]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (live[u]) {
                rows[u].load(a, x + (t0 + (uint64_t)u * blocks * per) * a.ld, lane);
            } else {
#pragma unroll
                for (int i = 0; i < C; ++i)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) rows[u].v[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            BalRow<T, VEC, C>& r = rows[u];
            const uint64_t t = t0 + (uint64_t)u * blocks * per;
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) m = fmaxf(m, r.v[i][j]);
            m = group_max(m, a.L);
            const float shift = shift_of(m);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    r.v[i][j] = exp2_fast((r.v[i][j] - shift) * 1.44269504f);
                    s += r.v[i][j];
                }
            s = group_sum(s, a.L);
            const float inv = live[u] ? 1.f / s : 0.f, lse = shift + logf(s);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    r.v[i][j] *= inv;
                    cs[i][j] += r.v[i][j];
                    dot = fmaf(hl[i][j], r.v[i][j], dot);
                }
            if (live[u] && lane == 0) zsum += (double)lse * lse;
            if (!a.grad) continue;
            dot = group_sum(dot, a.L);
            const float add = live[u] ? zs * lse - dot : 0.f;
            T* const g = static_cast<T*>(a.grad) + t * a.ld_grad;
            if (t >= a.T) continue;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const uint32_t c = (i * a.L + lane) * VEC;
                T w[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) RowIO<T>::put(&w[j], r.v[i][j] * (hl[i][j] + add));
                if (c < a.E) __builtin_memcpy(__builtin_assume_aligned(g + c, VEC * sizeof(T)), w, VEC * sizeof(T));
            }
        }
    }
    // the wave's groups, then the block's waves
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            for (uint32_t d = a.L; d < 64; d *= 2) cs[i][j] += __shfl_xor(cs[i][j], d);
            const uint32_t c = (i * a.L + lane) * VEC + j;
            if (threadIdx.x % 64 < a.L && c < a.E) wave_sums[threadIdx.x / 64][c] = cs[i][j];
        }
    for (uint32_t d = 1; d < 64; d *= 2) zsum += __shfl_xor(zsum, d);
    __shared__ double zw[BL_WAVES];
    if (threadIdx.x % 64 == 0) zw[threadIdx.x / 64] = zsum;
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < a.E; c += BL_NT) {
        float q = 0.f;
        for (int w = 0; w < BL_WAVES; ++w) q += wave_sums[w][c];
        sums[c] = q;
    }
    if (threadIdx.x == 0) {
        double q = 0.0;
        for (int w = 0; w < BL_WAVES; ++w) q += zw[w];
        *z = q;
    }
}

// h_e from a count
__device__ __forceinline__ float bal_slope(const BalArgs& a, uint32_t count, double n)
{
    return n > 0.0 ? (float)(a.alpha * a.E * (double)count / (a.k * n) / n) : 0.f;
}

// part[0 .. n)[stride] of column e, in fp64, by as many threads a column as
// there are; every thread of a column's first slice gets its sum in lds[e]
template <typename T, typename S>
__device__ __forceinline__ void bal_columns(const T* part, uint32_t n, uint32_t stride, uint32_t cols, S* lds, S* sums)
{
    uint32_t slices = BL_NT / cols; // lds: [slices][cols], at most BL_NT
    slices = slices < 1 ? 1 : slices > n ? n : slices;
    const uint32_t sl = threadIdx.x / cols;
    if (cols <= BL_NT) {
        const uint32_t e = threadIdx.x % cols;
        if (sl < slices) {
            S q = 0;
            constexpr uint32_t U = 16; // loads under way (65536 x 256 fp32: 58.4 us a call, with 8 58.7; 4096 x 1024 bf16 40.2, 42.3)
            for (uint32_t b = sl; b < n; b += U * slices) {
                T v[U];
#pragma unroll
                for (uint32_t i = 0; i < U; ++i)
                    v[i] = part[(b + i * slices < n ? b + i * slices : b) * stride + e];
#pragma unroll
                for (uint32_t i = 0; i < U; ++i) q += b + i * slices < n ? (S)v[i] : (S)0;
            }
            lds[sl * cols + e] = q;
        }
        __syncthreads();
        if (threadIdx.x < cols) {
            S q = 0;
            for (uint32_t i = 0; i < slices; ++i) q += lds[i * cols + e];
            sums[e] = q;
        }
    } else { // one column more than threads: the counts of 1024 experts and the rows
        for (uint32_t e = threadIdx.x; e < cols; e += BL_NT) {
            S q = 0;
            for (uint32_t b = 0; b < n; ++b) q += (S)part[(uint64_t)b * stride + e];
            sums[e] = q;
        }
    }
    __syncthreads();
}

// the loss from counts and column sums (in LDS) and the sum of lse^2; one block
__device__ __forceinline__ void bal_loss(const BalArgs& a, const uint32_t* hist, const double* sums, double z)
{
    const double n = (double)hist[a.E];
    double s = 0.0;
    for (uint32_t e = threadIdx.x; e < a.E; e += BL_NT) {
        const double q = n > 0.0 ? sums[e] / n : 0.0;
        a.prob[e] = (float)q;
        a.counts[e] = (int32_t)hist[e];
        s += n > 0.0 ? (double)hist[e] / (a.k * n) * q : 0.0;
    }
    for (uint32_t d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    __shared__ double w[BL_WAVES];
    if (threadIdx.x % 64 == 0) w[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double q = 0.0;
        for (int i = 0; i < BL_WAVES; ++i) q += w[i];
        *a.loss = (float)(q * a.alpha * a.E + (n > 0.0 ? a.zc * z / n : 0.0));
    }
}

template <typename T, int VEC, int C, int U>
__global__ __launch_bounds__(BL_NT) void balance_rows_kernel(BalArgs a, uint32_t count_blocks)
{
    __shared__ uint32_t hist[BL_MAX_E + 1];
    __shared__ float h[BL_MAX_E];
    __shared__ union {
        float waves[BL_WAVES][BL_MAX_E];
        uint32_t counts[BL_NT];
    } lds;
    bal_columns(a.count_part, count_blocks, a.E + 1, a.E + 1, lds.counts, hist);
    const double n = (double)hist[a.E];
    for (uint32_t e = threadIdx.x; e < a.E; e += BL_NT) h[e] = bal_slope(a, hist[e], n);
    if (blockIdx.x == 0)
        for (uint32_t e = threadIdx.x; e <= a.E; e += BL_NT) a.hist[e] = hist[e];
    __syncthreads();
    bal_rows<T, VEC, C, U>(a, blockIdx.x, gridDim.x, h, n, lds.waves, a.prob_part + (uint64_t)blockIdx.x * a.E,
                           a.z_part + blockIdx.x);
}

__global__ __launch_bounds__(BL_NT) void balance_loss_kernel(BalArgs a, uint32_t blocks)
{
    __shared__ uint32_t hist[BL_MAX_E + 1];
    __shared__ double sums[BL_MAX_E], slices[BL_NT];
    for (uint32_t e = threadIdx.x; e <= a.E; e += BL_NT) hist[e] = a.hist[e];
    bal_columns(a.prob_part, blocks, a.E, a.E, slices, sums);
    double z = 0.0;
    if (threadIdx.x < 64) {
        for (uint32_t b = threadIdx.x; b < blocks; b += 64) z += a.z_part[b];
        for (uint32_t d = 1; d < 64; d *= 2) z += __shfl_xor(z, d);
    }
    bal_loss(a, hist, sums, z);
}

template <typename T, int VEC, int C>
__global__ __launch_bounds__(BL_NT) void balance_few_kernel(BalArgs a)
{
    __shared__ uint32_t hist[BL_MAX_E + 1];
    __shared__ float h[BL_MAX_E], waves[BL_WAVES][BL_MAX_E], cols[BL_MAX_E];
    __shared__ double sums[BL_MAX_E], z;
    bal_count(a, 0, 1, hist);
    const double n = (double)hist[a.E];
    for (uint32_t e = threadIdx.x; e < a.E; e += BL_NT) h[e] = bal_slope(a, hist[e], n);
    __syncthreads();
    bal_rows<T, VEC, C, 1>(a, 0, 1, h, n, waves, cols, &z);
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < a.E; e += BL_NT) sums[e] = cols[e];
    bal_loss(a, hist, sums, z);
}

struct BalWs {
    uint32_t* count_part;
    float* prob_part;
    double* z_part;
    uint32_t* hist;
};
static BalWs bal_carve(Carver& cv, uint32_t E)
{
    BalWs w;
    w.count_part = cv.take<uint32_t>((uint64_t)BL_COUNT_BLOCKS * (E + 1));
    w.prob_part = cv.take<float>((uint64_t)BL_BLOCKS * E);
    w.z_part = cv.take<double>(BL_BLOCKS);
    w.hist = cv.take<uint32_t>(E + 1);
    return w;
}

template <typename T, int VEC, int C>
static int bal_launch(const BalArgs& a, hipStream_t st)
{
    // One launch instead of three while its one block is not the longer way.  us a call, one block and three
    // launches: 256 x 64 fp32 13, 20; 512 x 64 17, 20; 2048 x 16 17, 20; 256 x 256 33, 20; 4096 x 16 28, 20
    if (a.T * a.E <= BL_FEW) {
        balance_few_kernel<T, VEC, C><<<1, BL_NT, 0, st>>>(a);
        SG_TRY_LAUNCH();
        return SG_OK;
    }
    constexpr int U = VEC * C <= 4 ? 4 : VEC * C <= 8 ? 2 : 1; // 16 registers of row
    const uint64_t cb = ceil_div(a.T * a.k, 4 * BL_NT), rb = ceil_div(a.T, BL_NT / a.L);
    const uint32_t count_blocks = (uint32_t)(cb < BL_COUNT_BLOCKS ? cb : BL_COUNT_BLOCKS),
                   blocks = (uint32_t)(rb < BL_BLOCKS ? rb : BL_BLOCKS);
    balance_count_kernel<<<count_blocks, BL_NT, 0, st>>>(a);
    SG_TRY_LAUNCH();
    balance_rows_kernel<T, VEC, C, U><<<blocks, BL_NT, 0, st>>>(a, count_blocks);
    SG_TRY_LAUNCH();
    balance_loss_kernel<<<1, BL_NT, 0, st>>>(a, blocks);
    SG_TRY_LAUNCH();
    return SG_OK;
}

template <typename T>
static int bal_dispatch(BalArgs& a, hipStream_t st)
{
    const auto on = [](const void* p, uint64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && ld % 4 == 0;
    };
    const bool vec = a.E % 4 == 0 && on(a.x, a.ld) && (!a.grad || on(a.grad, a.ld_grad));
    const uint32_t units = vec ? a.E / 4 : a.E;
    a.L = 1;
    while (a.L < units && a.L < 64) a.L *= 2;
    const uint32_t c = (units + 63) / 64;
    if (vec) return c <= 1 ? bal_launch<T, 4, 1>(a, st) : c <= 2 ? bal_launch<T, 4, 2>(a, st) : bal_launch<T, 4, 4>(a, st);
    return c <= 1 ? bal_launch<T, 1, 1>(a, st) : c <= 4 ? bal_launch<T, 1, 4>(a, st) : bal_launch<T, 1, 16>(a, st);
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_balance_workspace_bytes(uint64_t T, uint32_t E, uint32_t k, sg_dtype dt)
{
    if (E == 0 || E > BL_MAX_E || T * E <= BL_FEW) return 0;
    Carver cv(nullptr);
    bal_carve(cv, E);
    return cv.bytes();
}

extern "C" int sg_balance_loss(const void* d_logits, sg_dtype dt, uint64_t T, uint32_t E, uint64_t ld,
                               const int32_t* d_idx, uint32_t k, const uint8_t* d_live, double balance_coef,
                               double z_coef, float* d_loss, int32_t* d_counts, float* d_prob, void* d_grad,
                               uint64_t ld_grad, void* d_ws, size_t ws_bytes, void* stream)
{
    if ((dt != SG_F32 && dt != SG_BF16) || E == 0 || k == 0 || T >= (1ull << 31)) return SG_EINVAL;
    if (!(balance_coef >= 0.0) || !(balance_coef <= 1e6) || !(z_coef >= 0.0) || !(z_coef <= 1e6)) return SG_EINVAL;
    const uint64_t es = dt == SG_F32 ? 4 : 2, far = 1ull << 40;
    if (ld < E || ld >= far || (d_grad && (ld_grad < E || ld_grad >= far))) return SG_EINVAL;
    if (reinterpret_cast<uintptr_t>(d_logits) % es || reinterpret_cast<uintptr_t>(d_grad) % es) return SG_EINVAL;
    if (d_grad == d_logits && d_grad && ld_grad != ld) return SG_EINVAL;
    if (!d_loss || !d_counts || !d_prob || (T > 0 && (!d_logits || !d_idx))) return SG_EINVAL;
    if (E > BL_MAX_E || k > E || T * k >= (1ull << 31)) return SG_EUNSUPPORTED;
    const size_t need = sg_balance_workspace_bytes(T, E, k, dt);
    if (need > 0 && !d_ws) return SG_EINVAL;
    if (ws_bytes < need) return SG_ECAPACITY;
    Carver cv(d_ws);
    const BalWs w = bal_carve(cv, E);
    BalArgs a = {d_logits, T, ld, E, k, 1, d_idx, d_live, d_loss, d_counts, d_prob, d_grad, ld_grad, balance_coef,
                 z_coef, w.count_part, w.prob_part, w.z_part, w.hist};
    if (dt == SG_BF16) return bal_dispatch<bf16_bits>(a, as_stream(stream));
    return bal_dispatch<float>(a, as_stream(stream));
}
