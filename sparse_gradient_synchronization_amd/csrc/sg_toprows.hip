// sg_toprows.hip -- the k largest logits of every row as COO rows with their
// log-probabilities.
//
// Selection is exact: a radix select of the k-th largest order key of the
// row, then one ordered pass that writes what lies above it and the first of
// its equals, so the indices come out ascending and ties go to the lowest.
//
// Bound: HBM, the row read once.
#include "sg_host.h"
#include "sg_rows.h"

namespace sg {

constexpr int TR_NT = 256;

// unsigned order of the values: -inf < ... < -0 = +0 < ... < +inf < NaN
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f); // + 0 makes -0 the same as +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

struct TopArgs {
    Rows r;
    uint32_t k;
    uint32_t* idx;
    float *logp, *lse;
};

template <typename E>
__global__ __launch_bounds__(TR_NT) void top_rows_kernel(TopArgs p)
{
    constexpr int VEC = RowIO<E>::VEC, NT = TR_NT, NW = NT / SG_WAVE;
    __shared__ uint32_t hist[256];
    __shared__ RowStat part[NW];
    __shared__ uint32_t sel[2]; // digit, rank left inside it
    __shared__ double log_s; // log S
    __shared__ float max_s;
    __shared__ uint32_t scan[NW + 1];
    const uint32_t t = threadIdx.x, V = p.r.V, nc = V / VEC;
    for (uint64_t row = blockIdx.x; row < p.r.T; row += gridDim.x) {
        const E* x = static_cast<const E*>(p.r.x) + row * p.r.ld;
        RowStat st = {-INFINITY, 0.f};
        for (uint32_t j = t; j < nc; j += NT) {
            float v[VEC];
            RowIO<E>::unpack(load_chunk(x + (uint64_t)j * VEC), v);
            stat_add<VEC>(st, v, p.r.c);
        }
        for (uint32_t i = nc * VEC + t; i < V; i += NT) {
            float v = RowIO<E>::get(x + i);
            stat_add<1>(st, &v, p.r.c);
        }
        st = wave_stat(st, p.r.c);
        if (lane_id() == 0) part[t / SG_WAVE] = st;
        __syncthreads();
        if (t == 0) {
            RowStat a = part[0];
            for (int w = 1; w < NW; ++w) a = stat_join(a, part[w], p.r.c);
            log_s = log((double)a.s);
            max_s = shift_of(a.m);
            if (p.lse) p.lse[row] = (float)(max_s * p.r.it + log_s);
        }
        // radix select: bits 31..24, 23..16, ...
        uint32_t prefix = 0, mask = 0, left = p.k;
        for (int shift = 24; shift >= 0; shift -= 8) {
            hist[t] = 0;
            __syncthreads();
            for (uint32_t i = t; i < V; i += NT) {
                const uint32_t key = order_key(RowIO<E>::get(x + i));
                if ((key & mask) == prefix) atomicAdd(&hist[key >> shift & 255u], 1u);
            }
            __syncthreads();
            if (t == 0) {
                uint32_t d = 255, before = 0;
                while (d > 0 && before + hist[d] < left) before += hist[d--];
                sel[0] = d;
                sel[1] = left - before;
            }
            __syncthreads();
            prefix |= sel[0] << shift;
            mask |= 255u << shift;
            left = sel[1];
        }
        // everything above `prefix`, and the first `left` of its equals
        uint32_t above = 0, equal = 0;
        const double ls = log_s, m = max_s;
        for (uint32_t base = 0; base < V; base += NT) {
            const uint32_t i = base + t;
            const float v = i < V ? RowIO<E>::get(x + i) : 0.f;
            const uint32_t key = i < V ? order_key(v) : 0u;
            const bool gt = i < V && key > prefix, eq = i < V && key == prefix;
            uint32_t total;
            __syncthreads();
            const uint32_t pos = block_excl_scan<NT>((gt ? 1u : 0u) | (eq ? 65536u : 0u), scan, &total);
            const uint32_t ng = above + (pos & 0xffffu), ne = equal + (pos >> 16);
            if (gt || (eq && ne < left)) {
                const uint64_t at = row * p.k + ng + (ne < left ? ne : left);
                p.idx[at] = i;
                p.logp[at] = v == -INFINITY ? v : (float)((v - m) * p.r.it - ls);
            }
            above += total & 0xffffu;
            equal += total >> 16;
        }
        __syncthreads();
    }
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_topk_rows_workspace_bytes(uint64_t T, uint64_t V, uint32_t k, sg_dtype dt) { return 0; }

extern "C" int sg_topk_rows(const void* d_logits, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld, double inv_temp,
                            uint32_t k, uint32_t* d_idx, float* d_logp, float* d_lse, void* d_ws, size_t ws_bytes,
                            void* stream)
{
    RowCheck c;
    int rc = rows_args(d_logits, dt, T, V, ld, inv_temp, &c);
    if (rc) return rc;
    if (k == 0 || k > V) return SG_EINVAL;
    if (T > 0 && (!d_idx || !d_logp)) return SG_EINVAL;
    if (k > SG_ROWS_MAX_K) return SG_EUNSUPPORTED;
    if (T == 0) return SG_OK;
    TopArgs p = {c.r, k, d_idx, d_logp, d_lse};
    hipStream_t st = as_stream(stream);
    if (dt == SG_BF16) top_rows_kernel<bf16_bits><<<c.grid, TR_NT, 0, st>>>(p);
    else top_rows_kernel<float><<<c.grid, TR_NT, 0, st>>>(p);
    SG_TRY_LAUNCH();
    return SG_OK;
}
