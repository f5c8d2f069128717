// sg_toprows.hip -- the k largest logits of every row as COO rows with their
// log-probabilities.
//
// One pass over the row takes its softmax sum and the maximum of every line
// (8 chunks, 128 bytes) into LDS.  The line maxima give a threshold that at
// least k elements reach: every wave takes a share of the lines and finds the
// value that its share of k of them reach; the lowest of those values is the
// threshold.  Only lines that reach it are read again (some 1.5 k of them,
// from the cache), their elements above it become the candidates, in index
// order, and a radix select over the candidates gives the exact k-th largest.
// The output is everything above it and the first of its equals, which keeps
// the indices ascending and gives ties to the lowest.
//
// Rows this does not fit (more candidates than the lists hold, such as many
// equal values, or a NaN or +inf, which sort above all numbers) take an exact
// radix select over the whole row.
//
// Bound: HBM, the row read once.
#include "sg_host.h"
#include "sg_rows.h"

namespace sg {

constexpr uint32_t TR_CAP = 4096;      // candidates
constexpr uint32_t TR_LINES = 1024;    // candidate lines
constexpr uint32_t TR_MAX_LINES = 8192; // lines of a row (1 MiB)
constexpr uint32_t TR_LINE = 8;        // chunks of a line

// unsigned order of the values: -inf < ... < -0 = +0 < ... < +inf < NaN
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f); // + 0 makes -0 the same as +0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// the value of a key (+0 for both zeros)
__device__ __forceinline__ float key_value(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

struct TopArgs {
    Rows r;
    uint32_t k;
    uint32_t* idx;
    float *logp, *lse;
};

template <int NT>
struct TopShared {
    static constexpr int NW = NT / SG_WAVE;
    uint32_t key[TR_CAP], idx[TR_CAP]; // candidates, ascending in index
    uint32_t line[TR_LINES];
    uint32_t hist[256];
    RowStat part[NW];
    float low[NW];
    uint32_t scan[NW + 1];
    uint32_t sel[2]; // digit, rank left inside it
    double log_s;
    float max;
};

// which bin of the histogram (from the top) holds rank `left`, and the rank
// inside it; wave 0, four bins a lane
template <class S>
__device__ __forceinline__ void pick_digit(S& sh, uint32_t left)
{
    const uint32_t l = lane_id();
    uint32_t c[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += c[i] = sh.hist[255 - 4 * l - i];
    uint32_t before = wave_incl_scan(sum) - sum;
    if (before < left && left <= before + sum) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (before < left && left <= before + c[i]) {
                sh.sel[0] = 255 - 4 * l - i;
                sh.sel[1] = left - before;
            }
            before += c[i];
        }
    }
}

// The k-th largest of the keys that get(i), i < n, yields, and how many of
// its equals belong to the k.  low_shift = 16: the keys are those of bf16
// values, whose lower half follows from the sign.
template <int NT, class S, class Get>
__device__ __forceinline__ uint32_t radix_select(S& sh, uint32_t n, uint32_t k, int low_shift, Get get, uint32_t* ties)
{
    uint32_t prefix = 0, mask = 0, left = k;
    for (int shift = 24; shift >= low_shift; shift -= 8) {
        if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < n; i += NT) {
            const uint32_t key = get(i);
            if ((key & mask) == prefix) atomicAdd(&sh.hist[key >> shift & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < SG_WAVE) pick_digit(sh, left);
        __syncthreads();
        prefix |= sh.sel[0] << shift;
        mask |= 255u << shift;
        left = sh.sel[1];
    }
    *ties = left;
    return low_shift && !(prefix & 0x80000000u) ? prefix | 0xffffu : prefix;
}

// Writes, in index order, the elements whose key is above `kth` and the first
// `ties` of its equals.  at(i, &key, &index) yields element i < n, ascending
// in index.
template <int NT, class S, class At>
__device__ __forceinline__ void emit_rows(const TopArgs& p, S& sh, uint64_t row, uint32_t n, uint32_t kth,
                                          uint32_t ties, At at)
{
    uint32_t above = 0, equal = 0;
    const double ls = sh.log_s, m = sh.max;
    for (uint32_t base = 0; base < n; base += NT) {
        const uint32_t i = base + threadIdx.x;
        uint32_t key = 0, index = 0, total;
        if (i < n) at(i, &key, &index);
        const bool gt = i < n && key > kth, eq = i < n && key == kth;
        __syncthreads(); // the scan's words are read to the end of it
        const uint32_t pos = block_excl_scan<NT>((gt ? 1u : 0u) | (eq ? 65536u : 0u), sh.scan, &total);
        const uint32_t ng = above + (pos & 0xffffu), ne = equal + (pos >> 16);
        if (gt || (eq && ne < ties)) {
            const uint64_t to = row * p.k + ng + (ne < ties ? ne : ties);
            const float v = key_value(key);
            p.idx[to] = index;
            p.logp[to] = v == -INFINITY ? v : (float)((v - m) * p.r.it - ls);
        }
        above += total & 0xffffu;
        equal += total >> 16;
    }
}

// maximum over the 8 lanes of a line, in each of them
__device__ __forceinline__ float line_max(float v)
{
    constexpr int kQuadXor1 = 0xb1, kQuadXor2 = 0x4e, kHalfMirror = 0x141;
    v = fmaxf(v, __uint_as_float(dpp_move<kQuadXor1>(0u, __float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(dpp_move<kQuadXor2>(0u, __float_as_uint(v))));
    return fmaxf(v, __uint_as_float(dpp_move<kHalfMirror>(0u, __float_as_uint(v))));
}

// A value that at least `want` of the wave's lines reach: the want-th largest
// line maximum cut to the upper 16 bits of its key; -inf if there are not so
// many.  The wave's lines are [lo, hi), at most 64 * R.
template <int R>
__device__ __forceinline__ float lines_reach(const float* lines, uint32_t lo, uint32_t hi, uint32_t want)
{
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t l = lo + lane_id() + r * SG_WAVE;
        key[r] = l < hi ? order_key(lines[l]) >> 16 : 0u;
    }
    uint32_t t = 0;
#pragma unroll
    for (int b = 15; b >= 0; --b) {
        const uint32_t c = t | 1u << b;
        uint32_t n = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) n += popc64(ballot(key[r] >= c));
        if (n >= want) t = c;
    }
    return t <= 0x007fu ? -INFINITY : key_value(t << 16); // 0x007f....: -inf
}

template <typename E, int NT>
__global__ __launch_bounds__(NT, 8) void top_rows_kernel(TopArgs p)
{
    constexpr int VEC = RowIO<E>::VEC, NW = NT / SG_WAVE, J = 4;
    constexpr int low_shift = sizeof(E) == 2 ? 16 : 0;
    extern __shared__ float tr_lines[]; // maximum of every line
    __shared__ TopShared<NT> sh;
    const uint32_t t = threadIdx.x, V = p.r.V;
    const uint64_t row = p.r.row0 + blockIdx.x;
    const E* x = static_cast<const E*>(p.r.x) + row * p.r.ld;
    const RowSpan sp = span_of(x, V);
    const E* xc = x + sp.head;
    const uint32_t nl = (sp.nc + TR_LINE - 1) / TR_LINE;
    const bool lined = V > TR_CAP && nl <= TR_MAX_LINES; // else all elements are candidates, or none

    RowStat st = {-INFINITY, 0.f};
#pragma unroll 1
    for (uint32_t j0 = t; j0 / TR_LINE < nl; j0 += J * NT) { // whole lines, so that their 8 lanes stay together
        u32x4 w[J];
        load_chunks<J, NT>(w, xc, j0, sp.nc);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t c = j0 + j * NT;
            float m = -INFINITY;
            if (c < sp.nc) {
                float v[VEC];
                RowIO<E>::unpack(w[j], v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[i]);
                stat_add<VEC>(st, v, p.r.c);
                if (V <= TR_CAP)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sh.key[sp.head + c * VEC + i] = order_key(v[i]);
            }
            if (lined) {
                m = line_max(m);
                if (c % TR_LINE == 0 && c < sp.nc) tr_lines[c / TR_LINE] = m;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (t < 2 * VEC) {
        const uint32_t i = loose_element(sp, VEC, t);
        if (i < V) {
            const float v = RowIO<E>::get(x + i);
            stat_add<1>(st, &v, p.r.c);
            if (V <= TR_CAP) sh.key[i] = order_key(v);
        }
    }
    st = wave_stat(st, p.r.c);
    if (lane_id() == 0) sh.part[t / SG_WAVE] = st;
    __syncthreads();
    st = sh.part[0];
#pragma unroll 1
    for (int w = 1; w < NW; ++w) st = stat_join(st, sh.part[w], p.r.c);
    if (t == 0) {
        sh.log_s = row_log((double)st.s);
        sh.max = shift_of(st.m);
        if (p.lse) p.lse[row] = (float)(sh.max * p.r.it + sh.log_s);
    }
    uint32_t n = V <= TR_CAP ? V : 0; // candidates; 0: none found this way
    if (lined && st.s == st.s) {
        const uint32_t w = uniform(t / SG_WAVE);
        const uint32_t lo = (uint32_t)((uint64_t)nl * w / NW), hi = (uint32_t)((uint64_t)nl * (w + 1) / NW);
        const uint32_t want = (p.k + NW - 1) / NW;
        constexpr int RMAX = (TR_MAX_LINES / NW + SG_WAVE - 1) / SG_WAVE;
        const float reach = hi - lo <= 2 * SG_WAVE ? lines_reach<2>(tr_lines, lo, hi, want)
                                                   : lines_reach<RMAX>(tr_lines, lo, hi, want);
        if (lane_id() == 0) sh.low[w] = reach;
        __syncthreads();
        float low = sh.low[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) low = fminf(low, sh.low[i]);
        if (low > -INFINITY) {
            // the lines that reach it, in order
            uint32_t nlc = 0;
            for (uint32_t base = 0; base < nl; base += NT) {
                const uint32_t l = base + t;
                const bool in = l < nl && tr_lines[l] >= low;
                uint32_t total;
                const uint32_t pos = nlc + block_excl_scan<NT>(in ? 1u : 0u, sh.scan, &total);
                if (in && pos < TR_LINES) sh.line[pos] = l;
                nlc += total;
                __syncthreads();
            }
            if (nlc <= TR_LINES) {
                // their elements that reach it, with those outside the chunks, in order: a lane per
                // chunk, lane 0 the elements before the chunks, the last lane those after
                const uint32_t items = 8 * nlc + 2;
                for (uint32_t base = 0; base < items; base += NT) {
                    const uint32_t q = base + t;
                    float v[VEC];
                    uint32_t first = 0, len = 0;
                    if (q == 0) {
                        len = sp.head;
                    } else if (q == items - 1) {
                        first = sp.head + sp.nc * VEC;
                        len = V - first;
                    } else if (q < items) {
                        const uint32_t c = sh.line[(q - 1) / 8] * TR_LINE + (q - 1) % 8;
                        first = sp.head + c * VEC;
                        if (c < sp.nc) len = VEC;
                    }
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[i] = -INFINITY;
                    if (len == VEC) RowIO<E>::unpack(load_chunk(x + first), v);
                    else
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            if (i < (int)len) v[i] = RowIO<E>::get(x + first + i);
                    uint32_t c = 0, total;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) c += v[i] >= low ? 1u : 0u;
                    uint32_t pos = n + block_excl_scan<NT>(c, sh.scan, &total);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        if (v[i] >= low) {
                            if (pos < TR_CAP) {
                                sh.key[pos] = order_key(v[i]);
                                sh.idx[pos] = first + i;
                            }
                            ++pos;
                        }
                    }
                    n += total;
                    __syncthreads();
                }
                if (n > TR_CAP) n = 0;
            }
        }
    }
    __syncthreads();
    uint32_t ties;
    if (n > 0) {
        const uint32_t kth = radix_select<NT>(sh, n, p.k, low_shift, [&](uint32_t i) { return sh.key[i]; }, &ties);
        const bool all = V <= TR_CAP;
        emit_rows<NT>(p, sh, row, n, kth, ties, [&](uint32_t i, uint32_t* key, uint32_t* index) {
            *key = sh.key[i];
            *index = all ? i : sh.idx[i];
        });
    } else {
        const uint32_t kth = radix_select<NT>(sh, V, p.k, 0, [&](uint32_t i) { return order_key(RowIO<E>::get(x + i)); },
                                              &ties);
        emit_rows<NT>(p, sh, row, V, kth, ties, [&](uint32_t i, uint32_t* key, uint32_t* index) {
            *key = order_key(RowIO<E>::get(x + i));
            *index = i;
        });
    }
}

template <typename E, int NT>
static int launch_top(const RowCheck& c, TopArgs p, hipStream_t st)
{
    const uint64_t lines = ceil_div(c.r.V / RowIO<E>::VEC + 1, TR_LINE);
    const size_t lds = c.r.V > TR_CAP && lines <= TR_MAX_LINES ? lines * sizeof(float) : 0;
    for (p.r.row0 = 0; p.r.row0 < p.r.T; p.r.row0 += ROWS_PER_LAUNCH) {
        const uint64_t left = p.r.T - p.r.row0;
        top_rows_kernel<E, NT><<<(unsigned)(left < ROWS_PER_LAUNCH ? left : ROWS_PER_LAUNCH), NT, lds, st>>>(p);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
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
    const bool wide = V * row_esize(dt) > 32768;
    if (dt == SG_BF16) return wide ? launch_top<bf16_bits, 1024>(c, p, st) : launch_top<bf16_bits, 256>(c, p, st);
    return wide ? launch_top<float, 1024>(c, p, st) : launch_top<float, 256>(c, p, st);
}
