// sg_toprows.hip -- the k largest logits of every row as COO rows with their
// log-probabilities.
//
// One pass over the row takes its softmax sum and the maximum of every group
// of neighbouring elements.  The group maxima give a threshold that at least k
// elements reach, cheaply: it need not be the k-th largest, only not above it.
// The elements that reach it (some 1.5 k) become the candidates, in index
// order, and the exact k-th largest is found among them.  The output is
// everything above it and the first of its equals, which keeps the indices
// ascending and gives ties to the lowest.
//
// Rows of up to 8 KiB: one wave holds the row in registers; a group is a
// 16-byte chunk.  Longer rows: one block; a group is a line of 8 chunks whose
// maximum goes to LDS, and only the lines that reach the threshold are read
// again (from the cache).  Few long rows: blocks take parts of a row and leave
// the k largest of each, which another block joins.
//
// Rows this does not fit take an exact radix select over the whole row: more
// candidates than the list holds (many equal values, or a region of the row well
// below the rest, since the threshold is the lowest of the waves' regions), more
// lines than LDS holds, a NaN or +inf, which sort above all numbers.  It costs some
// ten times the one pass (2000 x 262208 fp32, k = 64: 3635 us, 376 for 262144).
//
// Bound: HBM, the row read once.
#include "sg_host.h"
#include "sg_rows.h"

namespace sg {

constexpr uint32_t TR_LINE = 8;          // chunks of a line (1 where the row has few lines for its k)
constexpr uint32_t TR_MAX_LINES = 8192;  // lines of a row (1 MiB)

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

// the key of the k-th largest from its digits above low_shift (16: bf16 values, whose lower half follows from the sign)
__device__ __forceinline__ uint32_t whole_key(uint32_t prefix, int low_shift)
{
    return low_shift && !(prefix & 0x80000000u) ? prefix | 0xffffu : prefix;
}

// a threshold from the upper half of a key, cut down; -inf stays -inf
__device__ __forceinline__ float cut_value(uint32_t upper) { return upper <= 0x007fu ? -INFINITY : key_value(upper << 16); }

struct TopArgs {
    Rows r;
    uint32_t k;
    uint32_t* idx;
    float *logp, *lse;
    uint32_t shift; // a line is 1 << shift chunks
    bool lined;     // the LDS has room for the maxima of the lines of V elements, or of len
    // parts of a row: candidates and sums of each part
    uint32_t parts, len;
    uint32_t *part_key, *part_idx; // [rows][parts][k]
    RowStat* part_stat;            // [rows][parts]
};

// log-probability of a value; a NaN in the row (log_s is NaN then) stays
__device__ __forceinline__ float top_logp(float v, float m, double log_s, double it)
{
    return v == -INFINITY && log_s == log_s ? v : (float)(((double)v - m) * it - log_s);
}

// ---------------------------------------------------------------------------
// short rows: a wave per row
// ---------------------------------------------------------------------------
constexpr int TW_R = 8;             // chunks of a lane
constexpr uint32_t TW_CAP = 1024;   // candidates
constexpr uint32_t TW_MAX_K = 256;  // longer lists leave too many candidates

// the k-th largest of the keys a wave holds: count(c) says how many are at
// least c; from bit 31 down to low_bit
template <class Count>
__device__ __forceinline__ uint32_t wave_kth(uint32_t k, int low_bit, Count count)
{
    uint32_t t = 0;
    for (int b = 31; b >= low_bit; --b) {
        const uint32_t c = t | 1u << b;
        if (count(c) >= k) t = c;
    }
    return t;
}

// Passes on, in index order, the elements whose key is above `kth` and the
// first `ties` of its equals; at(i, &key, &index) yields element i < n.
template <class At, class Put>
__device__ __forceinline__ void wave_emit(uint32_t n, uint32_t kth, uint32_t ties, At at, Put put)
{
    uint32_t to = 0, equal = 0;
    for (uint32_t base = 0; base < n; base += SG_WAVE) {
        const uint32_t i = base + lane_id();
        uint32_t key = 0, index = 0;
        if (i < n) at(i, &key, &index);
        const bool eq = i < n && key == kth;
        const uint64_t eqs = ballot(eq);
        const bool sel = (i < n && key > kth) || (eq && equal + count_below(eqs) < ties);
        const uint64_t sels = ballot(sel);
        if (sel) put(to + count_below(sels), key, index);
        to += popc64(sels);
        equal += popc64(eqs);
    }
}

template <typename E>
__global__ __launch_bounds__(SG_WAVE, 6) void top_wave_kernel(TopArgs p)
{
    constexpr int VEC = RowIO<E>::VEC, R = TW_R;
    constexpr int low_shift = sizeof(E) == 2 ? 16 : 0;
    __shared__ uint32_t ckey[TW_CAP];
    __shared__ uint16_t cidx[TW_CAP]; // a row here has at most 4096 elements
    const uint32_t l = threadIdx.x, V = p.r.V, k = p.k;
    const uint64_t row = p.r.row0 + blockIdx.x;
    const E* x = static_cast<const E*>(p.r.x) + row * p.r.ld;
    const uint32_t nc = V / VEC, nr = (V + SG_WAVE * VEC - 1) / (SG_WAVE * VEC); // whole chunks, rounds
    u32x4 w[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t c = l + r * SG_WAVE;
        if (c < nc) {
            w[r] = load_chunk(chunk_at<E>(x, r * SG_WAVE, l));
        } else { // the last, short chunk; -inf past the row's end
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] = c * VEC + i < V ? RowIO<E>::get(x + c * VEC + i) : -INFINITY;
            w[r] = RowIO<E>::pack(v);
        }
    }
    RowStat st = {-INFINITY, 0.0};
    uint32_t top[R]; // upper half of the key of each chunk's maximum
#pragma unroll
    for (int r = 0; r < R; ++r) {
        top[r] = 0;
        if ((uint32_t)r < nr) {
            float v[VEC], m = -INFINITY;
            RowIO<E>::unpack(w[r], v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[i]);
            stat_add<VEC>(st, v, p.r.c);
            top[r] = order_key(m) >> 16;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    st = wave_stat(st, p.r.c);
    const double log_s = row_log(st.s);
    const float m = shift_of(st.m);
    if (l == 0 && p.lse) p.lse[row] = (float)(m * p.r.it + log_s);

    float low = -INFINITY;
    uint32_t n = TW_CAP + 1;
    if (st.s == st.s) {
        const uint32_t t = wave_kth(k, 16, [&](uint32_t c) {
            uint32_t h = 0;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if ((uint32_t)r < nr) h += popc64(ballot(top[r] >= c >> 16));
            return h;
        });
        low = cut_value(t >> 16);
        // the candidates, in index order: round by round, the lanes' counts scanned
        n = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if ((uint32_t)r < nr) {
                float v[VEC];
                RowIO<E>::unpack(w[r], v);
                const uint32_t first = (l + r * SG_WAVE) * VEC;
                uint32_t c = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) c += v[i] >= low && first + i < V ? 1u : 0u;
                const uint32_t inc = wave_incl_scan(c);
                uint32_t pos = n + inc - c;
                if (c)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        if (v[i] >= low && first + i < V) {
                            if (pos < TW_CAP) {
                                ckey[pos] = order_key(v[i]);
                                cidx[pos] = (uint16_t)(first + i);
                            }
                            ++pos;
                        }
                    }
                n += lane_value(inc, SG_WAVE - 1);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const auto put = [&](uint32_t place, uint32_t key, uint32_t index) {
        p.idx[row * k + place] = index;
        p.logp[row * k + place] = top_logp(key_value(key), m, log_s, p.r.it);
    };
    if (n <= TW_CAP) {
        wave_sync();
        // a lane holds candidates l, l + 64, ...: two or four in nearly all rows
        uint32_t key[TW_CAP / SG_WAVE];
        const uint32_t rounds = (n + SG_WAVE - 1) / SG_WAVE;
#pragma unroll
        for (uint32_t q = 0; q < TW_CAP / SG_WAVE; ++q) key[q] = l + q * SG_WAVE < n ? ckey[l + q * SG_WAVE] : 0u;
        const auto kth_of = [&](auto regs) {
            constexpr int Q = decltype(regs)::value;
            return wave_kth(k, low_shift, [&](uint32_t c) {
                uint32_t h = 0;
#pragma unroll
                for (int q = 0; q < Q; ++q) h += popc64(ballot(key[q] >= c));
                return h;
            });
        };
        const uint32_t kth = whole_key(rounds <= 2   ? kth_of(std::integral_constant<int, 2>())
                                       : rounds <= 4 ? kth_of(std::integral_constant<int, 4>())
                                                     : kth_of(std::integral_constant<int, TW_CAP / SG_WAVE>()),
                                       low_shift);
        uint32_t gt = 0;
#pragma unroll
        for (uint32_t q = 0; q < TW_CAP / SG_WAVE; ++q) gt += popc64(ballot(key[q] > kth));
        wave_emit(n, kth, k - gt, [&](uint32_t i, uint32_t* ky, uint32_t* index) {
            *ky = ckey[i];
            *index = cidx[i];
        }, put);
    } else { // the whole row, from the cache: a row of many equals
        const uint32_t kth = whole_key(wave_kth(k, low_shift, [&](uint32_t c) {
                                           uint32_t h = 0;
                                           for (uint32_t i = l; i < V; i += SG_WAVE)
                                               h += order_key(RowIO<E>::get(x + i)) >= c ? 1u : 0u;
                                           return wave_sum(h);
                                       }),
                                       low_shift);
        uint32_t gt = 0;
        for (uint32_t i = l; i < V; i += SG_WAVE) gt += order_key(RowIO<E>::get(x + i)) > kth ? 1u : 0u;
        const uint32_t ties = k - wave_sum(gt);
        wave_emit(V, kth, ties, [&](uint32_t i, uint32_t* key, uint32_t* index) {
            *key = order_key(RowIO<E>::get(x + i));
            *index = i;
        }, put);
    }
}

// ---------------------------------------------------------------------------
// longer rows: a block per row or part
// ---------------------------------------------------------------------------
template <int NT>
struct TopShared {
    static constexpr int NW = NT / SG_WAVE;
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
// its equals belong to the k.
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
    return whole_key(prefix, low_shift);
}

// Passes on, in index order, the elements whose key is above `kth` and the
// first `ties` of its equals: put(place, key, index).  at(i, &key, &index)
// yields element i < n, ascending in index.
template <int NT, class S, class At, class Put>
__device__ __forceinline__ void emit_rows(S& sh, uint32_t n, uint32_t kth, uint32_t ties, At at, Put put)
{
    uint32_t above = 0, equal = 0;
    for (uint32_t base = 0; base < n; base += NT) {
        const uint32_t i = base + threadIdx.x;
        uint32_t key = 0, index = 0, total;
        if (i < n) at(i, &key, &index);
        const bool gt = i < n && key > kth, eq = i < n && key == kth;
        __syncthreads(); // the scan's words are read to the end of it
        const uint32_t pos = block_excl_scan<NT>((gt ? 1u : 0u) | (eq ? 65536u : 0u), sh.scan, &total);
        const uint32_t ng = above + (pos & 0xffffu), ne = equal + (pos >> 16);
        if (gt || (eq && ne < ties)) put(ng + (ne < ties ? ne : ties), key, index);
        above += total & 0xffffu;
        equal += total >> 16;
    }
}

// The k of n candidates (ascending in index) in LDS.  For up to 64 of them a
// lane of one wave counts what its own is below, four keys a read; for more
// the radix rounds of three barriers for every 8 bits are shorter.  8000 x
// 8000 bf16 with counting up to 512, 128 and 64: top 128 83, 57 and 58 us,
// top 64 65, 66 and 55 us.
template <int NT, class S, class Put>
__device__ __forceinline__ void select_candidates(S& sh, const uint32_t* ckey, const uint32_t* cidx, uint32_t n,
                                                  uint32_t k, int low_shift, Put put)
{
    if (n <= SG_WAVE) {
        const uint32_t i = threadIdx.x, key = i < n ? ckey[i] : 0u;
        uint32_t rank = 0;
        if (uniform(i) < n) // waves without a candidate have nothing to count
            for (uint32_t j = 0; j < n; j += 4) { // the list is padded to a multiple of 4 with zeros
                const u32x4 o = *reinterpret_cast<const u32x4*>(ckey + j);
#pragma unroll
                for (int q = 0; q < 4; ++q) rank += o[q] > key || (o[q] == key && j + q < i) ? 1u : 0u;
            }
        const bool sel = i < n && rank < k;
        uint32_t total;
        const uint32_t pos = block_excl_scan<NT>(sel ? 1u : 0u, sh.scan, &total);
        if (sel) put(pos, key, cidx[i]);
        return;
    }
    uint32_t ties;
    const uint32_t kth = radix_select<NT>(sh, n, k, low_shift, [&](uint32_t i) { return ckey[i]; }, &ties);
    emit_rows<NT>(sh, n, kth, ties,
                  [&](uint32_t i, uint32_t* key, uint32_t* index) {
                      *key = ckey[i];
                      *index = cidx[i];
                  },
                  put);
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
    return cut_value(t);
}

// room for candidates: four times k, at least 1024; 4096 take any row of so many elements as it is
__host__ __device__ constexpr uint32_t top_cap(uint32_t k) { return k <= 256 ? 1024 : 4096; }

// Dynamic LDS: candidates' keys and indices [cap], then the maximum of every
// line, whose place the list of candidate lines takes once it is made.
template <typename E, int NT, bool PART>
__global__ __launch_bounds__(NT, 8) void top_rows_kernel(TopArgs p)
{
    constexpr int VEC = RowIO<E>::VEC, NW = NT / SG_WAVE, J = 4;
    constexpr int low_shift = sizeof(E) == 2 ? 16 : 0;
    constexpr int RMAX = (int)(TR_MAX_LINES / NW + SG_WAVE - 1) / SG_WAVE;
    extern __shared__ u32x4 tr_lds[];
    __shared__ TopShared<NT> sh;
    const uint32_t t = threadIdx.x, cap = top_cap(p.k);
    uint32_t* ckey = reinterpret_cast<uint32_t*>(tr_lds);
    uint32_t* cidx = ckey + cap;
    float* lines = reinterpret_cast<float*>(cidx + cap);
    const uint64_t row = p.r.row0 + (PART ? blockIdx.y : blockIdx.x);
    const uint32_t lo = PART ? blockIdx.x * p.len : 0, V = PART && p.r.V - lo < p.len ? p.r.V - lo : (PART ? p.len : p.r.V);
    const uint32_t k = PART && V < p.k ? V : p.k;
    const E* x = static_cast<const E*>(p.r.x) + row * p.r.ld + lo;
    const RowSpan sp = span_of(x, V);
    const E* xc = x + sp.head;
    const uint32_t shift = p.shift, per_line = 1u << shift, nl = (sp.nc + per_line - 1) >> shift;
    // Not nl <= TR_MAX_LINES: an unaligned row has a chunk less than the room was
    // sized for and the last part is shorter, so nl can pass a limit that they did not.
    const bool lined = p.lined;

    RowStat st = {-INFINITY, 0.0};
    const auto take = [&](u32x4 w, uint32_t c) { // chunk c of a line: whole lines, so that their 8 lanes stay together
        float m = -INFINITY;
        if (c < sp.nc) {
            float v[VEC];
            RowIO<E>::unpack(w, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = fmaxf(m, v[i]);
            stat_add<VEC>(st, v, p.r.c);
        }
        if (shift) m = line_max(m);
        if (lined && (c & (per_line - 1)) == 0) lines[c >> shift] = m;
        __builtin_amdgcn_sched_barrier(0);
    };
    uint32_t j0 = 0;
    u32x4 w[J];
#pragma unroll 1
    for (; j0 + J * NT <= sp.nc; j0 += J * NT) { // the whole block has chunks
#pragma unroll
        for (int j = 0; j < J; ++j) w[j] = load_chunk(chunk_at<E>(xc, j0 + j * NT, t));
#pragma unroll
        for (int j = 0; j < J; ++j) take(w[j], t + j0 + j * NT);
    }
    if (j0 < sp.nc) {
        load_chunks<J, NT>(w, xc, t + j0, sp.nc);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (t + j0 + j * NT < nl << shift) take(w[j], t + j0 + j * NT);
    }
    if (t < 2 * VEC) {
        const uint32_t i = loose_element(sp, VEC, t);
        if (i < V) {
            const float v = RowIO<E>::get(x + i);
            stat_add<1>(st, &v, p.r.c);
        }
    }
    st = wave_stat(st, p.r.c);
    if (lane_id() == 0) sh.part[t / SG_WAVE] = st;
    __syncthreads();
    st = wave_stat<next_pow2(NW)>(sh.part[lane_id() % NW], p.r.c); // NW is a power of two
    if (t == 0) {
        if (PART) {
            p.part_stat[row * p.parts + blockIdx.x] = st;
        } else {
            sh.log_s = row_log(st.s);
            sh.max = shift_of(st.m);
            if (p.lse) p.lse[row] = (float)(sh.max * p.r.it + sh.log_s);
        }
    }
    uint32_t n = 0; // candidates; 0: none found this way
    if (lined && st.s == st.s) {
        const uint32_t wv = uniform(t / SG_WAVE);
        const uint32_t l0 = (uint32_t)((uint64_t)nl * wv / NW), l1 = (uint32_t)((uint64_t)nl * (wv + 1) / NW);
        const uint32_t want = (k + NW - 1) / NW;
        const float reach = l1 - l0 <= 2 * SG_WAVE   ? lines_reach<2>(lines, l0, l1, want)
                            : l1 - l0 <= 4 * SG_WAVE ? lines_reach<4>(lines, l0, l1, want)
                            : l1 - l0 <= 8 * SG_WAVE ? lines_reach<8>(lines, l0, l1, want)
                                                     : lines_reach<RMAX>(lines, l0, l1, want);
        if (lane_id() == 0) sh.low[wv] = reach;
        __syncthreads();
        float low = sh.low[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) low = fminf(low, sh.low[i]);
        if (low > -INFINITY || V <= cap) {
            // the lines that reach it, in order: a thread takes `per` neighbours
            const uint32_t per = (nl + NT - 1) / NT, b0 = t * per < nl ? t * per : nl, b1 = b0 + per < nl ? b0 + per : nl;
            uint32_t c = 0, nlc;
            for (uint32_t b = b0; b < b1; ++b) c += lines[b] >= low ? 1u : 0u;
            uint32_t pos = block_excl_scan<NT>(c, sh.scan, &nlc);
            // (the candidates' indices are not in use yet)
            if (nlc <= cap)
                for (uint32_t b = b0; b < b1; ++b)
                    if (lines[b] >= low) cidx[pos++] = b;
            __syncthreads();
            if (nlc <= cap) {
                // their elements that reach it, with those outside the chunks, in order: an item a
                // chunk, before them the elements ahead of the chunks and after them those behind; a
                // thread takes neighbours again.  The list of lines moves over the line maxima.
                uint32_t* list = reinterpret_cast<uint32_t*>(lines);
                for (uint32_t i = t; i < nlc; i += NT) list[i] = cidx[i];
                __syncthreads();
                const uint32_t items = (nlc << shift) + 2;
                constexpr int B = 4; // neighbours to a thread, loaded together; one if that is enough
                const uint32_t per_t = items <= NT ? 1 : B;
                for (uint32_t q0 = 0; q0 < items; q0 += per_t * NT) {
                    u32x4 it[B];
                    uint32_t first[B], e = 0, total;
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        const uint32_t q = (uint32_t)i < per_t ? q0 + t * per_t + i : items;
                        uint32_t len = 0;
                        first[i] = 0;
                        if (q == 0) {
                            len = sp.head;
                        } else if (q == items - 1) {
                            first[i] = sp.head + sp.nc * VEC;
                            len = V - first[i];
                        } else if (q < items) {
                            const uint32_t ch = (list[(q - 1) >> shift] << shift) + ((q - 1) & (per_line - 1));
                            first[i] = sp.head + ch * VEC;
                            if (ch < sp.nc) len = VEC;
                        }
                        if (len == VEC) {
                            it[i] = load_chunk(x + first[i]);
                        } else {
                            float v[VEC];
#pragma unroll
                            for (int c = 0; c < VEC; ++c) // a NaN is no candidate
                                v[c] = c < (int)len ? RowIO<E>::get(x + first[i] + c) : __builtin_nanf("");
                            it[i] = RowIO<E>::pack(v);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < B; ++i) {
                        float v[VEC];
                        RowIO<E>::unpack(it[i], v);
#pragma unroll
                        for (int c = 0; c < VEC; ++c) e += v[c] >= low ? 1u : 0u;
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    uint32_t to = n + block_excl_scan<NT>(e, sh.scan, &total);
                    if (e)
#pragma unroll
                        for (int i = 0; i < B; ++i) {
                            float v[VEC];
                            RowIO<E>::unpack(it[i], v);
#pragma unroll
                            for (int c = 0; c < VEC; ++c)
                                if (v[c] >= low) {
                                    if (to < cap) {
                                        ckey[to] = order_key(v[c]);
                                        cidx[to] = first[i] + c;
                                    }
                                    ++to;
                                }
                        }
                    n += total;
                    __syncthreads(); // the scan's words
                }
                if (t < 4 && n + t < cap) ckey[n + t] = 0;
                if (n > cap) n = 0;
            }
        }
    }
    __syncthreads();
    const auto put = [&](uint32_t place, uint32_t key, uint32_t index) {
        if (PART) {
            const uint64_t to = (row * p.parts + blockIdx.x) * p.k + place;
            p.part_key[to] = key;
            p.part_idx[to] = lo + index;
        } else {
            const uint64_t to = row * p.k + place;
            p.idx[to] = index;
            p.logp[to] = top_logp(key_value(key), sh.max, sh.log_s, p.r.it);
        }
    };
    if (n > 0) {
        select_candidates<NT>(sh, ckey, cidx, n, k, low_shift, put);
    } else {
        uint32_t ties;
        const uint32_t kth = radix_select<NT>(sh, V, k, 0, [&](uint32_t i) { return order_key(RowIO<E>::get(x + i)); },
                                              &ties);
        emit_rows<NT>(sh, V, kth, ties,
                      [&](uint32_t i, uint32_t* key, uint32_t* index) {
                          *key = order_key(RowIO<E>::get(x + i));
                          *index = i;
                      },
                      put);
    }
}

// the candidates of a row's parts joined: the parts are in index order, and so is each
constexpr int TJ_NT = 512;
constexpr uint32_t TJ_CAP = 4096;

template <typename E>
__global__ __launch_bounds__(TJ_NT, 4) void top_join_kernel(TopArgs p)
{
    __shared__ TopShared<TJ_NT> sh;
    __shared__ __attribute__((aligned(16))) uint32_t ckey[TJ_CAP], cidx[TJ_CAP];
    const uint32_t t = threadIdx.x, last = p.r.V - (p.parts - 1) * p.len;
    const uint64_t row = p.r.row0 + blockIdx.x;
    const uint32_t n = (p.parts - 1) * p.k + (last < p.k ? last : p.k); // every other part has k
    for (uint32_t i = t; i < n; i += TJ_NT) {
        ckey[i] = p.part_key[row * p.parts * p.k + i];
        cidx[i] = p.part_idx[row * p.parts * p.k + i];
    }
    if (t < 4 && n + t < TJ_CAP) ckey[n + t] = 0;
    if (t < SG_WAVE) {
        const RowStat st = wave_stat(t < p.parts ? p.part_stat[row * p.parts + t] : RowStat{-INFINITY, 0.0}, p.r.c);
        if (t == 0) {
            sh.log_s = row_log(st.s);
            sh.max = shift_of(st.m);
            if (p.lse) p.lse[row] = (float)(sh.max * p.r.it + sh.log_s);
        }
    }
    __syncthreads();
    select_candidates<TJ_NT>(sh, ckey, cidx, n, p.k, sizeof(E) == 2 ? 16 : 0,
                             [&](uint32_t place, uint32_t key, uint32_t index) {
                                 const uint64_t to = row * p.k + place;
                                 p.idx[to] = index;
                                 p.logp[to] = top_logp(key_value(key), sh.max, sh.log_s, p.r.it);
                             });
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Parts of a row: as for the losses, few rows longer than 128 KiB, in parts of
// at least 32 KiB whose candidates one block can join.
static uint32_t top_parts(uint64_t T, uint64_t V, uint32_t k, uint64_t esize)
{
    uint64_t parts = row_parts(T, V, esize);
    if (parts > TJ_CAP / k) parts = TJ_CAP / k;
    return parts < 2 || ceil_div(V, parts) < k ? 1 : (uint32_t)parts;
}

struct TopWs {
    uint32_t *key, *idx;
    RowStat* stat;
};
static TopWs top_carve(Carver& cv, uint64_t T, uint32_t parts, uint32_t k)
{
    TopWs w = {};
    if (parts > 1) {
        w.key = cv.take<uint32_t>(T * parts * k);
        w.idx = cv.take<uint32_t>(T * parts * k);
        w.stat = cv.take<RowStat>(T * parts);
    }
    return w;
}

// A row with fewer than three lines to each of its k gives a threshold far
// below the k-th largest, or none: its groups are single chunks, as long as
// their maxima fit (top 128 of 8000 x 8000 bf16, 125 lines: 307 us with
// lines of 8, 84 us so).
template <typename E>
static uint32_t top_shift(uint64_t V, uint32_t k)
{
    const uint64_t chunks = V / RowIO<E>::VEC;
    return chunks / TR_LINE < 3ull * k && chunks <= TR_MAX_LINES ? 0 : 3;
}

// Lines and LDS of blocks that take up to V elements each.
template <typename E>
static size_t top_lines(TopArgs* p, uint64_t V)
{
    p->shift = top_shift<E>(V, p->k);
    const uint64_t lines = ceil_div(V / RowIO<E>::VEC, 1u << p->shift), cap = top_cap(p->k);
    p->lined = lines <= TR_MAX_LINES;
    // the lines' maxima, or the list of up to cap candidate lines in their place
    return cap * 8 + (p->lined && lines > cap ? lines : cap) * 4;
}

template <typename E, int NT>
static int launch_top(TopArgs p, hipStream_t st)
{
    const size_t lds = top_lines<E>(&p, p.r.V);
    for (p.r.row0 = 0; p.r.row0 < p.r.T; p.r.row0 += ROWS_PER_LAUNCH) {
        const uint64_t left = p.r.T - p.r.row0;
        top_rows_kernel<E, NT, false><<<(unsigned)(left < ROWS_PER_LAUNCH ? left : ROWS_PER_LAUNCH), NT, lds, st>>>(p);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}

template <typename E>
static int launch_top_of(TopArgs p, void* ws, hipStream_t st)
{
    const uint64_t bytes = (uint64_t)p.r.V * sizeof(E);
    p.parts = top_parts(p.r.T, p.r.V, p.k, sizeof(E));
    if (p.parts > 1) { // fewer than 128 rows
        Carver cv(ws);
        const TopWs w = top_carve(cv, p.r.T, p.parts, p.k);
        p.part_key = w.key;
        p.part_idx = w.idx;
        p.part_stat = w.stat;
        p.len = part_len(p.r.V, &p.parts);
        const size_t lds = top_lines<E>(&p, p.len);
        top_rows_kernel<E, 512, true><<<dim3(p.parts, (unsigned)p.r.T), 512, lds, st>>>(p);
        SG_TRY_LAUNCH();
        top_join_kernel<E><<<(unsigned)p.r.T, TJ_NT, 0, st>>>(p);
        SG_TRY_LAUNCH();
        return SG_OK;
    }
    if (bytes <= (uint64_t)SG_WAVE * TW_R * 16 && (p.k <= TW_MAX_K || p.r.V <= TW_CAP)) {
        for (p.r.row0 = 0; p.r.row0 < p.r.T; p.r.row0 += ROWS_PER_LAUNCH) {
            const uint64_t left = p.r.T - p.r.row0;
            top_wave_kernel<E><<<(unsigned)(left < ROWS_PER_LAUNCH ? left : ROWS_PER_LAUNCH), SG_WAVE, 0, st>>>(p);
            SG_TRY_LAUNCH();
        }
        return SG_OK;
    }
    // Four blocks of 512 on a compute unit hide each other's selection better
    // than two of 1024 (8192 x 131072 bf16: 513 us against 566 for k = 128),
    // until the lists are so long that the threads of one block count (950
    // against 705 us for k = 500); with few rows there is one block on a
    // compute unit anyway (200 x 262144 fp32: 58 against 49 us).
    // Rows of up to 32 KB: 256 threads, twice the blocks of 512 on a compute unit, so that one
    // selects while another reads (512 -> 256: top 20 of 8000 x 8000 bf16 92 -> 54 us, top 64 of
    // 8000 x 16000 133 -> 90 us).  Longer lists keep 512 for their selection (top 300 of 8000 x
    // 16000: 138 us with 512, 169 with 256).
    if (bytes <= 32 * 1024 && p.k <= 256) return launch_top<E, 256>(p, st);
    if (bytes <= 128 * 1024 || (p.k <= 256 && p.r.T >= 512)) return launch_top<E, 512>(p, st);
    return launch_top<E, 1024>(p, st);
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_topk_rows_workspace_bytes(uint64_t T, uint64_t V, uint32_t k, sg_dtype dt)
{
    if (T >= (1ull << 31) || V == 0 || V >= (1ull << 31) || k == 0 || k > SG_ROWS_MAX_K) return 0;
    if (dt != SG_F32 && dt != SG_BF16) return 0;
    const uint32_t parts = top_parts(T, V, k, row_esize(dt));
    Carver cv(nullptr);
    top_carve(cv, T, parts, k);
    return parts > 1 ? cv.bytes() : 0;
}

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
    const size_t need = sg_topk_rows_workspace_bytes(T, V, k, dt);
    if (need > 0 && !d_ws) return SG_EINVAL;
    if (ws_bytes < need) return SG_ECAPACITY;
    TopArgs p = {};
    p.r = c.r;
    p.k = k;
    p.idx = d_idx;
    p.logp = d_logp;
    p.lse = d_lse;
    if (dt == SG_BF16) return launch_top_of<bf16_bits>(p, d_ws, as_stream(stream));
    return launch_top_of<float>(p, d_ws, as_stream(stream));
}
