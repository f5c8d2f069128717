// sg_rowloss.hip -- losses over rows of logits with their gradients:
// distillation from a teacher's top logits, the clipped policy loss, and the
// paired preference loss.
//
// Mathematics.  z = x / temperature, lse = log sum exp z, log q_i = z_i - lse.
// Each loss is a function of lse and of the few logits it names (the token
// taken, the listed tokens), so one pass over the row with a running maximum
// and sum gives the loss, and its gradient has the dense part coef * q_i plus
// corrections at the named tokens.  Row scalars are in fp64: a loss is often
// the small difference of numbers near lse.
//
// Bound: HBM.  The row is read once for the sums; the gradient is written
// once.
#include "sg_host.h"
#include "sg_rows.h"

namespace sg {

constexpr uint32_t RL_MAX_K = SG_ROWS_MAX_K;
constexpr uint32_t RL_MAX_PARTS = 64;

// A row's gradient: coef * exp2(c * (x_i - m)) for the tokens it does not
// name; a, b and named_m are what the operator needs for those it names.
struct RowCoef {
    float m, coef, a, b, named_m;
};

// Where the gradient goes.  past: its stores go past the caches.
struct GradOut {
    void* g;
    uint64_t ld;
    bool past;
};

// What an operator with a list keeps of it, in dynamic LDS of the list's size:
// room for the longest list (20 KiB) left 7 blocks of short rows on a compute
// unit, where the registers allow 12.
struct RowList {
    float *z, *p;         // [k] logits, masses
    uint32_t *id, *chunk; // [k] tokens; the chunks that the list's wave adds
    uint32_t* flag;       // [threads] bit r: the chunk that data thread t takes in round r has listed tokens
    uint32_t* bitmap;     // of the row or part
};
struct NoList {
    uint32_t* bitmap;
};

// An element's bit of the bitmap is its place plus this, so that the bits of
// a chunk start at a multiple of the chunk's size.
template <typename E>
__device__ __forceinline__ uint32_t mark_pad(const RowSpan& sp)
{
    return (uint32_t)(-sp.head) % RowIO<E>::VEC;
}

// n (4, 8 or 1) bits of the bitmap from bit i0, a multiple of n
__device__ __forceinline__ uint32_t marked(const uint32_t* bm, uint32_t i0, int n)
{
    return bm[i0 / 32] >> (i0 % 32) & ((1u << n) - 1u);
}

// An operator says which rows it reads (live, skip), what it needs of the
// named logits (Named, gathered before a gradient may overwrite them), how
// the row's sum becomes loss and gradient (finish, by a wave), and the
// gradient of the named tokens in [lo, hi) of the row (named_grad, put_named;
// g is element lo).  kListed: tokens are listed, and left out of the
// streaming pass's sum; a wave of its own handles the list.

// log-probability of the logit za; a NaN in the row stays (its sum is NaN then, and
// S - S: a comparison more put registers of the widest kernels out to memory)
__device__ __forceinline__ double token_logp(const Rows& r, RowStat st, float za)
{
    return za == -INFINITY ? (st.s - st.s) - (double)INFINITY : ((double)za - st.m) * r.it - row_log(st.s);
}

// ---------------------------------------------------------------------------
// the clipped policy loss
// ---------------------------------------------------------------------------
struct PolicyOp {
    const int32_t* action;
    const float *old_logp, *ref_logp, *adv, *weight;
    float *loss, *logp;
    double lo, hi, kl;
    uint32_t V;

    static constexpr bool kListed = false, kGrad = true, kFine = false;
    typedef float Named; // the action's logit
    typedef NoList List;
    __device__ __forceinline__ NoList list(uint32_t*, uint32_t) const { return {nullptr}; }

    __device__ __forceinline__ bool live(uint64_t row) const
    {
        return (uint32_t)action[row] < V && (!weight || weight[row] != 0.f);
    }
    __device__ __forceinline__ void skip(uint64_t row) const
    {
        loss[row] = 0.f;
        if (logp) logp[row] = 0.f;
    }
    template <typename E>
    __device__ __forceinline__ Named named(const Rows&, uint64_t row, const E* x, NoList&) const
    {
        return RowIO<E>::get(x + action[row]);
    }
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, Named za, bool write) const
    {
        const double S = st.s;
        const double lp = token_logp(r, st, za);
        const double w = weight ? (double)weight[row] : 1.0;
        const double A = adv ? (double)adv[row] : 0.0;
        const double ratio = old_logp ? row_exp(lp - (double)old_logp[row]) : (S - S) + 1.0; // 1, or NaN
        const double bounded = ratio < lo ? lo : (ratio > hi ? hi : ratio);
        const double a = ratio * A, b = bounded * A;
        double L = a <= b ? -a : (b <= a ? -b : a + b); // a NaN stays
        // where the bounded product is the smaller one the loss does not move
        const bool clipped = (A > 0.0 && ratio > hi) || (A < 0.0 && ratio < lo);
        double slope = clipped ? 0.0 : -a;
        if (ref_logp) {
            const double d = (double)ref_logp[row] - lp, e = row_expm1(d);
            L += kl * (d == INFINITY ? d : e - d); // a token that the policy cannot take: +inf, not inf - inf
            slope -= kl * e;
        }
        if (write && lane_id() == 0) {
            loss[row] = (float)(w * L);
            if (logp) logp[row] = (float)lp;
        }
        const double g = w * slope * r.it;
        // at the action 1 - q without the cancellation
        return {st.m, (float)(-g * inverse_of(S)), (float)(g * -row_expm1(lp)), 0.f, 0.f};
    }
    __device__ __forceinline__ void named_grad(const Rows&, const RowCoef&, NoList&) const {}
    template <typename E>
    __device__ __forceinline__ void put_named(uint64_t row, E* g, const RowCoef& k, const NoList&, uint32_t lo_,
                                              uint32_t hi_) const
    {
        const uint32_t i = (uint32_t)action[row];
        if (lane_id() == 0 && i >= lo_ && i < hi_) RowIO<E>::put(g + (i - lo_), k.a);
    }
};

// ---------------------------------------------------------------------------
// the log-probability of one token per row (first pass of the preference
// loss); the row's maximum and 1/sum are kept for the gradient pass
// ---------------------------------------------------------------------------
struct TokenOp {
    const int32_t* label;
    double* logp;
    float *m, *inv;
    float* slope; // cleared here, set by the pair pass for rows of a sequence
    uint32_t V;

    static constexpr bool kListed = false, kGrad = false, kFine = true;
    typedef float Named;
    typedef NoList List;
    __device__ __forceinline__ NoList list(uint32_t*, uint32_t) const { return {nullptr}; }

    __device__ __forceinline__ bool live(uint64_t row) const { return (uint32_t)label[row] < V; }
    __device__ __forceinline__ void skip(uint64_t row) const
    {
        logp[row] = 0.0;
        slope[row] = 0.f;
    }
    template <typename E>
    __device__ __forceinline__ Named named(const Rows&, uint64_t row, const E* x, NoList&) const
    {
        return RowIO<E>::get(x + label[row]);
    }
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, Named za, bool write) const
    {
        if (write && lane_id() == 0) {
            logp[row] = token_logp(r, st, za);
            m[row] = st.m;
            inv[row] = (float)inverse_of(st.s);
            slope[row] = 0.f;
        }
        return {};
    }
};

// ---------------------------------------------------------------------------
// distillation from listed logits
// ---------------------------------------------------------------------------
// The student's sum is kept in two parts, over the listed tokens and over the
// others: the remainder's mass 1 - Q would otherwise be a difference of
// nearly equal numbers wherever the student agrees with the teacher.  A bitmap
// of the row in LDS tells the streaming pass which elements are listed.
struct DistillOp {
    const uint32_t* idx; // [T][k]
    const float* logp;   // [T][k]
    const float* weight;
    float* loss;
    uint32_t k, V;
    int mode;

    static constexpr bool kListed = true, kGrad = true, kFine = false;
    typedef RowList List;

    static __host__ __device__ constexpr uint32_t list_words(uint32_t k, uint32_t threads) { return 4 * k + threads; }
    __device__ __forceinline__ RowList list(uint32_t* lds, uint32_t threads) const
    {
        RowList ls;
        ls.z = reinterpret_cast<float*>(lds);
        ls.p = ls.z + k;
        ls.id = lds + 2 * k;
        ls.chunk = lds + 3 * k;
        ls.flag = lds + 4 * k;
        ls.bitmap = ls.flag + threads;
        return ls;
    }
    struct Named {
        double P, A, S; // mass, sum p (log p - (z - m)), sum exp(z - m), z scaled by inv_temp
        float m;        // maximum of the listed logits
        // RENORM: the maximum of the listed log-probabilities, otherwise 0.  p / P
        // is the same for p = exp(logp - top), and masses far below 1 keep 1 / P in
        // fp32's range.
        float top;
    };

    __device__ __forceinline__ bool live(uint64_t row) const { return !weight || weight[row] != 0.f; }
    __device__ __forceinline__ void skip(uint64_t row) const { loss[row] = 0.f; }
    // The list's wave, in four steps.  fetch: its first 64 tokens, asked for
    // before anything else, since the row's loads would hold them up.
    __device__ __forceinline__ uint32_t fetch(uint64_t row) const
    {
        return lane_id() < k ? idx[row * k + lane_id()] : V;
    }
    // mark: the tokens of [lo, hi) in the bitmap, and their chunks in the flags
    template <typename E, int ND>
    __device__ __forceinline__ void mark(uint64_t row, uint32_t i, uint32_t lo, uint32_t hi, const RowSpan& sp,
                                         RowList& ls, uint32_t* bm) const
    {
        constexpr uint32_t VEC = RowIO<E>::VEC;
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE) {
            if (j >= SG_WAVE) i = idx[row * k + j];
            ls.id[j] = i;
            ls.chunk[j] = ~0u;
            if (i < lo || i >= hi) continue;
            const uint32_t e = i - lo, at = e + mark_pad<E>(sp), was = atomicOr(&bm[at / 32], 1u << (at % 32));
            if (was >> (at % 32) & 1u) report_error(kDevErrUnsorted); // listed twice
            const uint32_t c = e >= sp.head ? (e - sp.head) / VEC : sp.nc, round = c / ND;
            if (c >= sp.nc) continue; // outside the chunks
            if (round < 32) atomicOr(&ls.flag[c % ND], 1u << round);
            // the first token of a chunk has it
            if ((was >> (at / VEC * VEC % 32) & ((1u << VEC) - 1u)) == 0) ls.chunk[j] = c;
        }
    }
    // the other tokens of the marked chunks
    template <typename E>
    __device__ __forceinline__ RowStat marked_chunks(const E* xc, const RowSpan& sp, const RowList& ls,
                                                     const uint32_t* bm, Scale c) const
    {
        constexpr uint32_t VEC = RowIO<E>::VEC;
        RowStat st = {-INFINITY, 0.0};
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE) {
            const uint32_t ch = ls.chunk[j];
            if (ch == ~0u) continue;
            float v[VEC];
            const uint32_t b = marked(bm, sp.head + mark_pad<E>(sp) + ch * VEC, VEC);
            RowIO<E>::unpack(RowIO<E>::without(load_chunk(chunk_at<E>(xc, ch, 0)), b), v);
            stat_add<VEC>(st, v, c);
        }
        return st;
    }
    // named: the listed logits and masses, and their sums
    template <typename E>
    __device__ __forceinline__ Named named(const Rows& r, uint64_t row, const E* x, RowList& ls) const
    {
        const float* lp = logp + row * k;
        float m = -INFINITY, top = -INFINITY;
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE) {
            const uint32_t i = ls.id[j];
            const float v = i < V ? RowIO<E>::get(x + i) : -INFINITY;
            ls.z[j] = v;
            m = fmaxf(m, v);
            const float t = lp[j]; // beside the logit's load, not after it
            ls.p[j] = t;
            if (i < V) top = fmaxf(top, t);
        }
        if (mode == SG_DISTILL_RENORM) {
#pragma unroll
            for (int d = 1; d < SG_WAVE; d <<= 1) { // both at once: the lanes' exchange is latency
                m = fmaxf(m, __shfl_xor(m, d, SG_WAVE));
                top = fmaxf(top, __shfl_xor(top, d, SG_WAVE));
            }
        } else {
            top = 0.f;
#pragma unroll
            for (int d = 1; d < SG_WAVE; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, SG_WAVE));
        }
        top = shift_of(top);
        const double shift = shift_of(m);
        double P = 0.0, A = 0.0, S = 0.0;
#pragma unroll 1
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE) {
            double p = 0.0;
            if (ls.id[j] < V) {
                const double t = (double)ls.p[j] - top, d = (ls.z[j] - shift) * r.it;
                p = row_exp(t);
                P += p;
                if (p != 0.0) A += p * (t - d);
                S += row_exp(d);
            }
            ls.p[j] = (float)p;
        }
        return {wave_sum_f64(P), wave_sum_f64(A), wave_sum_f64(S), m, top};
    }
    // finish: by the whole wave, so that the functions of several numbers run
    // side by side in its lanes
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, const Named& nm, bool write) const
    {
        const uint32_t l = lane_id();
        const float m = fmaxf(st.m, nm.m);
        const double shift = shift_of(m);
        const double scale = row_exp(((l ? (double)nm.m : (double)st.m) - shift) * r.it);
        const double rest = st.s * __shfl(scale, 0), own = nm.S * __shfl(scale, 1);
        const double S = rest + own;
        const double R0 = nm.P < 1.0 ? 1.0 - nm.P : 0.0, per_rest = 1.0 / rest, per_S = inverse_of(S);
        const double lg = row_log(l == 0 ? S : (l == 1 ? R0 * S * per_rest : nm.P));
        // lse less the listed maximum (a row may lie at the type's lowest
        // value, where lse itself holds no digit of log S); of a row of
        // nothing but -inf, A decides: S is 0, or NaN if the row has one
        const double lse = m == -INFINITY ? S : (shift - shift_of(nm.m)) * r.it + __shfl(lg, 0);
        const double log_tail = __shfl(lg, 1), log_mass = __shfl(lg, 2);
        const double w = weight ? (double)weight[row] : 1.0;
        double P = nm.P, R = 0.0, gp = 1.0, L;
        if (mode == SG_DISTILL_RENORM) {
            gp = P > 0.0 ? 1.0 / P : P; // nothing listed: no mass, no loss (a NaN stays, the row's too)
            L = P > 0.0 ? nm.A * gp - log_mass + lse : P * lse;
            P = P > 0.0 ? 1.0 : P;
        } else {
            L = nm.A + P * lse;
            // what is left for the unlisted tokens, where there are any
            if (mode == SG_DISTILL_TAIL && R0 > 0.0 && rest > 1e-300) {
                R = R0;
                L += R * log_tail;
            }
        }
        if (write && l == 0) loss[row] = (float)(w * L);
        const double g = w * r.it;
        const double below = __shfl(scale, 0), all = (P + R) * per_S, near = all * below;
        // The unlisted tokens' exponentials are taken from their own maximum.
        // From the row's they would be 0 in fp32 88 below it, and R / rest
        // beyond fp32's range, where together they are up to R.
        return {st.m, (float)(g * (R != 0.0 ? near - R * per_rest * below : near)), (float)(g * all), (float)(g * gp), m};
    }
    // ls.z[j] becomes the gradient of listed token j
    __device__ __forceinline__ void named_grad(const Rows& r, const RowCoef& co, RowList& ls) const
    {
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE)
            ls.z[j] = co.a * exp2_scaled<false>(ls.z[j] - shift_of(co.named_m), r.c) - co.b * ls.p[j];
    }
    template <typename E>
    __device__ __forceinline__ void put_named(uint64_t, E* g, const RowCoef&, const RowList& ls, uint32_t lo,
                                              uint32_t hi) const
    {
        for (uint32_t j = lane_id(); j < k; j += SG_WAVE) {
            const uint32_t i = ls.id[j];
            if (i >= lo && i < hi) RowIO<E>::put(g + (i - lo), ls.z[j]);
        }
    }
};

// ---------------------------------------------------------------------------
// the passes over (a part of) a row
// ---------------------------------------------------------------------------
template <bool PAST, typename E>
__device__ __forceinline__ void zero_row(E* g, uint32_t V, uint32_t t, uint32_t nt)
{
    constexpr int VEC = RowIO<E>::VEC;
    const RowSpan sp = span_of<128>(g, V);
    const u32x4 z = {0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t j = t; j < sp.nc; j += nt) store_chunk<PAST>(chunk_at<E>(g + sp.head, j, 0), z);
    for (uint32_t i = loose_element(sp, VEC, t); i < V; i = loose_element(sp, VEC, t += nt)) RowIO<E>::put(g + i, 0.f);
}

template <bool PAST, typename E>
__device__ __forceinline__ void grad_chunk(u32x4 w, E* g, float coef, float sh, Scale c)
{
    constexpr int VEC = RowIO<E>::VEC;
    float v[VEC];
    RowIO<E>::unpack(w, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = coef * exp2_scaled<false>(v[i] - sh, c);
    store_chunk<PAST>(g, RowIO<E>::pack(v));
}

// the elements outside the chunks
template <typename E>
__device__ __forceinline__ void grad_loose(const E* x, E* g, const RowSpan& sp, float coef, float sh, Scale c,
                                           uint32_t t, uint32_t nt)
{
    constexpr int VEC = RowIO<E>::VEC;
#pragma unroll 1
    for (uint32_t i = loose_element(sp, VEC, t); i < sp.V; i = loose_element(sp, VEC, t += nt))
        RowIO<E>::put(g + i, coef * exp2_scaled<false>(RowIO<E>::get(x + i) - sh, c));
}

// gradient of V elements: coef * exp2(c (x - m)).  x and g may be the same
// memory: every thread reads an element before it writes it, and nobody else
// touches it.
template <bool PAST, typename E>
__device__ __forceinline__ void grad_row(const E* x, E* g, uint32_t V, float coef, float m, Scale c, uint32_t t,
                                         uint32_t nt)
{
    const RowSpan sp = span_of<128>(g, V);
    const float sh = shift_of(m);
#pragma unroll 2
    for (uint32_t j = t; j < sp.nc; j += nt)
        grad_chunk<PAST, E>(load_chunk(chunk_at<E>(x + sp.head, j, 0)), chunk_at<E>(g + sp.head, j, 0), coef, sh, c);
    grad_loose(x, g, sp, coef, sh, c, t, nt);
}

// Chunks j0, j0 + ND, ... whose loads are in w.  LISTED: chunks with listed
// tokens are left out (the list's wave takes them); bit j of `flags` says
// whether chunk j0 + j * ND is one.
template <typename E, int J, int ND, class Op>
__device__ __forceinline__ void stat_chunks(RowStat& st, const u32x4* w, uint32_t flags, uint32_t j0, uint32_t nc,
                                            Scale c)
{
    constexpr int VEC = RowIO<E>::VEC;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (j0 + j * ND < nc && !(Op::kListed && (flags >> j & 1u))) {
            float v[VEC];
            RowIO<E>::unpack(w[j], v);
            stat_add<VEC, Op::kFine>(st, v, c);
        }
        __builtin_amdgcn_sched_barrier(0); // a chunk at a time: unpacked, a chunk takes twice its registers
    }
}

// The chunks from round `first` on (thread t takes chunk t + round * ND), M
// loads in flight.  Rounds beyond the 32 that the flags hold look the chunk up
// in the bitmap, b0 the bit of chunk 0.
template <typename E, int M, int ND, class Op>
__device__ __forceinline__ void stat_more(RowStat& st, const E* xc, uint32_t flags, const uint32_t* bm, uint32_t b0,
                                          uint32_t t, uint32_t first, uint32_t nc, Scale c)
{
    constexpr int VEC = RowIO<E>::VEC;
    uint32_t round = first;
    u32x4 more[M];
#pragma unroll 1
    for (; (round + M) * ND <= nc && (!Op::kListed || round + M <= 32); round += M) { // the whole block has chunks in these rounds
#pragma unroll
        for (int j = 0; j < M; ++j) more[j] = load_chunk(chunk_at<E>(xc, (round + j) * ND, t));
        stat_chunks<E, M, ND, Op>(st, more, flags >> round, t + round * ND, nc, c);
    }
#pragma unroll 1
    for (; t + round * ND < nc; ++round) {
        more[0] = load_chunk(chunk_at<E>(xc, round * ND, t));
        uint32_t f = 0;
        if (Op::kListed) f = round < 32 ? flags >> round : (marked(bm, b0 + (t + round * ND) * VEC, VEC) ? 1u : 0u);
        stat_chunks<E, 1, ND, Op>(st, more, f, t + round * ND, nc, c);
    }
}

template <typename E, int ND, class Op>
__device__ __forceinline__ void stat_loose(RowStat& st, const E* x, const RowSpan& sp, const uint32_t* bm, uint32_t t,
                                           Scale c)
{
    constexpr int VEC = RowIO<E>::VEC;
#pragma unroll 1
    for (uint32_t i = loose_element(sp, VEC, t); i < sp.V; i = loose_element(sp, VEC, t += ND)) {
        float v = RowIO<E>::get(x + i);
        if (Op::kListed && marked(bm, i + mark_pad<E>(sp), 1)) v = -INFINITY;
        stat_add<1, Op::kFine>(st, &v, c);
    }
}

// ---------------------------------------------------------------------------
// one block per row
// ---------------------------------------------------------------------------
// No loop over rows: the constants of the fp64 functions would be hoisted out
// of it into registers that the row needs.  With GRAD the first ND * J chunks
// of the row stay in registers from the sums to the gradient, so the row is
// read from HBM once; what is beyond them is read again (from the last-level
// cache, the blocks in flight hold few rows).  Without GRAD nothing is kept
// and J is the number of loads a thread has in flight.
//
// A listed operator's last wave handles the list and no chunks: its gathers
// and fp64 functions run beside the streaming pass of the others.
template <typename E, int NT, int J, class Op, bool GRAD, bool PAST, int WAVES>
__global__ __launch_bounds__(NT, WAVES) void row_loss_kernel(Rows r, Op op, GradOut out)
{
    constexpr bool LISTED = Op::kListed;
    constexpr int ND = LISTED ? NT - SG_WAVE : NT, NW = ND / SG_WAVE; // data threads
    constexpr int VEC = RowIO<E>::VEC;
    extern __shared__ uint32_t rl_lds[];
    typename Op::List ls = op.list(rl_lds, ND);
    uint32_t* const rl_bitmap = ls.bitmap;
    __shared__ RowStat part[NT / SG_WAVE];
    __shared__ RowCoef coef;
    const uint32_t t = threadIdx.x;
    const bool own = LISTED ? t >= ND : t < SG_WAVE; // the wave of the named tokens
    const uint64_t row = r.row0 + blockIdx.x;
    const E* x = static_cast<const E*>(r.x) + row * r.ld;
    E* g = GRAD ? static_cast<E*>(out.g) + row * out.ld : nullptr;
    uint32_t first = 0;
    if constexpr (LISTED)
        if (own) first = op.fetch(row);
    if (!op.live(row)) { // the same for the whole block
        if (t == 0) op.skip(row);
        if (GRAD) zero_row<PAST>(g, r.V, t, NT);
        return;
    }
    const RowSpan sp = span_of<128>(x, r.V);
    const E* xc = x + sp.head;
    const uint32_t b0 = sp.head + mark_pad<E>(sp);
    constexpr int KEPT = GRAD ? J : 0;
    u32x4 kept[J];
    typename Op::Named nm;
    uint32_t flags = 0;
    if (!LISTED) nm = op.named(r, row, x, ls); // one address: the same load for all lanes
    if constexpr (GRAD)
        if ((!LISTED || t < ND) && sp.nc > 0) load_chunks<J, ND>(kept, xc, t, sp.nc);
    if constexpr (LISTED) {
        for (uint32_t i = t; i < (r.V + VEC + 31) / 32; i += NT) rl_bitmap[i] = 0;
        if (t < ND) ls.flag[t] = 0;
        __syncthreads();
        if (own) op.template mark<E, ND>(row, first, 0, r.V, sp, ls, rl_bitmap);
        __syncthreads();
        if (own) {
            const RowStat st = wave_stat(op.marked_chunks(xc, sp, ls, rl_bitmap, r.c), r.c);
            if (lane_id() == 0) part[NW] = st;
            nm = op.named(r, row, x, ls);
        } else {
            flags = ls.flag[t];
        }
    }
    if (!LISTED || t < ND) {
        RowStat st = {-INFINITY, 0.0};
        if constexpr (GRAD) stat_chunks<E, J, ND, Op>(st, kept, flags, t, sp.nc, r.c);
        stat_more<E, GRAD ? 2 : J, ND, Op>(st, xc, flags, rl_bitmap, b0, t, KEPT, sp.nc, r.c);
        stat_loose<E, ND, Op>(st, x, sp, rl_bitmap, t, r.c);
        st = wave_stat<SG_WAVE, Op::kFine>(st, r.c);
        if (lane_id() == 0) part[t / SG_WAVE] = st;
    }
    __syncthreads();
    if (own) {
        const uint32_t l = lane_id();
        const RowStat a = wave_stat<SG_WAVE, Op::kFine>(l < NT / SG_WAVE ? part[l] : RowStat{-INFINITY, 0.0}, r.c);
        const RowCoef k = op.finish(r, row, a, nm, true);
        if (l == 0) coef = k;
    }
    if constexpr (GRAD) {
        __syncthreads();
        if (!LISTED || t < ND) {
            E* gc = g + sp.head;
            const float cf = coef.coef, sh = shift_of(coef.m);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                asm volatile("" : "+v"(kept[j])); // unpack again rather than keep the unpacked values
                if (t + j * ND < sp.nc) grad_chunk<PAST, E>(kept[j], chunk_at<E>(gc, j * ND, t), cf, sh, r.c);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll 1
            for (uint32_t j = t + J * ND; j < sp.nc; j += ND)
                grad_chunk<PAST, E>(load_chunk(chunk_at<E>(xc, j, 0)), chunk_at<E>(gc, j, 0), cf, sh, r.c);
            grad_loose(x, g, sp, cf, sh, r.c, t, ND);
        }
        if (own) op.named_grad(r, coef, ls);
        __syncthreads(); // the named tokens' gradients replace elements that other threads wrote
        if (own) op.template put_named<E>(row, g, coef, ls, 0, r.V);
    }
}

// ---------------------------------------------------------------------------
// few long rows: several blocks per row, the sums first, then the rest
// ---------------------------------------------------------------------------
struct SplitArgs {
    RowStat* stat; // [rows][parts]
    uint32_t parts, len; // len elements to a part, a multiple of a chunk
};

constexpr int SP_NT = 512;

// Sums of one part.  Part 0 also gathers what the operator needs of the named
// tokens: a gradient in place overwrites them in the next kernel.
template <typename E, class Op>
__global__ __launch_bounds__(SP_NT, 4) void row_part_kernel(Rows r, Op op, SplitArgs s, typename Op::Named* keep)
{
    constexpr bool LISTED = Op::kListed;
    constexpr int ND = LISTED ? SP_NT - SG_WAVE : SP_NT, NW = ND / SG_WAVE, VEC = RowIO<E>::VEC;
    extern __shared__ uint32_t rl_lds[];
    typename Op::List ls = op.list(rl_lds, ND);
    uint32_t* const rl_bitmap = ls.bitmap;
    __shared__ RowStat part[SP_NT / SG_WAVE];
    const uint32_t t = threadIdx.x, lo = blockIdx.x * s.len;
    const uint64_t row = r.row0 + blockIdx.y;
    if (!op.live(row)) return;
    const bool own = LISTED ? t >= ND : t < SG_WAVE;
    const uint32_t n = r.V - lo < s.len ? r.V - lo : s.len;
    const E* xr = static_cast<const E*>(r.x) + row * r.ld;
    const E* x = xr + lo;
    const RowSpan sp = span_of<128>(x, n);
    uint32_t flags = 0;
    if constexpr (LISTED) {
        const uint32_t first = own ? op.fetch(row) : 0;
        for (uint32_t i = t; i < (n + VEC + 31) / 32; i += SP_NT) rl_bitmap[i] = 0;
        if (t < ND) ls.flag[t] = 0;
        __syncthreads();
        if (own) op.template mark<E, ND>(row, first, lo, lo + n, sp, ls, rl_bitmap);
        __syncthreads();
        if (own) {
            const RowStat st = wave_stat(op.marked_chunks(x + sp.head, sp, ls, rl_bitmap, r.c), r.c);
            if (lane_id() == 0) part[NW] = st;
        } else {
            flags = ls.flag[t];
        }
    }
    if (own && blockIdx.x == 0) {
        const typename Op::Named nm = op.named(r, row, xr, ls);
        if (lane_id() == 0) keep[row] = nm;
    }
    if (t < ND) {
        RowStat st = {-INFINITY, 0.0};
        stat_more<E, 4, ND, Op>(st, x + sp.head, flags, rl_bitmap, sp.head + mark_pad<E>(sp), t, 0, sp.nc, r.c);
        stat_loose<E, ND, Op>(st, x, sp, rl_bitmap, t, r.c);
        st = wave_stat<SG_WAVE, Op::kFine>(st, r.c);
        if (lane_id() == 0) part[t / SG_WAVE] = st;
    }
    __syncthreads();
    if (t < SG_WAVE) {
        const RowStat a = wave_stat<SG_WAVE, Op::kFine>(t < SP_NT / SG_WAVE ? part[t] : RowStat{-INFINITY, 0.0}, r.c);
        if (t == 0) s.stat[row * s.parts + blockIdx.x] = a;
    }
}

// The row's sums joined (by every block of the row), loss and gradient.
// Without GRAD one wave a row.
template <typename E, class Op, bool GRAD>
__global__ __launch_bounds__(SP_NT, 4) void row_join_kernel(Rows r, Op op, SplitArgs s, const typename Op::Named* keep,
                                                            GradOut out)
{
    extern __shared__ uint32_t rl_lds[];
    typename Op::List ls = op.list(rl_lds, 0);
    __shared__ RowCoef coef;
    const uint32_t t = threadIdx.x;
    const uint64_t row = r.row0 + blockIdx.y;
    const uint32_t lo = blockIdx.x * s.len, n = r.V - lo < s.len ? r.V - lo : s.len;
    const E* x = static_cast<const E*>(r.x) + row * r.ld + lo;
    E* g = GRAD ? static_cast<E*>(out.g) + row * out.ld + lo : nullptr;
    if (!op.live(row)) {
        if (t == 0 && blockIdx.x == 0) op.skip(row);
        if (GRAD) zero_row<false>(g, n, t, SP_NT);
        return;
    }
    if (t < SG_WAVE) {
        const RowStat a = wave_stat<SG_WAVE, Op::kFine>(t < s.parts ? s.stat[row * s.parts + t] : RowStat{-INFINITY, 0.0}, r.c);
        const RowCoef k = op.finish(r, row, a, keep[row], blockIdx.x == 0);
        if (t == 0) coef = k;
        if constexpr (GRAD && Op::kListed) // the part's listed logits, before the gradient may overwrite them
            for (uint32_t j = t; j < op.k; j += SG_WAVE) {
                const uint32_t i = op.idx[row * op.k + j];
                ls.id[j] = i;
                ls.z[j] = i >= lo && i < lo + n ? RowIO<E>::get(x + (i - lo)) : 0.f;
                ls.p[j] = (float)row_exp((double)op.logp[row * op.k + j] - keep[row].top);
            }
    }
    if constexpr (GRAD) {
        __syncthreads();
        grad_row<false>(x, g, n, coef.coef, coef.m, r.c, t, SP_NT);
        if (t < SG_WAVE) op.named_grad(r, coef, ls);
        __syncthreads();
        if (t < SG_WAVE) op.template put_named<E>(row, g, coef, ls, lo, lo + n);
    }
}

// ---------------------------------------------------------------------------
// the pair pass and the gradient pass of the preference loss
// ---------------------------------------------------------------------------
struct PairArgs {
    const uint64_t* off; // [2 * pairs + 1]
    const float *ref, *weight;
    const int32_t* label;
    const double* row_logp;
    float* slope;
    float *loss, *logp;
    uint64_t T;
    uint32_t pairs, V;
    int kind, average, grad;
    double beta, eps;
};

constexpr int PF_NT = 256;

struct PairTerm {
    uint64_t lo[2], hi[2]; // the rows of both sequences
    double S[2], each[2];  // sums, and the loss's derivative with respect to every token's log-probability
    double loss;
};

// One pair, by a block: both sequences' sums in a fixed order, the loss and
// its derivatives.  All threads hold the result.
template <int NT>
__device__ __forceinline__ PairTerm pair_term(const PairArgs& p, uint32_t b, bool report)
{
    __shared__ double part[2][NT / SG_WAVE][2];
    __shared__ double out[3];
    PairTerm q;
    double n[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t s = b + c * p.pairs;
        const uint64_t o0 = p.off[s], o1 = p.off[s + 1];
        q.lo[c] = o0 < p.T ? o0 : p.T;
        q.hi[c] = o1 < p.T ? o1 : p.T;
        if (report && (o1 > p.T || o0 > o1) && threadIdx.x == 0) report_error(kDevErrBadOffsets);
        if (q.hi[c] < q.lo[c]) q.hi[c] = q.lo[c];
        double a = 0.0, k = 0.0;
#pragma unroll 4
        for (uint64_t t = q.lo[c] + threadIdx.x; t < q.hi[c]; t += NT) {
            a += p.row_logp[t]; // 0 where the label does not count
            k += (uint32_t)p.label[t] < p.V ? 1.0 : 0.0;
        }
        a = wave_sum_f64(a);
        k = wave_sum_f64(k);
        if (lane_id() == 0) {
            part[c][threadIdx.x / SG_WAVE][0] = a;
            part[c][threadIdx.x / SG_WAVE][1] = k;
        }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        q.S[c] = n[c] = 0.0;
        for (int w = 0; w < NT / SG_WAVE; ++w) {
            q.S[c] += part[c][w][0];
            n[c] += part[c][w][1];
        }
        if (!p.average || n[c] < 1.0) n[c] = 1.0;
        q.S[c] /= n[c];
    }
    if (threadIdx.x == 0) {
        const double w = p.weight ? (double)p.weight[b] : 1.0;
        double d = q.S[0] - q.S[1];
        if (p.ref) d = (q.S[0] - (double)p.ref[b]) - (q.S[1] - (double)p.ref[b + p.pairs]);
        double L, g;
        if (p.kind == SG_PREF_IPO) {
            const double gap = d - 0.5 / p.beta;
            L = gap * gap;
            g = 2.0 * gap;
        } else if (p.kind == SG_PREF_HINGE) {
            const double gap = 1.0 - p.beta * d;
            L = gap <= 0.0 ? 0.0 : gap; // a NaN stays, in the gradient too
            g = gap <= 0.0 ? 0.0 : (gap > 0.0 ? -p.beta : gap);
        } else {
            const double h = p.beta * d, u = row_exp(-fabs(h)), l = row_log1p(u);
            const double up = l + (h < 0.0 ? -h : 0.0), down = l + (h > 0.0 ? h : 0.0);
            L = (1.0 - p.eps) * up + (p.eps != 0.0 ? p.eps * down : 0.0);
            const double sig = h >= 0.0 ? 1.0 / (1.0 + u) : u / (1.0 + u);
            const double com = h >= 0.0 ? u / (1.0 + u) : 1.0 / (1.0 + u);
            g = p.beta * (p.eps * sig - (1.0 - p.eps) * com);
        }
        if (w == 0.0) L = g = 0.0;
        out[0] = w * L;
        out[1] = w * g / n[0];
        out[2] = -w * g / n[1];
    }
    __syncthreads();
    q.loss = out[0];
    q.each[0] = out[1];
    q.each[1] = out[2];
    return q;
}

__device__ __forceinline__ void put_pair(const PairArgs& p, uint32_t b, const PairTerm& q)
{
    p.loss[b] = (float)q.loss;
    if (p.logp) {
        p.logp[b] = (float)q.S[0];
        p.logp[b + p.pairs] = (float)q.S[1];
    }
}

// one block per pair: its loss, and the slope of every row of its sequences
template <int NT>
__global__ __launch_bounds__(NT) void pref_pair_kernel(PairArgs p)
{
    for (uint32_t b = blockIdx.x; b < p.pairs; b += gridDim.x) {
        const PairTerm q = pair_term<NT>(p, b, true);
        if (threadIdx.x == 0) put_pair(p, b, q);
        if (p.grad)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                for (uint64_t t = q.lo[c] + threadIdx.x; t < q.hi[c]; t += NT)
                    p.slope[t] = (uint32_t)p.label[t] < p.V ? (float)q.each[c] : 0.f;
        __syncthreads();
    }
}

// gradient rows from the kept maximum and 1/sum: slope * (1[i = y] - q_i).
// gridDim.x parts of len elements to a row.
template <typename E, bool PAST, int NT>
__device__ __forceinline__ void pref_grad_part(const Rows& r, const TokenOp& op, uint64_t row, uint32_t lo, uint32_t n,
                                               float slope, const GradOut& out)
{
    const E* x = static_cast<const E*>(r.x) + row * r.ld + lo;
    E* g = static_cast<E*>(out.g) + row * out.ld + lo;
    if (slope == 0.f) {
        zero_row<PAST>(g, n, threadIdx.x, NT);
        return;
    }
    grad_row<PAST>(x, g, n, -slope * op.inv[row], op.m[row], r.c, threadIdx.x, NT);
    __syncthreads();
    const uint32_t y = (uint32_t)op.label[row];
    if (threadIdx.x == 0 && y >= lo && y < lo + n)
        RowIO<E>::put(g + (y - lo), (float)((double)slope * -row_expm1(op.logp[row])));
}

template <typename E, bool PAST, int NT>
__global__ __launch_bounds__(NT) void pref_grad_kernel(Rows r, TokenOp op, uint32_t len, GradOut out)
{
    const uint32_t lo = blockIdx.x * len, n = r.V - lo < len ? r.V - lo : len;
    // last row first: the token pass has just read the last rows, which are
    // still in the last-level cache (6000 x 131072 bf16: 731 -> 706 us)
    for (uint64_t y = blockIdx.y; y < r.T; y += gridDim.y) {
        const uint64_t row = r.T - 1 - y;
        pref_grad_part<E, PAST, NT>(r, op, row, lo, n, op.slope[row], out);
    }
}

// The pair pass and the gradient pass in one launch, for few rows: every block
// of a row works its pair out for itself (blockIdx.y < T), and blocks after
// them write the pairs' losses.
template <typename E>
__global__ __launch_bounds__(PF_NT) void pref_both_kernel(Rows r, TokenOp op, PairArgs p, uint32_t len, GradOut out)
{
    const uint32_t t = threadIdx.x;
    if (blockIdx.y >= p.T) {
        const uint32_t b = blockIdx.y - (uint32_t)p.T;
        if (blockIdx.x > 0) return;
        const PairTerm q = pair_term<PF_NT>(p, b, true);
        if (t == 0) put_pair(p, b, q);
        return;
    }
    __shared__ uint32_t found;
    const uint64_t row = blockIdx.y;
    const uint32_t lo = blockIdx.x * len, n = r.V - lo < len ? r.V - lo : len;
    if (t == 0) found = 2 * p.pairs;
    __syncthreads();
    for (uint32_t s = t; s < 2 * p.pairs; s += PF_NT) // one sequence has the row, or none
        if (p.off[s] <= row && row < p.off[s + 1]) found = s;
    __syncthreads();
    const uint32_t s = found;
    float slope = 0.f;
    if (s < 2 * p.pairs && (uint32_t)p.label[row] < p.V) { // the same for the whole block
        const bool chosen = s < p.pairs;
        const PairTerm q = pair_term<PF_NT>(p, chosen ? s : s - p.pairs, false);
        slope = (float)(chosen ? q.each[0] : q.each[1]);
    }
    pref_grad_part<E, false, PF_NT>(r, op, row, lo, n, slope, out);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr uint64_t ROWS_PER_LAUNCH = 1u << 20; // a launch holds fewer than 2^32 threads
constexpr uint64_t GRID_Y = 65535;

struct RowCheck {
    Rows r;
};

static uint64_t row_esize(sg_dtype dt) { return dt == SG_BF16 ? 2 : 4; }

// the checks every rows call shares
static int rows_args(const void* x, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld, double inv_temp, RowCheck* out,
                     bool fine = false)
{
    if (dt != SG_F32 && dt != SG_BF16) return SG_EINVAL;
    if (V == 0 || V >= (1ull << 31) || T >= (1ull << 31) || ld < V || ld >= (1ull << 40)) return SG_EINVAL;
    // below 1e-37 the fp32 scale would lose its digits, then be 0: -inf * 0 = NaN
    if (!(inv_temp >= 1e-37) || !(inv_temp <= 1e6)) return SG_EINVAL;
    if (T > 0 && (!x || reinterpret_cast<uintptr_t>(x) % row_esize(dt) != 0)) return SG_EINVAL;
    out->r.x = x;
    out->r.T = T;
    out->r.row0 = 0;
    out->r.ld = ld;
    out->r.V = (uint32_t)V;
    const double c = inv_temp * 1.4426950408889634074; // log2(e)
    out->r.c.hi = (float)c;
    out->r.c.lo = 0.f;
    out->r.it = out->r.c.hi * kLn2;
    if (fine) {
        if (out->r.c.hi >= c) out->r.c.hi = nextafterf(out->r.c.hi, 0.0f);
        out->r.c.lo = (float)(c - out->r.c.hi);
        out->r.it = inv_temp;
    }
    return SG_OK;
}

static int grad_args(const void* x, uint64_t ld, const void* grad, sg_dtype dt, uint64_t V, uint64_t ldg)
{
    if (!grad) return SG_OK;
    if (grad == x && ldg != ld) return SG_EINVAL; // in place: the same rows
    if (ldg < V || ldg >= (1ull << 40) || reinterpret_cast<uintptr_t>(grad) % row_esize(dt) != 0) return SG_EINVAL;
    return SG_OK;
}

// A gradient larger than the 256 MB last-level cache leaves nothing in it for
// its reader, so its stores go past the caches (8192 x 131072 bf16: 660 ->
// 623 us).  Where logits and gradient lie differently in their lines a wave's
// stores do not fill lines, and that costs more than it gains (6000 x 100003:
// 482 -> 520 us).
static GradOut grad_out(const RowCheck& c, sg_dtype dt, void* grad, uint64_t ldg)
{
    const uint64_t e = row_esize(dt);
    const uintptr_t apart = reinterpret_cast<uintptr_t>(grad) - reinterpret_cast<uintptr_t>(c.r.x);
    const bool alike = apart % 128 == 0 && (ldg - c.r.ld) * e % 128 == 0;
    return {grad, ldg, alike && c.r.T * c.r.V * e > (256ull << 20)};
}

// Few rows leave most of the chip idle with a block per row, and one compute
// unit takes some 11 us for 128 KiB of row; parts of 32 KiB in two launches
// take about 10 us and 4 us more on the host, so rows longer than that are
// split when there are fewer than 128.
static uint32_t row_parts(uint64_t T, uint64_t V, uint64_t esize)
{
    const uint64_t bytes = V * esize;
    if (T >= 128 || bytes <= 128 * 1024) return 1;
    const uint64_t p = ceil_div(bytes, 32 * 1024);
    return (uint32_t)(p < RL_MAX_PARTS ? p : RL_MAX_PARTS);
}

// elements to a part: whole chunks, and no part empty
static uint32_t part_len(uint64_t V, uint32_t* parts)
{
    const uint64_t len = align_up(ceil_div(V, *parts), 64);
    *parts = (uint32_t)ceil_div(V, len);
    return (uint32_t)len;
}

template <class Op>
struct SplitWs {
    RowStat* stat;
    typename Op::Named* keep;
};

template <class Op>
static SplitWs<Op> split_carve(Carver& cv, uint64_t T, uint32_t parts)
{
    SplitWs<Op> w = {nullptr, nullptr};
    if (parts > 1) {
        w.stat = cv.take<RowStat>(T * parts);
        w.keep = cv.take<typename Op::Named>(T);
    }
    return w;
}

// a listed row, or its part, has its bitmap in LDS (32 KiB): longer rows are split whatever their number
constexpr uint64_t RL_MAX_BITS = 1u << 18;
template <class Op>
static uint32_t op_parts(uint64_t T, uint64_t V, sg_dtype dt)
{
    uint32_t parts = row_parts(T, V, row_esize(dt));
    if (Op::kListed && V > RL_MAX_BITS * parts) parts = (uint32_t)ceil_div(V, RL_MAX_BITS);
    return parts;
}

template <class Op>
static size_t split_bytes(uint64_t T, uint64_t V, sg_dtype dt)
{
    if (T >= (1ull << 31) || V == 0 || V >= (1ull << 31) || (dt != SG_F32 && dt != SG_BF16)) return 0;
    const uint32_t parts = op_parts<Op>(T, V, dt);
    Carver cv(nullptr);
    split_carve<Op>(cv, T, parts);
    return parts > 1 ? cv.bytes() : 0;
}

// dynamic LDS of a kernel whose blocks take V elements: the list and its bitmap
template <class Op>
static size_t list_lds(const Op& op, uint32_t threads, uint64_t V)
{
    if constexpr (Op::kListed) return 4 * (Op::list_words(op.k, threads) + (V > 0 ? ceil_div(V + 8, 32) : 0));
    return 0;
}

template <typename E, int NT, int J, int WAVES, class Op>
static int launch_rows(const RowCheck& c, const Op& op, const GradOut& out, hipStream_t st)
{
    const size_t lds = list_lds(op, NT - SG_WAVE, c.r.V);
    Rows r = c.r;
    for (r.row0 = 0; r.row0 < r.T; r.row0 += ROWS_PER_LAUNCH) {
        const uint64_t left = r.T - r.row0;
        const unsigned grid = (unsigned)(left < ROWS_PER_LAUNCH ? left : ROWS_PER_LAUNCH);
        if constexpr (Op::kGrad) {
            if (out.g && out.past) row_loss_kernel<E, NT, J, Op, true, true, WAVES><<<grid, NT, lds, st>>>(r, op, out);
            if (out.g && !out.past) row_loss_kernel<E, NT, J, Op, true, false, WAVES><<<grid, NT, lds, st>>>(r, op, out);
        }
        if (!out.g) row_loss_kernel<E, NT, 2, Op, false, false, 8><<<grid, NT, lds, st>>>(r, op, out);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}

template <typename E, class Op>
static int launch_split(const RowCheck& c, const Op& op, uint32_t parts, const GradOut& out, void* ws,
                        hipStream_t st)
{
    Carver cv(ws);
    const SplitWs<Op> w = split_carve<Op>(cv, c.r.T, parts);
    SplitArgs s = {w.stat, parts, 0};
    s.len = part_len(c.r.V, &s.parts);
    const size_t lds = list_lds(op, SP_NT - SG_WAVE, s.len), lds_join = list_lds(op, 0, 0);
    Rows r = c.r;
    typename Op::Named* keep = w.keep;
    for (r.row0 = 0; r.row0 < c.r.T; r.row0 += GRID_Y) {
        const unsigned rows = (unsigned)(c.r.T - r.row0 < GRID_Y ? c.r.T - r.row0 : GRID_Y);
        row_part_kernel<E, Op><<<dim3(s.parts, rows), SP_NT, lds, st>>>(r, op, s, keep);
        SG_TRY_LAUNCH();
        if constexpr (Op::kGrad)
            if (out.g) row_join_kernel<E, Op, true><<<dim3(s.parts, rows), SP_NT, lds_join, st>>>(r, op, s, keep, out);
        if (!out.g) row_join_kernel<E, Op, false><<<dim3(1, rows), SG_WAVE, 0, st>>>(r, op, s, keep, out);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}

// Threads, chunks kept and waves per SIMD by the row's bytes, measured on
// rows of bf16 with a policy gradient (TB/s read and written): 8 KB 4.6 with
// 256 threads, 2.8 with 512; 32 KB 5.2 with 512, 4.8 with 256; 100 KB 5.1
// with 512 threads that keep 16 chunks, 4.5 with 1024; 200 KB 5.05 with 1024,
// 4.7 with 512 (which keep half of it and read the rest again).  A listed row
// of up to 32 KB takes 512 threads that keep 5 chunks, three blocks to a
// compute unit: with 9, two blocks, 8000 x 16000 bf16 took 174 us, not 143.
template <typename E, class Op>
static int launch_row_loss_of(const RowCheck& c, const Op& op, const GradOut& out, void* ws, sg_dtype dt,
                              hipStream_t st)
{
    const uint32_t parts = op_parts<Op>(c.r.T, c.r.V, dt);
    if (parts > 1) return launch_split<E>(c, op, parts, out, ws, st);
    const uint64_t bytes = (uint64_t)c.r.V * sizeof(E);
    constexpr bool L = Op::kListed; // one wave less for the row
    if (bytes <= 4 * 1024) return launch_rows<E, L ? 128 : 64, 4, L ? 6 : 8>(c, op, out, st);
    if (bytes <= 16 * 1024) return launch_rows<E, 256, L ? 6 : 4, L ? 6 : 8>(c, op, out, st);
    if (L && bytes <= 32 * 1024) return launch_rows<E, 512, 5, 6>(c, op, out, st);
    if (bytes <= 64 * 1024) return launch_rows<E, 512, L ? 9 : 8, L ? 4 : 8>(c, op, out, st);
    if (bytes <= 128 * 1024) return launch_rows<E, 512, L ? 18 : 16, 4>(c, op, out, st);
    return launch_rows<E, 1024, L ? 17 : 16, 4>(c, op, out, st);
}

template <class Op>
static int launch_row_loss(const RowCheck& c, sg_dtype dt, const Op& op, const GradOut& out, void* ws,
                           hipStream_t st)
{
    if (dt == SG_BF16) return launch_row_loss_of<bf16_bits>(c, op, out, ws, dt, st);
    return launch_row_loss_of<float>(c, op, out, ws, dt, st);
}

// a split call's workspace
template <class Op>
static int check_split_ws(uint64_t T, uint64_t V, sg_dtype dt, const void* ws, size_t ws_bytes)
{
    const size_t need = split_bytes<Op>(T, V, dt);
    if (need > 0 && !ws) return SG_EINVAL;
    return ws_bytes < need ? SG_ECAPACITY : SG_OK;
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_distill_workspace_bytes(uint64_t T, uint64_t V, uint32_t k, sg_dtype dt)
{
    return split_bytes<DistillOp>(T, V, dt);
}

extern "C" int sg_distill_loss(const void* d_logits, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld,
                               double inv_temp, const uint32_t* d_idx, const float* d_logp, uint32_t k,
                               sg_distill_mode mode, const float* d_weight, float* d_loss, void* d_grad,
                               uint64_t ld_grad, void* d_ws, size_t ws_bytes, void* stream)
{
    RowCheck c;
    int rc = rows_args(d_logits, dt, T, V, ld, inv_temp, &c);
    if (rc) return rc;
    if (k == 0) return SG_EINVAL;
    if (mode != SG_DISTILL_PLAIN && mode != SG_DISTILL_RENORM && mode != SG_DISTILL_TAIL) return SG_EINVAL;
    if ((rc = grad_args(d_logits, ld, d_grad, dt, V, ld_grad))) return rc;
    if (T > 0 && (!d_idx || !d_logp || !d_loss)) return SG_EINVAL;
    if (k > SG_ROWS_MAX_K || V > RL_MAX_BITS * RL_MAX_PARTS) return SG_EUNSUPPORTED;
    if (T == 0) return SG_OK;
    if ((rc = check_split_ws<DistillOp>(T, V, dt, d_ws, ws_bytes))) return rc;
    DistillOp op = {d_idx, d_logp, d_weight, d_loss, k, (uint32_t)V, (int)mode};
    return launch_row_loss(c, dt, op, grad_out(c, dt, d_grad, ld_grad), d_ws, as_stream(stream));
}

extern "C" size_t sg_policy_workspace_bytes(uint64_t T, uint64_t V, sg_dtype dt)
{
    return split_bytes<PolicyOp>(T, V, dt);
}

extern "C" int sg_policy_loss(const void* d_logits, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld, double inv_temp,
                              const int32_t* d_action, const float* d_old_logp, const float* d_ref_logp,
                              const float* d_adv, const float* d_weight, double clip_low, double clip_high,
                              double kl_coef, float* d_loss, float* d_logp, void* d_grad, uint64_t ld_grad,
                              void* d_ws, size_t ws_bytes, void* stream)
{
    RowCheck c;
    int rc = rows_args(d_logits, dt, T, V, ld, inv_temp, &c);
    if (rc) return rc;
    if (!(clip_low >= 0.0) || !(clip_low <= 1.0) || !(clip_high >= 0.0) || !(clip_high <= 1e6)) return SG_EINVAL;
    if (!(kl_coef >= 0.0) || !(kl_coef <= 1e6)) return SG_EINVAL;
    if ((rc = grad_args(d_logits, ld, d_grad, dt, V, ld_grad))) return rc;
    if (T > 0 && (!d_action || !d_loss)) return SG_EINVAL;
    if (T == 0) return SG_OK;
    if ((rc = check_split_ws<PolicyOp>(T, V, dt, d_ws, ws_bytes))) return rc;
    PolicyOp op = {d_action, d_old_logp, kl_coef != 0.0 ? d_ref_logp : nullptr, d_adv, d_weight, d_loss, d_logp,
                   1.0 - clip_low, 1.0 + clip_high, kl_coef, (uint32_t)V};
    return launch_row_loss(c, dt, op, grad_out(c, dt, d_grad, ld_grad), d_ws, as_stream(stream));
}

namespace sg {
struct PrefWs {
    double* logp;
    float *m, *inv, *slope;
    void* split; // of the token pass
};
static PrefWs pref_carve(Carver& cv, uint64_t T, uint64_t V, sg_dtype dt)
{
    PrefWs w;
    w.split = cv.take<char>(split_bytes<TokenOp>(T, V, dt));
    w.logp = cv.take<double>(T);
    w.m = cv.take<float>(T);
    w.inv = cv.take<float>(T);
    w.slope = cv.take<float>(T);
    return w;
}
} // namespace sg

extern "C" size_t sg_preference_workspace_bytes(uint64_t T, uint64_t V, sg_dtype dt)
{
    if (T >= (1ull << 31) || V == 0 || V >= (1ull << 31) || (dt != SG_F32 && dt != SG_BF16)) return 0;
    Carver cv(nullptr);
    pref_carve(cv, T, V, dt);
    return cv.bytes();
}

extern "C" int sg_preference_loss(const void* d_logits, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld,
                                  const int32_t* d_label, const uint64_t* d_seq_off, uint32_t pairs,
                                  const float* d_ref_logp, const float* d_weight, sg_pref_kind kind, double beta,
                                  double smoothing, int average, float* d_loss, float* d_logp, void* d_grad,
                                  uint64_t ld_grad, void* d_ws, size_t ws_bytes, void* stream)
{
    RowCheck c;
    int rc = rows_args(d_logits, dt, T, V, ld, 1.0, &c, TokenOp::kFine);
    if (rc) return rc;
    if (kind != SG_PREF_SIGMOID && kind != SG_PREF_HINGE && kind != SG_PREF_IPO) return SG_EINVAL;
    if (!(beta > 0.0) || !(beta <= 1e6) || !(smoothing >= 0.0) || !(smoothing < 0.5)) return SG_EINVAL;
    if (smoothing != 0.0 && kind != SG_PREF_SIGMOID) return SG_EINVAL;
    if (pairs >= (1u << 30)) return SG_EINVAL;
    if ((rc = grad_args(d_logits, ld, d_grad, dt, V, ld_grad))) return rc;
    if ((T > 0 && !d_label) || (pairs > 0 && (!d_seq_off || !d_loss)) || !d_ws) return SG_EINVAL;
    if (ws_bytes < sg_preference_workspace_bytes(T, V, dt)) return SG_ECAPACITY;
    hipStream_t st = as_stream(stream);
    Carver cv(d_ws);
    const PrefWs w = pref_carve(cv, T, V, dt);
    TokenOp op = {d_label, w.logp, w.m, w.inv, w.slope, (uint32_t)V};
    if (T > 0 && (rc = launch_row_loss(c, dt, op, GradOut{nullptr, 0, false}, w.split, st))) return rc;
    const PairArgs p = {d_seq_off, d_ref_logp, d_weight, d_label, w.logp, w.slope, d_loss, d_logp, T, pairs,
                        (uint32_t)V, (int)kind, average ? 1 : 0, d_grad ? 1 : 0, beta, smoothing};
    const GradOut out = grad_out(c, dt, d_grad, ld_grad);
    // gradient: enough blocks to fill the chip, at least 16 KiB of row to each
    uint32_t parts = 1;
    if (T > 0 && d_grad) {
        const uint64_t most = ceil_div(V * row_esize(dt), 16 * 1024), want = ceil_div(1024, T);
        parts = (uint32_t)(want < most ? want : most);
    }
    const uint32_t len = part_len(V, &parts);
    // A launch less (4 us on the host, 5 on the GPU for 90 rows) while a
    // block's own sums over its pair are short.  us a call, joint and apart,
    // bf16: 90 x 32000 15.7, 18.3; 1024 x 32000 39.9, 41.7; 1024 x 131072 166.7, 169.0;
    // 2048 x 131072 320, 292 (its row order and stores past the caches are not
    // used).  The pairs bound a block's search for its sequence, 2 offsets a
    // thread at 256: 1024 x 4000 15.7, 18.4 with 256 pairs, and still 15.7, 18.5 with 512.
    if (T > 0 && d_grad && pairs > 0 && T <= 1024 && pairs <= 256) {
        const dim3 grid(parts, (unsigned)(T + pairs));
        if (dt == SG_BF16) pref_both_kernel<bf16_bits><<<grid, PF_NT, 0, st>>>(c.r, op, p, len, out);
        else pref_both_kernel<float><<<grid, PF_NT, 0, st>>>(c.r, op, p, len, out);
        SG_TRY_LAUNCH();
        return SG_OK;
    }
    if (pairs > 0) {
        const unsigned blocks = pairs < 65536u ? pairs : 65536u;
        // long sequences: more loads in flight; short ones: fewer waves to join.
        // us a call, 256 and 1024 threads: 2 pairs of 20000 x 64 bf16 20.9, 19.5, of 40000 x 64 32.9, 29.9;
        // within 2% of each other from 2000 to 8000 rows a pair; 24 pairs of 5000 x 65536 120.1, 121.3
        if (T / pairs > 2048) pref_pair_kernel<1024><<<blocks, 1024, 0, st>>>(p);
        else pref_pair_kernel<PF_NT><<<blocks, PF_NT, 0, st>>>(p);
        SG_TRY_LAUNCH();
    }
    if (T > 0 && d_grad) {
        const dim3 grid(parts, (unsigned)(T < GRID_Y ? T : GRID_Y));
        const bool narrow = V * row_esize(dt) <= 4 * 1024; // a wave a row
        const auto go = [&](auto e) {
            typedef decltype(e) E;
            if (out.past) pref_grad_kernel<E, true, PF_NT><<<grid, PF_NT, 0, st>>>(c.r, op, len, out);
            else if (narrow) pref_grad_kernel<E, false, SG_WAVE><<<grid, SG_WAVE, 0, st>>>(c.r, op, len, out);
            else pref_grad_kernel<E, false, PF_NT><<<grid, PF_NT, 0, st>>>(c.r, op, len, out);
        };
        if (dt == SG_BF16) go(bf16_bits());
        else go(float());
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}
