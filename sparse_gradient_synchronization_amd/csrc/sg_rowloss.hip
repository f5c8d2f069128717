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

constexpr int RL_NT = 256;
constexpr uint32_t RL_MAX_K = SG_ROWS_MAX_K;

// the dense part of a row's gradient: coef * exp2(c * (x_i - m))
struct RowCoef {
    float m, coef;
};

// ---------------------------------------------------------------------------
// the clipped policy loss
// ---------------------------------------------------------------------------
struct PolicyOp {
    const int32_t* action;
    const float *old_logp, *ref_logp, *adv, *weight;
    float *loss, *logp;
    double lo, hi, kl;
    uint32_t V;

    static constexpr bool kListed = false, kGrad = true;
    struct Shared {
        float za, fix;
    };

    __device__ __forceinline__ bool live(uint64_t row) const
    {
        return (uint32_t)action[row] < V && (!weight || weight[row] != 0.f);
    }
    __device__ __forceinline__ void skip(uint64_t row) const
    {
        loss[row] = 0.f;
        if (logp) logp[row] = 0.f;
    }
    template <typename E, int NT>
    __device__ __forceinline__ void begin(const Rows&, uint64_t row, const E* x, uint32_t, Shared& sh, uint32_t*) const
    {
        if (threadIdx.x == 0) sh.za = RowIO<E>::get(x + action[row]);
    }
    // lane 0 of wave 0
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, Shared& sh) const
    {
        const double S = st.s;
        const double lp = sh.za == -INFINITY ? -(double)INFINITY : ((double)sh.za - st.m) * r.it - row_log(S);
        const double w = weight ? (double)weight[row] : 1.0;
        const double A = adv ? (double)adv[row] : 0.0;
        const double ratio = old_logp ? row_exp(lp - (double)old_logp[row]) : 1.0;
        const double bounded = ratio < lo ? lo : (ratio > hi ? hi : ratio);
        const double a = ratio * A, b = bounded * A;
        double L = a <= b ? -a : (b <= a ? -b : a + b); // a NaN stays
        // where the bounded product is the smaller one the loss does not move
        const bool clipped = (A > 0.0 && ratio > hi) || (A < 0.0 && ratio < lo);
        double slope = clipped ? 0.0 : -a;
        if (ref_logp) {
            const double d = (double)ref_logp[row] - lp, e = row_expm1(d);
            L += kl * (e - d);
            slope -= kl * e;
        }
        loss[row] = (float)(w * L);
        if (logp) logp[row] = (float)lp;
        const double g = w * slope * r.it;
        sh.fix = (float)(g * -row_expm1(lp)); // 1 - q of the token, without the cancellation
        return {st.m, (float)(-g * inverse_of(S))};
    }
    template <typename E, int NT>
    __device__ __forceinline__ void fix(const Rows& r, uint64_t row, E* g, const Shared& sh, RowCoef) const
    {
        if (threadIdx.x == 0) RowIO<E>::put(g + action[row], sh.fix);
    }
    __device__ __forceinline__ uint32_t bits(const uint32_t*, uint32_t, int) const { return 0; }
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

    static constexpr bool kListed = false, kGrad = false;
    struct Shared {
        float za;
    };
    __device__ __forceinline__ bool live(uint64_t row) const { return (uint32_t)label[row] < V; }
    __device__ __forceinline__ void skip(uint64_t row) const
    {
        logp[row] = 0.0;
        slope[row] = 0.f;
    }
    template <typename E, int NT>
    __device__ __forceinline__ void begin(const Rows&, uint64_t row, const E* x, uint32_t, Shared& sh, uint32_t*) const
    {
        if (threadIdx.x == 0) sh.za = RowIO<E>::get(x + label[row]);
    }
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, Shared& sh) const
    {
        logp[row] = sh.za == -INFINITY ? -(double)INFINITY : ((double)sh.za - st.m) * r.it - row_log((double)st.s);
        m[row] = st.m;
        inv[row] = (float)inverse_of(st.s);
        slope[row] = 0.f;
        return {st.m, 0.f};
    }
    __device__ __forceinline__ uint32_t bits(const uint32_t*, uint32_t, int) const { return 0; }
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

    static constexpr bool kListed = true, kGrad = true;
    struct Shared {
        float z[RL_MAX_K]; // the listed logits, read before the gradient may overwrite them
        double P, A, S;    // mass, sum p (log p - (z - m)), sum exp(z - m), z scaled by inv_temp
        float m;
        double gp;           // scale of p in the gradient
        float within;        // the listed tokens' factor of exp2(c (x - m))
    };
    __device__ __forceinline__ bool live(uint64_t row) const { return !weight || weight[row] != 0.f; }
    __device__ __forceinline__ void skip(uint64_t row) const { loss[row] = 0.f; }
    template <typename E, int NT>
    __device__ __forceinline__ void begin(const Rows& r, uint64_t row, const E* x, uint32_t pad, Shared& sh,
                                          uint32_t* bm) const
    {
        const uint32_t* id = idx + row * k;
        const float* lp = logp + row * k;
        for (uint32_t i = threadIdx.x; i < (V + pad + 31) / 32; i += NT) bm[i] = 0;
        __syncthreads();
        for (uint32_t j = threadIdx.x; j < k; j += NT) {
            const uint32_t i = id[j];
            if (i >= V) continue;
            const uint32_t at = i + pad, was = atomicOr(&bm[at / 32], 1u << (at % 32));
            if (was >> (at % 32) & 1u) report_error(kDevErrUnsorted); // listed twice
            sh.z[j] = RowIO<E>::get(x + i);
        }
        __syncthreads();
        if (threadIdx.x < SG_WAVE) {
            float m = -INFINITY;
            for (uint32_t j = threadIdx.x; j < k; j += SG_WAVE)
                if (id[j] < V) m = fmaxf(m, sh.z[j]);
            for (int d = 1; d < SG_WAVE; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, SG_WAVE));
            const double shift = shift_of(m);
            double P = 0.0, A = 0.0, S = 0.0;
            for (uint32_t j = threadIdx.x; j < k; j += SG_WAVE) {
                if (id[j] >= V) continue;
                const double t = lp[j], z = sh.z[j], p = row_exp(t);
                P += p;
                if (p != 0.0) A += p * (t - (z - shift) * r.it);
                S += row_exp((z - shift) * r.it);
            }
            P = wave_sum_f64(P);
            A = wave_sum_f64(A);
            S = wave_sum_f64(S);
            if (threadIdx.x == 0) {
                sh.P = P;
                sh.A = A;
                sh.S = S;
                sh.m = m;
            }
        }
    }
    __device__ __forceinline__ RowCoef finish(const Rows& r, uint64_t row, RowStat st, Shared& sh) const
    {
        const float m = fmaxf(st.m, sh.m);
        const double shift = shift_of(m);
        const double rest = (double)st.s * row_exp(((double)st.m - shift) * r.it);
        const double own = sh.S * row_exp(((double)sh.m - shift) * r.it);
        const double S = rest + own;
        // lse less the listed maximum (a row may lie at the type's lowest
        // value, where lse itself holds no digit of log S); of a row of
        // nothing but -inf, A decides
        const double lse = m == -INFINITY ? 0.0 : (shift - shift_of(sh.m)) * r.it + row_log(S);
        const double w = weight ? (double)weight[row] : 1.0;
        double P = sh.P, A = sh.A, R = 0.0, gp = 1.0, L;
        if (mode == SG_DISTILL_RENORM) {
            gp = P > 0.0 ? 1.0 / P : P; // nothing listed: no mass, no loss (a NaN stays)
            L = P > 0.0 ? A * gp - row_log(P) + lse : P;
            P = P > 0.0 ? 1.0 : P;
        } else {
            L = A + P * lse;
            // what is left for the unlisted tokens, where there are any
            if (mode == SG_DISTILL_TAIL && P < 1.0 && rest != 0.0) {
                R = 1.0 - P;
                L += R * (row_log(R) + row_log(S / rest));
            }
        }
        loss[row] = (float)(w * L);
        const double g = w * r.it;
        const double all = (P + R) * inverse_of(S);
        sh.gp = g * gp;
        sh.within = (float)(g * all);
        return {m, (float)(g * (R != 0.0 ? all - R / rest : all))};
    }
    template <typename E, int NT>
    __device__ __forceinline__ void fix(const Rows& r, uint64_t row, E* g, const Shared& sh, RowCoef co) const
    {
        const uint32_t* id = idx + row * k;
        const float* lp = logp + row * k;
        for (uint32_t j = threadIdx.x; j < k; j += NT) {
            const uint32_t i = id[j];
            if (i >= V) continue;
            const float e = exp2_fast((sh.z[j] - shift_of(co.m)) * r.c);
            RowIO<E>::put(g + i, (float)((double)sh.within * e - sh.gp * row_exp((double)lp[j])));
        }
    }
    // bit v of the result: element i0 + v - pad is listed (i0 a multiple of n = 4 or 8, or n = 1); pad is
    // what makes the first element of a chunk a multiple of the chunk's size
    __device__ __forceinline__ uint32_t bits(const uint32_t* bm, uint32_t i0, int n) const
    {
        return bm[i0 / 32] >> (i0 % 32) & ((1u << n) - 1u);
    }
};

// ---------------------------------------------------------------------------
// one block per row
// ---------------------------------------------------------------------------
template <typename E>
__device__ __forceinline__ void zero_row(E* g, uint32_t V, uint32_t t, uint32_t nt)
{
    constexpr int VEC = RowIO<E>::VEC;
    const RowSpan sp = span_of(g, V);
    const u32x4 z = {0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t j = t; j < sp.nc; j += nt) store_chunk(chunk_at<E>(g + sp.head, j, 0), z);
    for (uint32_t i = loose_element(sp, VEC, t); i < V; i = loose_element(sp, VEC, t += nt)) RowIO<E>::put(g + i, 0.f);
}

template <typename E>
__device__ __forceinline__ void grad_chunk(u32x4 w, E* g, RowCoef k, float c)
{
    constexpr int VEC = RowIO<E>::VEC;
    const float sh = shift_of(k.m);
    float v[VEC];
    RowIO<E>::unpack(w, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = k.coef * exp2_fast((v[i] - sh) * c);
    store_chunk(g, RowIO<E>::pack(v));
}

// the elements outside the chunks
template <typename E>
__device__ __forceinline__ void grad_loose(const E* x, E* g, const RowSpan& sp, RowCoef k, float c, uint32_t t,
                                           uint32_t nt)
{
    constexpr int VEC = RowIO<E>::VEC;
    const float sh = shift_of(k.m);
#pragma unroll 1
    for (uint32_t i = loose_element(sp, VEC, t); i < sp.V; i = loose_element(sp, VEC, t += nt))
        RowIO<E>::put(g + i, k.coef * exp2_fast((RowIO<E>::get(x + i) - sh) * c));
}

// gradient of a row: coef * exp2(c (x - m)).  x and g may be the same row:
// every thread reads an element before it writes it, and nobody else touches
// it.
template <typename E>
__device__ __forceinline__ void grad_row(const E* x, E* g, uint32_t V, RowCoef k, float c, uint32_t t, uint32_t nt)
{
    const RowSpan sp = span_of(x, V);
#pragma unroll 2
    for (uint32_t j = t; j < sp.nc; j += nt)
        grad_chunk<E>(load_chunk(chunk_at<E>(x + sp.head, j, 0)), chunk_at<E>(g + sp.head, j, 0), k, c);
    grad_loose(x, g, sp, k, c, t, nt);
}

template <typename E, int J, int NT, class Op>
__device__ __forceinline__ void stat_chunks(RowStat& st, const u32x4* w, const Op& op, const uint32_t* bm, uint32_t j0,
                                            uint32_t nc, float c)
{
    constexpr int VEC = RowIO<E>::VEC;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if (j0 + j * NT < nc) {
            float v[VEC];
            u32x4 u = w[j];
            if (Op::kListed) {
                const uint32_t b = op.bits(bm, (j0 + j * NT + 1) * VEC, VEC);
                if (b) u = RowIO<E>::without(u, b);
                asm volatile("" : "+v"(u)); // one unpacked form of the chunk, not one for each side of the branch
            }
            RowIO<E>::unpack(u, v);
            stat_add<VEC>(st, v, c);
        }
        __builtin_amdgcn_sched_barrier(0); // a chunk at a time: unpacked, a chunk takes twice its registers
    }
}

// One block per row (no loop over rows: the constants of the fp64 functions
// would be hoisted out of it into registers that the row needs).  With GRAD
// the first NT * J chunks of the row stay in registers from the sums to the
// gradient, so the row is read from HBM once; what is beyond them is read
// again (from the last-level cache, the blocks in flight hold few rows).
// Without GRAD nothing is kept and J is the number of loads a thread has in
// flight.
template <typename E, int NT, int J, class Op, bool GRAD>
__global__ __launch_bounds__(NT, GRAD ? 4 : 8) void row_loss_kernel(Rows r, Op op, void* grad, uint64_t ldg)
{
    constexpr int VEC = RowIO<E>::VEC, NW = NT / SG_WAVE;
    extern __shared__ uint32_t rl_bitmap[];
    __shared__ typename Op::Shared sh;
    __shared__ RowStat part[NW];
    __shared__ RowCoef coef;
    const uint32_t t = threadIdx.x;
    const uint64_t row = r.row0 + blockIdx.x;
    const E* x = static_cast<const E*>(r.x) + row * r.ld;
    E* g = GRAD ? static_cast<E*>(grad) + row * ldg : nullptr;
    if (!op.live(row)) { // the same for the whole block
        if (t == 0) op.skip(row);
        if (GRAD) zero_row(g, r.V, t, NT);
        return;
    }
    const RowSpan sp = span_of(x, r.V);
    const E* xc = x + sp.head;
    u32x4 kept[J];
    load_chunks<J, NT>(kept, xc, t, sp.nc);
    op.template begin<E, NT>(r, row, x, VEC - sp.head, sh, rl_bitmap);
    RowStat st = {-INFINITY, 0.f};
    stat_chunks<E, J, NT>(st, kept, op, rl_bitmap, t, sp.nc, r.c);
    constexpr int M = GRAD ? 2 : J; // chunks in flight beyond the kept ones
#pragma unroll 1
    for (uint32_t j = t + J * NT; j < sp.nc; j += M * NT) {
        u32x4 more[M];
        load_chunks<M, NT>(more, xc, j, sp.nc);
        stat_chunks<E, M, NT>(st, more, op, rl_bitmap, j, sp.nc, r.c);
    }
    if (t < 2 * VEC) {
        const uint32_t i = loose_element(sp, VEC, t);
        if (i < r.V) {
            float v = RowIO<E>::get(x + i);
            if (Op::kListed && op.bits(rl_bitmap, i + VEC - sp.head, 1)) v = -INFINITY;
            stat_add<1>(st, &v, r.c);
        }
    }
    st = wave_stat(st, r.c);
    if (lane_id() == 0) part[t / SG_WAVE] = st;
    __syncthreads();
    if (t < NW) {
        const RowStat a = wave_stat<NW>(part[t], r.c);
        if (t == 0) coef = op.finish(r, row, a, sh);
    }
    if constexpr (GRAD) {
        __syncthreads();
        const RowCoef k = coef;
        E* gc = g + sp.head;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            asm volatile("" : "+v"(kept[j])); // unpack again rather than keep the unpacked values
            if (t + j * NT < sp.nc) grad_chunk<E>(kept[j], chunk_at<E>(gc, j * NT, t), k, r.c);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        for (uint32_t j = t + J * NT; j < sp.nc; j += NT)
            grad_chunk<E>(load_chunk(chunk_at<E>(xc, j, 0)), chunk_at<E>(gc, j, 0), k, r.c);
        grad_loose(x, g, sp, k, r.c, t, NT);
        __syncthreads(); // the corrections overwrite elements of other threads
        op.template fix<E, NT>(r, row, g, sh, k);
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

// one block per pair: both sequences' sums in a fixed order, the loss, and
// the derivative with respect to every token's log-probability
__global__ __launch_bounds__(PF_NT) void pref_pair_kernel(PairArgs p)
{
    __shared__ double part[PF_NT / SG_WAVE][2];
    __shared__ double each[2];
    for (uint32_t b = blockIdx.x; b < p.pairs; b += gridDim.x) {
        uint64_t lo[2], hi[2];
        double S[2], n[2];
        for (int c = 0; c < 2; ++c) {
            const uint32_t s = b + c * p.pairs;
            lo[c] = p.off[s] < p.T ? p.off[s] : p.T;
            hi[c] = p.off[s + 1] < p.T ? p.off[s + 1] : p.T;
            if ((p.off[s + 1] > p.T || p.off[s] > p.off[s + 1]) && threadIdx.x == 0) report_error(kDevErrBadOffsets);
            if (hi[c] < lo[c]) hi[c] = lo[c];
            double a = 0.0, k = 0.0;
            for (uint64_t t = lo[c] + threadIdx.x; t < hi[c]; t += PF_NT) {
                a += p.row_logp[t]; // 0 where the label does not count
                k += (uint32_t)p.label[t] < p.V ? 1.0 : 0.0;
            }
            a = wave_sum_f64(a);
            k = wave_sum_f64(k);
            __syncthreads();
            if (lane_id() == 0) {
                part[threadIdx.x / SG_WAVE][0] = a;
                part[threadIdx.x / SG_WAVE][1] = k;
            }
            __syncthreads();
            S[c] = n[c] = 0.0;
            for (int w = 0; w < PF_NT / SG_WAVE; ++w) {
                S[c] += part[w][0];
                n[c] += part[w][1];
            }
            if (!p.average || n[c] < 1.0) n[c] = 1.0;
            S[c] /= n[c];
        }
        if (threadIdx.x == 0) {
            const double w = p.weight ? (double)p.weight[b] : 1.0;
            double d = S[0] - S[1];
            if (p.ref) d = (S[0] - (double)p.ref[b]) - (S[1] - (double)p.ref[b + p.pairs]);
            double L, g;
            if (p.kind == SG_PREF_IPO) {
                const double gap = d - 0.5 / p.beta;
                L = gap * gap;
                g = 2.0 * gap;
            } else if (p.kind == SG_PREF_HINGE) {
                const double gap = 1.0 - p.beta * d;
                L = gap <= 0.0 ? 0.0 : gap; // a NaN stays
                g = gap <= 0.0 ? 0.0 : -p.beta;
            } else {
                const double h = p.beta * d, u = row_exp(-fabs(h)), l = row_log1p(u);
                const double up = l + (h < 0.0 ? -h : 0.0), down = l + (h > 0.0 ? h : 0.0);
                L = (1.0 - p.eps) * up + (p.eps != 0.0 ? p.eps * down : 0.0);
                const double sig = h >= 0.0 ? 1.0 / (1.0 + u) : u / (1.0 + u);
                const double com = h >= 0.0 ? u / (1.0 + u) : 1.0 / (1.0 + u);
                g = p.beta * (p.eps * sig - (1.0 - p.eps) * com);
            }
            if (w == 0.0) L = g = 0.0;
            p.loss[b] = (float)(w * L);
            if (p.logp) {
                p.logp[b] = (float)S[0];
                p.logp[b + p.pairs] = (float)S[1];
            }
            each[0] = w * g / n[0];
            each[1] = -w * g / n[1];
        }
        __syncthreads();
        if (p.grad)
            for (int c = 0; c < 2; ++c)
                for (uint64_t t = lo[c] + threadIdx.x; t < hi[c]; t += PF_NT)
                    p.slope[t] = (uint32_t)p.label[t] < p.V ? (float)each[c] : 0.f;
        __syncthreads();
    }
}

// gradient rows from the kept maximum and 1/sum: slope * (1[i = y] - q_i)
template <typename E>
__global__ __launch_bounds__(RL_NT) void pref_grad_kernel(Rows r, TokenOp op, void* grad, uint64_t ldg)
{
    for (uint64_t row = blockIdx.x; row < r.T; row += gridDim.x) {
        const E* x = static_cast<const E*>(r.x) + row * r.ld;
        E* g = static_cast<E*>(grad) + row * ldg;
        const float slope = op.slope[row];
        if (slope == 0.f) {
            zero_row(g, r.V, threadIdx.x, RL_NT);
            continue;
        }
        grad_row(x, g, r.V, RowCoef{op.m[row], -slope * op.inv[row]}, r.c, threadIdx.x, RL_NT);
        __syncthreads();
        if (threadIdx.x == 0)
            RowIO<E>::put(g + op.label[row], (float)((double)slope * -row_expm1(op.logp[row])));
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr uint64_t ROWS_PER_LAUNCH = 1u << 20; // a launch holds fewer than 2^32 threads

struct RowCheck {
    Rows r;
    unsigned grid;
};

static uint64_t row_esize(sg_dtype dt) { return dt == SG_BF16 ? 2 : 4; }

// the checks every rows call shares
static int rows_args(const void* x, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld, double inv_temp, RowCheck* out)
{
    if (dt != SG_F32 && dt != SG_BF16) return SG_EINVAL;
    if (V == 0 || V >= (1ull << 31) || T >= (1ull << 31) || ld < V || ld >= (1ull << 40)) return SG_EINVAL;
    if (!(inv_temp > 0.0) || !(inv_temp <= 1e6)) return SG_EINVAL;
    if (T > 0 && (!x || reinterpret_cast<uintptr_t>(x) % row_esize(dt) != 0)) return SG_EINVAL;
    out->r.x = x;
    out->r.T = T;
    out->r.row0 = 0;
    out->r.ld = ld;
    out->r.V = (uint32_t)V;
    out->r.it = inv_temp;
    out->r.c = (float)(inv_temp * 1.4426950408889634074); // log2(e)
    out->grid = (unsigned)(T < (1u << 20) ? T : (1u << 20));
    return SG_OK;
}

static int grad_args(const void* x, uint64_t ld, const void* grad, sg_dtype dt, uint64_t V, uint64_t ldg)
{
    if (!grad) return SG_OK;
    if (grad == x && ldg != ld) return SG_EINVAL; // in place: the same rows
    if (ldg < V || ldg >= (1ull << 40) || reinterpret_cast<uintptr_t>(grad) % row_esize(dt) != 0) return SG_EINVAL;
    return SG_OK;
}

template <typename E, int NT, int J, class Op>
static int launch_rows(const RowCheck& c, const Op& op, size_t lds, void* grad, uint64_t ldg, hipStream_t st)
{
    Rows r = c.r;
    for (r.row0 = 0; r.row0 < r.T; r.row0 += ROWS_PER_LAUNCH) {
        const uint64_t left = r.T - r.row0;
        const unsigned grid = (unsigned)(left < ROWS_PER_LAUNCH ? left : ROWS_PER_LAUNCH);
        if constexpr (Op::kGrad)
            if (grad) row_loss_kernel<E, NT, J, Op, true><<<grid, NT, lds, st>>>(r, op, grad, ldg);
        if (!grad) row_loss_kernel<E, NT, 4, Op, false><<<grid, NT, lds, st>>>(r, op, grad, ldg);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}

template <typename E, class Op>
static int launch_row_loss_of(const RowCheck& c, const Op& op, size_t lds, void* grad, uint64_t ldg, hipStream_t st)
{
    const uint64_t bytes = (uint64_t)c.r.V * sizeof(E);
    if (bytes <= 256 * 8 * 16) return launch_rows<E, 256, 8>(c, op, lds, grad, ldg, st);
    if (bytes <= 512 * 16 * 16) return launch_rows<E, 512, 16>(c, op, lds, grad, ldg, st);
    return launch_rows<E, 1024, 16>(c, op, lds, grad, ldg, st);
}

template <class Op>
static int launch_row_loss(const RowCheck& c, sg_dtype dt, const Op& op, size_t lds, void* grad, uint64_t ldg,
                           hipStream_t st)
{
    if (dt == SG_BF16) return launch_row_loss_of<bf16_bits>(c, op, lds, grad, ldg, st);
    return launch_row_loss_of<float>(c, op, lds, grad, ldg, st);
}

} // namespace sg

using namespace sg;

extern "C" size_t sg_distill_workspace_bytes(uint64_t T, uint64_t V, uint32_t k, sg_dtype dt) { return 0; }

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
    if (k > SG_ROWS_MAX_K || V > 14 * 32768u) return SG_EUNSUPPORTED;
    if (T == 0) return SG_OK;
    DistillOp op = {d_idx, d_logp, d_weight, d_loss, k, (uint32_t)V, (int)mode};
    return launch_row_loss(c, dt, op, ceil_div(V + 8, 32) * 4, d_grad, ld_grad, as_stream(stream));
}

extern "C" size_t sg_policy_workspace_bytes(uint64_t T, uint64_t V, sg_dtype dt) { return 0; }

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
    PolicyOp op = {d_action, d_old_logp, kl_coef != 0.0 ? d_ref_logp : nullptr, d_adv, d_weight, d_loss, d_logp,
                   1.0 - clip_low, 1.0 + clip_high, kl_coef, (uint32_t)V};
    return launch_row_loss(c, dt, op, 0, d_grad, ld_grad, as_stream(stream));
}

namespace sg {
struct PrefWs {
    double* logp;
    float *m, *inv, *slope;
};
static PrefWs pref_carve(Carver& cv, uint64_t T)
{
    PrefWs w;
    w.logp = cv.take<double>(T);
    w.m = cv.take<float>(T);
    w.inv = cv.take<float>(T);
    w.slope = cv.take<float>(T);
    return w;
}
} // namespace sg

extern "C" size_t sg_preference_workspace_bytes(uint64_t T, uint64_t V, sg_dtype dt)
{
    if (T >= (1ull << 31) || V == 0 || V >= (1ull << 31)) return 0;
    Carver cv(nullptr);
    pref_carve(cv, T);
    return cv.bytes();
}

extern "C" int sg_preference_loss(const void* d_logits, sg_dtype dt, uint64_t T, uint64_t V, uint64_t ld,
                                  const int32_t* d_label, const uint64_t* d_seq_off, uint32_t pairs,
                                  const float* d_ref_logp, const float* d_weight, sg_pref_kind kind, double beta,
                                  double smoothing, int average, float* d_loss, float* d_logp, void* d_grad,
                                  uint64_t ld_grad, void* d_ws, size_t ws_bytes, void* stream)
{
    RowCheck c;
    int rc = rows_args(d_logits, dt, T, V, ld, 1.0, &c);
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
    const PrefWs w = pref_carve(cv, T);
    TokenOp op = {d_label, w.logp, w.m, w.inv, w.slope, (uint32_t)V};
    if (T > 0 && (rc = launch_row_loss(c, dt, op, 0, nullptr, 0, st))) return rc;
    if (pairs > 0) {
        PairArgs p = {d_seq_off, d_ref_logp, d_weight, d_label, w.logp, w.slope, d_loss, d_logp, T, pairs,
                      (uint32_t)V, (int)kind, average ? 1 : 0, d_grad ? 1 : 0, beta, smoothing};
        pref_pair_kernel<<<pairs < 65536u ? pairs : 65536u, PF_NT, 0, st>>>(p);
        SG_TRY_LAUNCH();
    }
    if (T > 0 && d_grad) {
        if (dt == SG_BF16) pref_grad_kernel<bf16_bits><<<c.grid, RL_NT, 0, st>>>(c.r, op, d_grad, ld_grad);
        else pref_grad_kernel<float><<<c.grid, RL_NT, 0, st>>>(c.r, op, d_grad, ld_grad);
        SG_TRY_LAUNCH();
    }
    return SG_OK;
}
