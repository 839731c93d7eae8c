// Distillation from a teacher's top tokens: a divergence between the teacher's probabilities on a
// row's support and the student's, from the student's logits, with its gradient.
//
// Outcomes o: the support's tokens and, with `tail`, the rest of the vocabulary as one more.  With p
// the teacher's and P = softmax(z / T) the student's probabilities,
//   L = sum_o f(p_o, P_o),      dL/dz_j = P_j / T (g_o(j) - A),   A = sum_o P_o g_o,   g_o = df/dP_o
//   forward  f = p ln(p / P)                                 g = -p / P
//   reverse  f = P ln(P / p)                                 g = ln(P / p) (+ 1, which cancels)
//   jsd      f = b p ln(p / m) + (1 - b) P ln(P / m),  m = b p + (1 - b) P,     g = (1 - b) ln(P / m)
// All tokens outside the support have the g of the rest (0 without a tail), so the gradient is one
// factor times their softmax, and the support's entries are put in after.
//
// One kernel, a cluster of blocks a row: each block brings its slice of the row into shared memory by one
// bulk copy, while it works through the row's support (few entries, every block of the cluster does them all);
// takes the support out of the slice (-inf), so that the rest's sum is a sum and not a difference of nearly equal ones;
// then the cluster exchanges (maximum, sum) of its slices, and each block turns its slice into the gradient
// in place and sends it off by one bulk copy.  So logits are read once and gradients written once.
//
// A divergence is a small difference of the outcomes' terms: they are carried as pairs of floats (2^-44), with
// the rest's sum of fp32 exponentials the only fp32 part; an error of it moves L in second order
// only, since all probabilities are divided by the same total.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ff.cuh"
#include "internal.h"

namespace rl {

constexpr int kDistThreads = 256;
constexpr int kDistWarps = kDistThreads / 32;
constexpr float kMinTail = 0x1p-20f;            // what fp32 log-probabilities leave certain of a teacher's rest

struct DistArgs {
    rl_distill_args a;
    int32_t* status;
    FF inv_t;              // 1 / T
    float c;               // log2(e) / T
    int cs;                // blocks a row
    int slice;             // elements of a slice, a multiple of 32 bytes
    bool grad;             // fwd_bwd: gradients too
    uint64_t wait_ns;
};

// What the forward leaves for the backward.
struct DistSaved {
    float* M;              // [N] the row's largest logit
    float* rest;           // [N] d L / d z of a token outside the support over its exp((z - M) / T)
    float* entry;          // [nnz] d L / d z of the support's entries
};
static DistSaved dist_saved(void* base, int64_t N, int64_t nnz, size_t* bytes) {
    Carve c(base);
    DistSaved s;
    s.M = c.take<float>(static_cast<size_t>(N));
    s.rest = c.take<float>(static_cast<size_t>(N));
    s.entry = c.take<float>(static_cast<size_t>(nnz));
    if (bytes) *bytes = align_up(c.off, 256);
    return s;
}

RL_DEVINL float to_f32(float x) { return x; }
RL_DEVINL float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
RL_DEVINL float to_f32(__half x) { return __half2float(x); }
template <typename T>
RL_DEVINL T from_f32(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
    else return __float2bfloat16_rn(x);
}

// 16 bytes of logits
template <typename T>
struct Pack {
    static constexpr int E = 16 / sizeof(T);
    T t[E];
    RL_DEVINL void load(const void* p) {
        const uint4 q = *static_cast<const uint4*>(p);
        memcpy(t, &q, 16);
    }
    RL_DEVINL void store(void* p) const {
        uint4 q;
        memcpy(&q, t, 16);
        *static_cast<uint4*>(p) = q;
    }
};

RL_DEVINL FF warp_sum_ff(FF v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = ff_add(v, {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
    return v;
}

struct DistShared {
    uint64_t bar;
    float2 part;                 // (maximum, sum) of the block's slice without the support
    FF red[kDistWarps][2];
    float redf[kDistWarps][2];
};

// Block sums of two pairs, in a fixed order; every thread gets them.
RL_DEVINL void block_sum2(DistShared& s, FF& a, FF& b) {
    a = warp_sum_ff(a);
    b = warp_sum_ff(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        s.red[threadIdx.x >> 5][0] = a;
        s.red[threadIdx.x >> 5][1] = b;
    }
    __syncthreads();
    a = s.red[0][0];
    b = s.red[0][1];
#pragma unroll
    for (int w = 1; w < kDistWarps; ++w) {
        a = ff_add(a, s.red[w][0]);
        b = ff_add(b, s.red[w][1]);
    }
}
RL_DEVINL void block_max2(DistShared& s, float& a, float& b) {
    a = warp_max(a);
    b = warp_max(b);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        s.redf[threadIdx.x >> 5][0] = a;
        s.redf[threadIdx.x >> 5][1] = b;
    }
    __syncthreads();
    a = s.redf[0][0];
    b = s.redf[0][1];
#pragma unroll
    for (int w = 1; w < kDistWarps; ++w) {
        a = fmaxf(a, s.redf[w][0]);
        b = fmaxf(b, s.redf[w][1]);
    }
}

RL_DEVINL float2 cluster_read(const float2* mine, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr(mine, rank)) : "memory");
    return v;
}
RL_DEVINL void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
                 "r"(smem_addr(src)), "r"(bytes)
                 : "memory");
}

// One support entry of a row.
struct Entry {
    int id;
    float z, lq;
    bool in;               // it counts: a token of the vocabulary with a log-probability above -inf
};
// Its terms: P, f and P g.
struct Term {
    FF P, f, g;
    bool inf;              // f is infinite (and 0 here: pairs hold finite numbers)
};

// f and P g of an outcome with logs lt = ln p and lp = ln P (-inf: P is 0).
RL_DEVINL Term term_of(int kind, float beta, FF t, FF lt, FF P, FF lp) {
    Term r;
    r.P = P;
    r.inf = false;
    const bool none = lp.hi == -INFINITY;          // (NaN goes on)
    if (kind == RL_DISTILL_FORWARD) {
        // (a token that the teacher wants and the student cannot give makes the row's loss infinite)
        r.inf = none && t.hi > 0.f;
        r.f = t.hi > 0.f && !none ? ff_mul(t, ff_add(lt, ff_neg(lp))) : FF{0.f, 0.f};
        r.g = ff_neg(t);
    } else if (kind == RL_DISTILL_REVERSE) {
        r.f = none ? FF{0.f, 0.f} : ff_mul(P, ff_add(lp, ff_neg(lt)));
        r.g = r.f;
    } else {
        const FF b = {beta, 0.f}, a = two_sum(1.f, -beta);
        const FF m = ff_add(ff_mul(b, t), ff_mul(a, P));
        r.f = r.g = {0.f, 0.f};
        if (m.hi != 0.f) {
            const FF lm = ln_pair(m);
            if (t.hi > 0.f) r.f = ff_mul(ff_mul(b, t), ff_add(lt, ff_neg(lm)));
            if (!none) r.g = ff_mul(ff_mul(a, P), ff_add(lp, ff_neg(lm)));
            r.f = ff_add(r.f, r.g);
        }
    }
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kDistThreads) distill_kernel(const DistArgs p, const DistSaved sv) {
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ DistShared s;
    const rl_distill_args& a = p.a;
    constexpr int E = Pack<T>::E;
    const int tid = threadIdx.x;
    const long long row = blockIdx.x / static_cast<unsigned>(p.cs);
    const int rank = static_cast<int>(blockIdx.x - row * p.cs);
    const int V = static_cast<int>(a.V);
    const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
    // Places: the row's element i lies at place i + phase, so that a multiple of E places is 16-byte
    // aligned in memory and in shared memory alike.  This block has places [q0, q0 + slice).
    const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const long long q0 = static_cast<long long>(rank) * p.slice;
    const int i0 = static_cast<int>(max(q0 - phase, 0ll)), i1 = static_cast<int>(min(max(q0 + p.slice - phase, 0ll), static_cast<long long>(V)));
    const int n = max(i1 - i0, 0);                               // the slice's elements
    const int l0 = static_cast<int>(i0 + phase - q0), l1 = l0 + n;     // their places in shared memory
    const int b0 = (l0 + E - 1) / E * E, b1 = l1 / E * E;        // the aligned stretch of them
    const int packs = n > 0 ? (l1 + E - 1) / E : 0;
    T* buf = reinterpret_cast<T*>(raw);
    int bits = 0;

    long long eb = a.offsets[row], ee = a.offsets[row + 1];
    if (eb < 0 || ee < eb || ee > a.nnz) {
        bits |= RL_STATUS_OFFSETS;
        eb = ee = 0;
    }
    const float w = a.dloss && p.grad ? a.dloss[row] : 0.f;
    if (tid == 0) {
        mbar_init(&s.bar, 1);
        fence_mbar_init();
        if (n > 0 && b1 > b0) {
            mbar_arrive_expect_tx(&s.bar, static_cast<uint32_t>((b1 - b0) * sizeof(T)));
            bulk_load(buf + b0, z + (b0 - l0 + i0), static_cast<uint32_t>((b1 - b0) * sizeof(T)), &s.bar);
        } else {
            mbar_arrive(&s.bar);
        }
    }
    // the edges by themselves; places that are not the row's hold -inf
    const int lead = b1 > b0 ? b0 : packs * E, trail = b1 > b0 ? b1 : packs * E;
    auto edge = [&](int q) { buf[q] = q >= l0 && q < l1 ? z[q - l0 + i0] : from_f32<T>(-INFINITY); };
    for (int q = tid; q < lead; q += kDistThreads) edge(q);
    for (int q = trail + tid; q < packs * E; q += kDistThreads) edge(q);

    // ---- the support, while the slice is on its way
    auto entry_at = [&](long long e) -> Entry {
        Entry x;
        x.id = a.ids[e];
        x.lq = a.logq[e];
        x.in = x.id >= 0 && x.id < V && x.lq > -INFINITY && x.lq < INFINITY;
        x.z = x.in ? to_f32(z[x.id]) : -INFINITY;
        return x;
    };
    Entry first{-1, -INFINITY, 0.f, false};
    float mS = -INFINITY, mT = -INFINITY;
    for (long long e = eb + tid; e < ee; e += kDistThreads) {
        const Entry x = entry_at(e);
        if (e == eb + tid) first = x;
        if (x.id < 0 || x.id >= V) bits |= RL_STATUS_ID_RANGE;
        if (!(x.lq < INFINITY) || (a.tail && x.lq > 1e-6f)) bits |= RL_STATUS_LOGQ;
        if (e > eb && x.id <= a.ids[e - 1]) bits |= RL_STATUS_ROW_ORDER;
        if (x.in) {
            mS = fmaxf(mS, x.z);
            mT = fmaxf(mT, x.lq);
        }
    }
    block_max2(s, mS, mT);
    const bool any = mT > -INFINITY;             // the row has a teacher
    // f(entry, its index) for the entries that count; the thread's first is in registers
    auto each = [&](auto f) {
        for (long long e = eb + tid; e < ee; e += kDistThreads) {
            const Entry x = e == eb + tid ? first : entry_at(e);
            if (x.in) f(x, e);
        }
    };
    // (z - m) / T
    auto scaled = [&](float v, float m) -> FF { return v == -INFINITY ? FF{-INFINITY, 0.f} : ff_mul(two_sum(v, -m), p.inv_t); };
    FF wS = {0.f, 0.f}, wT = {0.f, 0.f};
    if (any) {
        each([&](const Entry& x, long long) {
            if (mS > -INFINITY) wS = ff_add(wS, exp_pair(scaled(x.z, mS)));
            wT = ff_add(wT, a.tail ? exp_ff(x.lq) : exp_pair(scaled(x.lq, mT)));
        });
        block_sum2(s, wS, wT);
    }
    if (!mbar_wait(&s.bar, 0, p.status, p.wait_ns)) mbar_wait(&s.bar, 0, p.status);   // (the copy lands before the block goes on)
    __syncthreads();
    // ---- the rest of the slice
    if (any)
        for (long long e = eb + tid; e < ee; e += kDistThreads) {
            const Entry x = e == eb + tid ? first : entry_at(e);
            if (x.in && x.id >= i0 && x.id < i1) buf[x.id - i0 + l0] = from_f32<T>(-INFINITY);
        }
    __syncthreads();
    float m = -INFINITY, unused = 0.f;
    for (int k = tid; k < packs; k += kDistThreads) {
        Pack<T> v;
        v.load(buf + k * E);
#pragma unroll
        for (int j = 0; j < E; ++j) m = fmaxf(m, to_f32(v.t[j]));
    }
    block_max2(s, m, unused);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    const float mc = m > -INFINITY ? m : 0.f;
    for (int k = tid; k < packs; k += kDistThreads) {
        Pack<T> v;
        v.load(buf + k * E);
#pragma unroll
        for (int j = 0; j < E; ++j) sum[j & 3] += exp2_approx((to_f32(v.t[j]) - mc) * p.c);
    }
    {
        FF t = ff_add(two_sum(sum[0], sum[1]), two_sum(sum[2], sum[3])), none = {0.f, 0.f};
        block_sum2(s, t, none);
        if (tid == 0) s.part = make_float2(m, t.hi + t.lo);
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    float M = mS;
    for (int k = 0; k < p.cs; ++k) M = fmaxf(M, cluster_read(&s.part, k).x);
    float rest = 0.f;
    for (int k = 0; k < p.cs; ++k) {
        const float2 v = cluster_read(&s.part, k);
        rest += v.x > -INFINITY ? v.y * exp2f((v.x - M) * p.c) : v.y;      // (a sum without a maximum is 0 or NaN)
    }
    // ---- the outcomes
    FF loss = {0.f, 0.f}, A = {0.f, 0.f}, P0 = {0.f, 0.f}, g0 = {0.f, 0.f};
    FF lnT = {0.f, 0.f}, lnW = {0.f, 0.f};
    float k_rest = 0.f;                                 // the gradient's factor outside the support, times T
    float mass = 0.f;
    int infinite = 0;
    auto terms = [&](const Entry& x) -> Term {
        const FF X = scaled(x.z, M);
        const FF lp = X.hi == -INFINITY ? X : ff_add(X, ff_neg(lnT));
        FF t, lt;
        if (a.tail) {
            t = exp_ff(x.lq);
            lt = {x.lq, 0.f};
        } else {
            lt = ff_add(scaled(x.lq, mT), ff_neg(lnW));
            t = exp_pair(lt);
        }
        return term_of(a.kind, a.beta, t, lt, exp_pair(lp), lp);
    };
    if (any) {
        const FF held = mS > -INFINITY ? ff_mul(wS, exp_pair(scaled(mS, M))) : FF{0.f, 0.f};
        const FF total = ff_add({rest, 0.f}, held);
        lnT = ln_pair(total);
        if (!a.tail) lnW = ln_pair(wT);
        bool inf = false;
        each([&](const Entry& x, long long) {
            const Term t = terms(x);
            loss = ff_add(loss, t.f);
            A = ff_add(A, t.g);
            inf |= t.inf;
        });
        block_sum2(s, loss, A);
        infinite = __syncthreads_or(inf);
        P0 = ff_div({rest, 0.f}, total);
        if (a.tail && rest > 0.f) {
            FF t0 = ff_add({1.f, 0.f}, ff_neg(wT));
            if (!(t0.hi >= kMinTail)) t0 = {kMinTail, 0.f};
            const Term t = term_of(a.kind, a.beta, t0, ln_pair(t0), P0, ln_pair(P0));
            loss = ff_add(loss, t.f);
            A = ff_add(A, t.g);
            g0 = t.g;
        }
        // g of the rest less A, over the total
        const FF d = ff_add(rest > 0.f ? ff_div(g0, P0) : FF{0.f, 0.f}, ff_neg(A));
        k_rest = (d.hi + d.lo) / (total.hi + total.lo);
        mass = (held.hi + held.lo) / (total.hi + total.lo);
        if (infinite || !(fabsf(loss.hi) < INFINITY) || !(total.hi > 0.f)) bits |= RL_STATUS_NONFINITE;
    }
    const float l = infinite && loss.hi == loss.hi ? INFINITY : loss.hi + loss.lo;
    if (rank == 0 && tid == 0) {
        if (a.loss) a.loss[row] = l;
        if (a.mass) a.mass[row] = mass;
    }
    const float inv_T = p.inv_t.hi;
    if (!p.grad) {
        if (sv.M) {
            if (rank == 0 && tid == 0) {
                sv.M[row] = M;
                sv.rest[row] = any ? k_rest * inv_T : 0.f;
            }
            if (rank == 0)
                for (long long e = eb + tid; e < ee; e += kDistThreads) {
                    const Entry x = e == eb + tid ? first : entry_at(e);
                    float d = 0.f;
                    if (x.in) {
                        const Term t = terms(x);
                        const FF v = ff_add(t.g, ff_neg(ff_mul(t.P, A)));
                        d = (v.hi + v.lo) * inv_T;
                    }
                    sv.entry[e] = d;
                }
        }
        set_status(p.status, bits);
        __syncthreads();
        cluster_arrive();                       // nobody leaves while its part may be read
        cluster_wait();
        return;
    }
    // ---- the gradient, in place
    const float kr = any ? w * inv_T * k_rest : 0.f;
    const bool zero = !any || w == 0.f;
    for (int k = tid; k < packs; k += kDistThreads) {
        Pack<T> v;
        v.load(buf + k * E);
#pragma unroll
        for (int j = 0; j < E; ++j) v.t[j] = from_f32<T>(zero ? 0.f : kr * exp2_approx((to_f32(v.t[j]) - M) * p.c));
        v.store(buf + k * E);
    }
    __syncthreads();
    if (!zero)
        each([&](const Entry& x, long long) {
            if (x.id < i0 || x.id >= i1) return;
            const Term t = terms(x);
            const FF v = ff_add(t.g, ff_neg(ff_mul(t.P, A)));
            buf[x.id - i0 + l0] = from_f32<T>(w * inv_T * (v.hi + v.lo));
        });
    set_status(p.status, bits);
    fence_proxy_async_smem();
    __syncthreads();
    cluster_arrive();                           // all of the row's logits have been read: the gradient may take their place
    cluster_wait();
    T* d = static_cast<T*>(a.dlogits) + row * a.grad_stride;
    const bool same = (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == static_cast<unsigned>(phase);
    if (same) {
        if (tid == 0 && b1 > b0) {
            bulk_store(d + (b0 - l0 + i0), buf + b0, static_cast<uint32_t>((b1 - b0) * sizeof(T)));
            bulk_commit();
        }
        for (int q = l0 + tid; q < min(lead, l1); q += kDistThreads) d[q - l0 + i0] = buf[q];
        for (int q = trail + tid; q < l1; q += kDistThreads) d[q - l0 + i0] = buf[q];
        if (tid == 0) bulk_wait_read<0>();
    } else {
        for (int q = l0 + tid; q < l1; q += kDistThreads) d[q - l0 + i0] = buf[q];
    }
}

// ---- the backward alone: gradients from what the forward saved --------------------------------
constexpr int kBwdThreads = 256;
constexpr int kBwdStep = 4096;                  // elements of a block

template <typename T>
__global__ void __launch_bounds__(kBwdThreads) distill_bwd_kernel(const DistArgs p, const DistSaved sv) {
    const rl_distill_args& a = p.a;
    constexpr int E = Pack<T>::E;
    const long long row = blockIdx.x;
    const int V = static_cast<int>(a.V);
    const int i0 = static_cast<int>(blockIdx.y) * kBwdStep, i1 = min(i0 + kBwdStep, V);
    const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
    T* d = static_cast<T*>(a.dlogits) + row * a.grad_stride;
    const float w = a.dloss[row], M = sv.M[row];
    long long eb = a.offsets[row], ee = a.offsets[row + 1];
    if (eb < 0 || ee < eb || ee > a.nnz) eb = ee = 0;
    const bool zero = w == 0.f || eb == ee;
    const float k = zero ? 0.f : w * sv.rest[row];
    const bool vec = ((reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(d)) & 15) == 0;
    const int packed = vec ? (i1 - i0) / E : 0;
    for (int q = threadIdx.x; q < packed; q += kBwdThreads) {
        Pack<T> v;
        v.load(z + i0 + q * E);
#pragma unroll
        for (int j = 0; j < E; ++j) v.t[j] = from_f32<T>(k == 0.f ? 0.f : k * exp2_approx((to_f32(v.t[j]) - M) * p.c));
        v.store(d + i0 + q * E);
    }
    for (int i = i0 + packed * E + threadIdx.x; i < i1; i += kBwdThreads)
        d[i] = from_f32<T>(k == 0.f ? 0.f : k * exp2_approx((to_f32(z[i]) - M) * p.c));
    if (zero) return;
    __syncthreads();
    long long lo = eb, hi = ee;                 // first entry with id >= i0
    while (lo < hi) {
        const long long mid = (lo + hi) >> 1;
        if (a.ids[mid] < i0) lo = mid + 1;
        else hi = mid;
    }
    for (long long e = lo + threadIdx.x; e < ee; e += kBwdThreads) {
        const int id = a.ids[e];
        if (id >= i1) break;
        if (id < i0 || !(a.logq[e] > -INFINITY && a.logq[e] < INFINITY)) continue;
        d[id] = from_f32<T>(w * sv.entry[e]);
    }
}

// ---- host ----------------------------------------------------------------------------------
static DistArgs dist_args(const rl_distill_args* a, int32_t* status) {
    DistArgs p;
    p.a = *a;
    p.status = status;
    const double inv = 1.0 / static_cast<double>(a->temperature);
    p.inv_t.hi = static_cast<float>(inv);
    p.inv_t.lo = static_cast<float>(inv - static_cast<double>(p.inv_t.hi));
    p.c = static_cast<float>(1.4426950408889634074 * inv);
    p.wait_ns = wait_limit_ns();
    return p;
}

constexpr int kSliceTarget = 40 * 1024;         // bytes: five blocks a multiprocessor, whose loads, sums and stores overlap
constexpr int kSliceLeast = 4 * 1024;
static_assert(kDistillRowBytes <= 8 * (kDistillSliceBytes - 64), "a cluster of eight holds the longest row");

template <typename T>
static int distill_run(DistArgs p, const DistSaved& sv, cudaStream_t stream) {
    const long long bytes = p.a.V * static_cast<long long>(sizeof(T));
    // the fewest blocks a row whose slices leave room for others on the multiprocessor; more of them where
    // there are too few rows to fill the GPU
    int cs = 1;
    while (cs < 8 && (bytes / cs > kSliceTarget || (p.a.N * cs < num_sms() && bytes / cs >= 2 * kSliceLeast))) cs *= 2;
    const int quantum = 32 / static_cast<int>(sizeof(T));
    p.cs = cs;
    p.slice = static_cast<int>(((p.a.V + 16 / sizeof(T)) + cs * quantum - 1) / (cs * quantum)) * quantum;
    if (p.a.N * cs >= (1ll << 31)) {
        set_last_error("too many rows");
        return RL_ERR_UNSUPPORTED;
    }
    const int smem = p.slice * static_cast<int>(sizeof(T));
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(distill_kernel<T>, kDistillSliceBytes, done)) return RL_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.N * cs), 1, 1);
    cfg.blockDim = dim3(kDistThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ProfScope prof(RL_PROF_OTHER, stream);
    if (cudaLaunchKernelEx(&cfg, distill_kernel<T>, p, sv) != cudaSuccess) return RL_ERR_CUDA;
    count_launch();
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <typename T>
static int distill_bwd_run(const DistArgs& p, const DistSaved& sv, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.a.N), static_cast<unsigned>((p.a.V + kBwdStep - 1) / kBwdStep), 1);
    ProfScope prof(RL_PROF_OTHER, stream);
    distill_bwd_kernel<T><<<grid, kBwdThreads, 0, stream>>>(p, sv);
    count_launch();
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

size_t distill_saved_bytes(int64_t N, int64_t nnz) {
    size_t b = 0;
    dist_saved(nullptr, N, nnz, &b);
    return b;
}

int distill_impl(const rl_distill_args* a, int pass, void* saved, int32_t* status, cudaStream_t stream) {
    if (a->N == 0) return RL_OK;
    DistArgs p = dist_args(a, status);
    p.grad = pass == kDistillBoth;
    DistSaved sv{nullptr, nullptr, nullptr};
    if (saved) sv = dist_saved(saved, a->N, a->nnz, nullptr);
    if (pass == kDistillBwd)
        return a->dtype == RL_DTYPE_F32 ? distill_bwd_run<float>(p, sv, stream)
               : a->dtype == RL_DTYPE_BF16 ? distill_bwd_run<__nv_bfloat16>(p, sv, stream) : distill_bwd_run<__half>(p, sv, stream);
    return a->dtype == RL_DTYPE_F32 ? distill_run<float>(p, sv, stream)
           : a->dtype == RL_DTYPE_BF16 ? distill_run<__nv_bfloat16>(p, sv, stream) : distill_run<__half>(p, sv, stream);
}

}  // namespace rl
