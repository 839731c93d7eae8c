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
// takes the support out of the slice (-inf), so that the rest's sum is a sum and not a difference of nearly equal ones,
// kept relative to the rest's own largest logit where that lies far below the support's;
// then the blocks send each other (reference, sum) of their slices, and each block turns its slice into the gradient
// in place and sends it off by one bulk copy.  So logits are read once and gradients written once.
//
// HBM bounds it for long rows: 4096 bf16 rows of 151,936 logits 411 us (89 % of a copy's rate), 2048 fp32 rows 431 us with a rest
// and up to 128 entries (85 %), 387 us without (95 %).  Each row waits for its support and its cluster; slices of
// 75 KB leave room for three blocks on a multiprocessor, whose loads, sums and stores fill one another's waits.  The forward
// alone, whose blocks store nothing, is at 70 % (260 us): their loads do not follow one another closely enough.
//
// A divergence is a small difference of the outcomes' terms: a second kernel takes it in pairs of floats (2^-38), with
// the rest's sum of fp32 exponentials the only fp32 part; an error of it moves L in second order
// only, since all probabilities are divided by the same total.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ff.cuh"
#include "internal.h"
#include "weights.cuh"

namespace rl {

constexpr int kDistWarps = 8;                   // most of a block
constexpr float kMinTail = 0x1p-20f;            // what fp32 log-probabilities leave certain of a teacher's rest
constexpr float kRestGone = -745.f;             // ln of a ratio to the row's largest weight below which the rest is no outcome (0 in 64 bits)

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

// What the pass over the logits leaves for the loss and for the backward.
struct DistSaved {
    float* M;              // [N] the row's reference logit
    float* ref;            // [N] the reference logit of what is outside the support (-inf: nothing is)
    float* sum;            // [N] sum of e^((z - ref) / T) there
    float* z;              // [nnz] the support's logits
    float* rest;           // [N] d L / d z of a token outside the support over its exp((z - ref) / T)
    float* entry;          // [nnz] d L / d z of the support's entries
};
static DistSaved dist_saved(void* base, int64_t N, int64_t nnz, size_t* bytes) {
    Carve c(base);
    DistSaved s;
    s.M = c.take<float>(static_cast<size_t>(N));
    s.ref = c.take<float>(static_cast<size_t>(N));
    s.sum = c.take<float>(static_cast<size_t>(N));
    s.z = c.take<float>(static_cast<size_t>(nnz));
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
    // the largest that is a number (16-bit types two at a time)
    RL_DEVINL float largest() const {
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
        } else if constexpr (std::is_same<T, __half>::value) {
            __half2 h[4];
            memcpy(h, t, 16);
            const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            __nv_bfloat162 h[4];
            memcpy(h, t, 16);
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    RL_DEVINL void put(const float (&x)[E]) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int j = 0; j < E; ++j) t[j] = x[j];
        } else {
#pragma unroll
            for (int j = 0; j < E; j += 2) {
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(x[j], x[j + 1]);
                    memcpy(t + j, &h, 4);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[j], x[j + 1]);
                    memcpy(t + j, &h, 4);
                }
            }
        }
    }
};

// (low parts are added up as they are, and the pair put in order at the end)
RL_DEVINL FF warp_sum_ff(FF v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const FF x = two_sum(v.hi, __shfl_xor_sync(0xffffffffu, v.hi, o));
        v = {x.hi, x.lo + (v.lo + __shfl_xor_sync(0xffffffffu, v.lo, o))};
    }
    return fast_two_sum(v.hi, v.lo);
}

struct DistShared {              // (small: three blocks with slices of 76 KB are to fit on a multiprocessor)
    uint64_t bar, xbar;          // the slice has landed; the parts of the row's blocks have
    float2 xpart[8];             // (reference, sum) of each block of the cluster, without the support
    float2 part[kDistWarps];     // of each warp of this block
    float4 sup[kDistWarps];      // of each support warp: largest logit, largest of the teacher's, sums relative to the block's largest
    FF sum[kDistWarps];          // pairs to be added up over the support warps
    float A[kDistWarps];
    float rest_ref;              // of the rest: reference logit,
    float unit, x0, g0;          // the probability of a weight of 1 in the sum, P g, and P g over the sum
};

// v into another block's `to`, counted by its barrier `bar` (both given by this block's own addresses).
RL_DEVINL void cluster_send(float2 v, const float2* to, const uint64_t* bar, int rank) {
    const unsigned long long x = static_cast<unsigned long long>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x);
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(cluster_addr(to, rank)), "l"(x),
                 "r"(cluster_addr(bar, rank))
                 : "memory");
}
// Largest of a warp's values (NaN is not looked at).
RL_DEVINL float warp_largest(float v) { return z_of(__reduce_max_sync(0xffffffffu, key_of(v + 0.f))); }
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
template <typename T>
RL_DEVINL Entry entry_of(const rl_distill_args& a, const T* z, long long e) {
    Entry x;
    x.id = a.ids[e];
    x.lq = a.logq[e];
    x.in = x.id >= 0 && x.id < a.V && x.lq > -INFINITY && x.lq < INFINITY;
    x.z = x.in ? to_f32(z[x.id]) : -INFINITY;
    return x;
}
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
            const FF lm = ln_table(m);
            if (t.hi > 0.f) r.f = ff_mul(ff_mul(b, t), ff_add(lt, ff_neg(lm)));
            if (!none) r.g = ff_mul(ff_mul(a, P), ff_add(lp, ff_neg(lm)));
            r.f = ff_add(r.f, r.g);
        }
    }
    return r;
}

// P g of an outcome in fp32, for gradients.
RL_DEVINL float slope_of(int kind, float beta, float t, float lt, float P, float lp) {
    if (kind == RL_DISTILL_FORWARD) return -t;
    if (lp == -INFINITY) return 0.f;
    if (kind == RL_DISTILL_REVERSE) return P * (lp - lt);
    const float a = 1.f - beta, m = fmaf(beta, t, a * P);
    return m != 0.f ? a * P * (lp - logf(m)) : 0.f;          // (both of them underflow: NaN goes on)
}
// Sum of v over the first n warps' threads (they alone call it), as a pair in every lane.
RL_DEVINL FF support_sum(FF* part, FF v, int n) {
    v = warp_sum_ff(v);
    if (n == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    asm volatile("bar.sync 1, %0;" ::"r"(n * 32) : "memory");
    v = part[0];
    for (int w = 1; w < n; ++w) v = ff_add(v, part[w]);
    return v;
}
RL_DEVINL FF rest_of(FF held) {                  // the teacher's probability of the rest
    const FF t0 = ff_add({1.f, 0.f}, ff_neg(held));
    return t0.hi >= kMinTail ? t0 : FF{kMinTail, 0.f};
}

template <typename T, int NT, int kBlocks>
__global__ void __launch_bounds__(NT, kBlocks) distill_kernel(const __grid_constant__ DistArgs p, const DistSaved sv) {
    extern __shared__ __align__(128) uint8_t raw[];
    __shared__ DistShared s;
    const rl_distill_args& a = p.a;
    constexpr int E = Pack<T>::E, kWarps = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / static_cast<unsigned>(p.cs);
    const int rank = static_cast<int>(blockIdx.x - row * p.cs);
    const int V = static_cast<int>(a.V);
    long long eb = a.offsets[row], ee = a.offsets[row + 1];
    const float w = a.dloss && p.grad ? a.dloss[row] : 0.f;
    const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
    // Places: the row's element i lies at place i + phase, so that a multiple of E places is 16-byte
    // aligned in memory and in shared memory alike.  This block has places [q0, q0 + slice), of which [l0, l1) are
    // the row's and [b0, b1) whole 16 bytes of it.
    const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const long long q0 = static_cast<long long>(rank) * p.slice;
    const int i0 = static_cast<int>(max(q0 - phase, 0ll)), i1 = static_cast<int>(min(max(q0 + p.slice - phase, 0ll), static_cast<long long>(V)));
    const int n = max(i1 - i0, 0);
    const int l0 = static_cast<int>(i0 + phase - q0), l1 = l0 + n;
    const int b0 = (l0 + E - 1) / E * E, b1 = max(l1 / E * E, b0);
    const int at0 = i0 - l0;                                     // place q holds the row's element q + at0
    const int packs = n > 0 ? (l1 + E - 1) / E : 0;
    T* buf = reinterpret_cast<T*>(raw);
    int bits = 0;

    let_next_start();
    if (tid == NT - 1) {
        mbar_init(&s.bar, 1);
        mbar_init(&s.xbar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&s.xbar, static_cast<uint32_t>(p.cs) * 8u);
        if (b1 > b0) {
            mbar_arrive_expect_tx(&s.bar, static_cast<uint32_t>((b1 - b0) * sizeof(T)));
            bulk_load(buf + b0, z + b0 + at0, static_cast<uint32_t>((b1 - b0) * sizeof(T)), &s.bar);
        } else {
            mbar_arrive(&s.bar);
        }
    }
    __syncwarp();
    cluster_arrive_relaxed();                    // the barriers are there (fence_mbar_init is their release)
    // the places that the copy leaves out: the row's edges, and -inf beside them
    auto edges = [&](auto f) {
        for (int q = tid; q < min(packs * E, b0); q += NT) f(q);
        for (int q = b1 + tid; q < packs * E; q += NT) f(q);
    };
    edges([&](int q) { buf[q] = q >= l0 && q < l1 ? z[q + at0] : from_f32<T>(-INFINITY); });

    // ---- the support, while the slice is on its way: by as few warps as hold it, the same in every block of the cluster
    if (eb < 0 || ee < eb || ee > a.nnz) {
        bits |= RL_STATUS_OFFSETS;
        eb = ee = 0;
    }
    const int nw = static_cast<int>(min(static_cast<long long>(kWarps), (ee - eb + 31) / 32)), stride = nw * 32;
    const bool mine = warp < nw, listed = ee - eb <= NT;         // a thread has one entry at most, which stays in registers
    auto entry_at = [&](long long e) { return entry_of(a, z, e); };
    Entry first{-1, -INFINITY, 0.f, false};
    // f(entry, whether it is the thread's first, its index) for the support warps' entries that count
    auto each = [&](auto f) {
        for (long long e = eb + tid; e < ee; e += stride) {
            const bool is_first = e == eb + tid;
            const Entry x = is_first ? first : entry_at(e);
            if (x.in) f(x, is_first, e);
        }
    };
    FF wT = {0.f, 0.f};                          // tail: the teacher's probabilities of the support
    if (mine) {
        float mS = -INFINITY, mT = -INFINITY;
        for (long long e = eb + tid; e < ee; e += stride) {
            const Entry x = entry_at(e);
            if (e == eb + tid) first = x;
            if (x.id < 0 || x.id >= V) bits |= RL_STATUS_ID_RANGE;
            if (!(x.lq < INFINITY) || (a.tail && x.lq > 1e-6f)) bits |= RL_STATUS_LOGQ;
            if (e > eb && x.id <= a.ids[e - 1]) bits |= RL_STATUS_ROW_ORDER;
            if (x.in) {
                mS = fmaxf(mS, x.z);
                mT = fmaxf(mT, x.lq);
            }
            if (rank == 0) sv.z[e] = x.z;
        }
        mS = warp_largest(mS);
        mT = warp_largest(mT);
        if (lane == 0) s.sup[warp] = make_float4(mS, mT, 0.f, 0.f);
    }
    __syncthreads();
    float mS = -INFINITY, mT = -INFINITY;
    for (int k = 0; k < nw; ++k) {
        mS = fmaxf(mS, s.sup[k].x);
        mT = fmaxf(mT, s.sup[k].y);
    }
    const bool any = mT > -INFINITY;             // the row has a teacher
    if (!mbar_wait(&s.bar, 0, p.status, p.wait_ns)) mbar_wait(&s.bar, 0, p.status);   // (the copy lands before the block goes on)
    // ---- the rest of the slice: the support out of it, then each warp's maximum and sum
    if (mine)
        each([&](const Entry& x, bool, long long) {
            if (x.id >= i0 && x.id < i1) buf[x.id - at0] = from_f32<T>(-INFINITY);
        });
    __syncthreads();
    {
        // e^((z - m) / T) as 2^(z c - fl(m c)): one rounding of the argument, and the sum is put right for fl(m c) after.  The
        // reference m need not be the largest logit: the support's largest will do, unless the sum leaves the range
        float sum[4], t = 0.f, m = mS;
        auto add = [&](float pm) -> float {
            sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
            for (int k = tid; k < packs; k += NT) {
                Pack<T> v;
                v.load(buf + k * E);
#pragma unroll
                for (int j = 0; j < E; ++j) sum[j & 3] += exp2_approx(fmaf(to_f32(v.t[j]), p.c, -pm));
            }
            return warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
        };
        bool far = !(fabsf(m * p.c) < kFusedRef);
        if (!far) {
            t = add(m * p.c);
            far = !(t < 1e30f && t > 1e-25f);
        }
        if (any && far) {
            m = -INFINITY;
            for (int k = tid; k < packs; k += NT) {
                Pack<T> v;
                v.load(buf + k * E);
                m = fmaxf(m, v.largest());
            }
            m = warp_largest(m);
            if (fabsf(m * p.c) < kFusedRef) {
                t = add(m * p.c);
            } else {
                const float mc = m > -INFINITY ? m : 0.f;
                sum[0] = 0.f;
                for (int k = tid; k < packs; k += NT)
#pragma unroll 1
                    for (int j = 0; j < E; ++j) sum[0] += exp2_approx((to_f32(buf[k * E + j]) - mc) * p.c);
                t = warp_sum(sum[0]);
            }
        }
        if (fabsf(m * p.c) < kFusedRef) t *= exp2f(-fmaf(m, p.c, -(m * p.c)));
        if (lane == 0) s.part[warp] = make_float2(m, t);
    }
    // (reference, sum) of n parts, a lane each (a sum without a reference is 0 or NaN)
    auto join = [&](const float2* v, int parts) -> float2 {
        const float2 x = lane < parts ? v[lane] : make_float2(-INFINITY, 0.f);
        const float m = warp_largest(x.x);
        return make_float2(m, warp_sum(x.x > -INFINITY ? x.y * exp2f((x.x - m) * p.c) : x.y));
    };
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        const float2 v = join(s.part, kWarps);
        if (lane < p.cs) cluster_send(v, &s.xpart[rank], &s.xbar, lane);
    }
    // (while the parts are on their way) the support's sums, of the student's weights and of the teacher's
    if (mine) {
        float sS = 0.f, sT = 0.f;
        each([&](const Entry& x, bool, long long) {
            sS += x.z == -INFINITY ? 0.f : exp2f((x.z - mS) * p.c);
            if (a.tail) wT = ff_add(wT, exp_table({x.lq, 0.f}));
            else sT += exp2f((x.lq - mT) * p.c);
        });
        sS = warp_sum(sS);
        if (!a.tail) sT = warp_sum(sT);
        if (lane == 0) s.sup[warp] = make_float4(0.f, 0.f, sS, sT);
        if (a.tail) wT = support_sum(s.sum, wT, nw);
        else if (nw > 1) asm volatile("bar.sync 1, %0;" ::"r"(stride) : "memory");
        __syncwarp();
    }
    if (!mbar_wait(&s.xbar, 0, p.status, p.wait_ns)) mbar_wait(&s.xbar, 0, p.status);
    // ---- the outcomes
    // The rest stays relative to its own reference: its probability may underflow, and its share of the gradient not (the
    // forward kind's teacher wants t0 of it, however little the student gives).
    const float inv_T = p.inv_t.hi;
    float M = 0.f, total = 1.f, inv_total = 1.f, lnT = 0.f, sT = 1.f, inv_sT = 1.f, lnW = 0.f;
    // P g of an entry, and P
    auto slope = [&](const Entry& x, float& P) -> float {
        float t, lt;
        if (a.tail) {
            lt = x.lq;
            t = expf(lt);
        } else {
            lt = (x.lq - mT) * inv_T - lnW;
            t = exp2f((x.lq - mT) * p.c) * inv_sT;
        }
        const float d = x.z - M, lp = x.z == -INFINITY ? -INFINITY : d * inv_T - lnT;
        P = x.z == -INFINITY ? 0.f : exp2f(d * p.c) * inv_total;
        return slope_of(a.kind, a.beta, t, lt, P, lp);
    };
    float P1 = 0.f, g1 = 0.f;                    // of the first entry
    if (mine) {
        const float2 v = join(s.xpart, p.cs);
        M = fmaxf(v.x, mS);
        const float scale = v.x == M ? 1.f : v.y != 0.f ? exp2f((v.x - M) * p.c) : 0.f, rest = v.y * scale;
        float held = 0.f;
        sT = 0.f;
        for (int k = 0; k < nw; ++k) {
            held += s.sup[k].z;
            sT += s.sup[k].w;
        }
        if (mS > -INFINITY) held *= exp2f((mS - M) * p.c);
        total = rest + held;
        inv_total = 1.f / total;
        lnT = logf(total);
        if (!a.tail) {
            lnW = logf(sT);
            inv_sT = 1.f / sT;
        }
        float x0 = 0.f, g0 = 0.f, A = 0.f;
        const float far = (v.x - M) * inv_T;
        if (a.tail && v.y != 0.f && !(far < kRestGone)) {
            const float t0 = rest_of(wT).hi;
            x0 = slope_of(a.kind, a.beta, t0, logf(t0), rest * inv_total, far + logf(v.y) - lnT);
            g0 = x0 / v.y;
        }
        each([&](const Entry& x, bool is_first, long long) {
            float P;
            const float g = slope(x, P);
            if (is_first) {
                P1 = P;
                g1 = g;
            }
            A += g;
        });
        A = warp_sum(A);
        if (lane == 0) s.A[warp] = A;
        if (tid == 0) {
            s.rest_ref = v.x;
            s.unit = scale * inv_total;
            s.x0 = x0;
            s.g0 = g0;
            if (rank == 0) {
                sv.M[row] = M;
                sv.ref[row] = v.x;
                sv.sum[row] = v.y;
            }
        }
    }
    __syncthreads();
    // the gradient's factor outside the support (over a weight of the sum, times T), and A
    const float ref = s.rest_ref;
    float k_rest = 0.f, A = 0.f;
    if (any) {
        for (int k = 0; k < nw; ++k) A += s.A[k];
        A += s.x0;
        k_rest = s.g0 - A * s.unit;
    }
    if (!listed) {                               // (in place: its logits are read again until here)
        __syncthreads();
        cluster_arrive();
        cluster_wait();
    }
    if (!p.grad) {
        if (rank == 0) {
            if (tid == 0) {
                sv.rest[row] = any ? k_rest * inv_T : 0.f;
            }
            if (mine)
                for (long long e = eb + tid; e < ee; e += stride) {
                    const Entry x = e == eb + tid ? first : entry_at(e);
                    float P = P1, g = g1;
                    if (x.in && e != eb + tid) g = slope(x, P);
                    sv.entry[e] = x.in ? (g - P * A) * inv_T : 0.f;
                }
        }
        set_status(p.status, bits);
        return;
    }
    // ---- the gradient, in place
    const bool zero = !any || w == 0.f;
    if (zero || k_rest == 0.f) {
        for (int k = tid; k < packs; k += NT) *reinterpret_cast<uint4*>(buf + k * E) = make_uint4(0, 0, 0, 0);
    } else {
        const float kr = w * inv_T * k_rest, pm = ref * p.c;
        if (fabsf(pm) < kFusedRef) {
            const float k2 = kr * exp2f(-fmaf(ref, p.c, -pm));
            for (int k = tid; k < packs; k += NT) {
                Pack<T> v;
                v.load(buf + k * E);
                float d[E];
#pragma unroll
                for (int j = 0; j < E; ++j) d[j] = k2 * exp2_approx(fmaf(to_f32(v.t[j]), p.c, -pm));
                v.put(d);
                v.store(buf + k * E);
            }
        } else {
            for (int k = tid; k < packs; k += NT) {
                Pack<T> v;
                v.load(buf + k * E);
                float d[E];
#pragma unroll
                for (int j = 0; j < E; ++j) d[j] = kr * exp2_approx((to_f32(v.t[j]) - ref) * p.c);
                v.put(d);
                v.store(buf + k * E);
            }
        }
    }
    if (!zero) {
        __syncthreads();
        if (mine)
            each([&](const Entry& x, bool is_first, long long) {
                if (x.id < i0 || x.id >= i1) return;
                float P = P1, g = g1;
                if (!is_first) g = slope(x, P);
                buf[x.id - at0] = from_f32<T>(w * inv_T * (g - P * A));
            });
    }
    // (Every block of the row has read the support's logits: it sent its part after that.  So the gradient may take the
    // logits' place.)
    fence_proxy_async_smem();
    __syncthreads();
    T* d = static_cast<T*>(a.dlogits) + row * a.grad_stride;
    const bool same = (reinterpret_cast<uintptr_t>(d) & 15) / sizeof(T) == static_cast<unsigned>(phase);
    if (same) {
        if (tid == NT - 1 && b1 > b0) {
            bulk_store(d + b0 + at0, buf + b0, static_cast<uint32_t>((b1 - b0) * sizeof(T)));
            bulk_commit();
        }
        edges([&](int q) {
            if (q >= l0 && q < l1) d[q + at0] = buf[q];
        });
    } else {
        for (int q = l0 + tid; q < l1; q += NT) d[q + at0] = buf[q];
    }
    set_status(p.status, bits);
    if (same && tid == NT - 1) bulk_wait_read<0>();
}

// ---- the loss, in pairs of floats --------------------------------------------------------------
// A block a row, as many of its warps as hold the support.  A kernel of its own: as the last step of a row's first
// block it kept that block's slice of the multiprocessor for 9000 cycles, half as long again as the pass itself.
// Latency, so blocks on a multiprocessor count: ten of 48 registers a thread (4096 fp32 rows of 1000 logits, both kernels 32.1 us), not
// eight of 64 (35.0).
constexpr int kLossThreads = 128, kLossWarps = kLossThreads / 32;

__global__ void __launch_bounds__(kLossThreads, 10) distill_loss_kernel(const __grid_constant__ DistArgs p, const DistSaved sv) {
    __shared__ FF part[3][kLossWarps];
    __shared__ float largest[kLossWarps];
    __shared__ int infinite[kLossWarps];
    const rl_distill_args& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    long long eb = a.offsets[row], ee = a.offsets[row + 1];
    if (eb < 0 || ee < eb || ee > a.nnz) eb = ee = 0;
    const int nw = static_cast<int>(min(static_cast<long long>(kLossWarps), max((ee - eb + 31) / 32, 1ll))), stride = nw * 32;
    if (warp >= nw) return;
    auto entry_at = [&](long long e) -> Entry {
        Entry x;
        x.id = a.ids[e];
        x.lq = a.logq[e];
        x.in = x.id >= 0 && x.id < a.V && x.lq > -INFINITY && x.lq < INFINITY;
        x.z = -INFINITY;
        return x;
    };
    Entry first{-1, -INFINITY, 0.f, false};
    float mT = -INFINITY;
    for (long long e = eb + tid; e < ee; e += stride) {
        const Entry x = entry_at(e);
        if (e == eb + tid) first = x;
        if (x.in) mT = fmaxf(mT, x.lq);
    }
    mT = warp_largest(mT);
    if (nw > 1) {
        if (lane == 0) largest[warp] = mT;
        asm volatile("bar.sync 1, %0;" ::"r"(stride) : "memory");
        for (int k = 0; k < nw; ++k) mT = fmaxf(mT, largest[k]);
    }
    wait_for_previous();
    if (!(mT > -INFINITY)) {                     // no teacher
        if (tid == 0) {
            a.loss[row] = 0.f;
            if (a.mass) a.mass[row] = 0.f;
        }
        return;
    }
    const float M = sv.M[row], ref = sv.ref[row], rest = sv.sum[row];
    // (v - m) / T; past the range of floats (the type's lowest number at T < 1, say) it is -inf, which pairs do not carry through
    auto scaled = [&](float v, float m) -> FF {
        return (v - m) * p.inv_t.hi == -INFINITY ? FF{-INFINITY, 0.f} : ff_mul(two_sum(v, -m), p.inv_t);
    };
    // f(entry, W, Q) with the weights of the student's and the teacher's softmax; the thread's first stay in registers
    FF W1 = {0.f, 0.f}, Q1 = {0.f, 0.f};
    auto each = [&](bool again, auto f) {
        for (long long e = eb + tid; e < ee; e += stride) {
            const bool is_first = e == eb + tid;
            Entry x = is_first ? first : entry_at(e);
            if (!x.in) continue;
            if (!is_first || !again) x.z = sv.z[e];
            FF W = W1, Q = Q1;
            if (!is_first || !again) {
                W = exp_table(scaled(x.z, M));
                Q = exp_table(a.tail ? FF{x.lq, 0.f} : scaled(x.lq, mT));
            }
            if (is_first && !again) {
                first.z = x.z;
                W1 = W;
                Q1 = Q;
            }
            f(x, W, Q);
        }
    };
    FF wS = {0.f, 0.f}, wQ = {0.f, 0.f};
    each(false, [&](const Entry&, FF W, FF Q) {
        wS = ff_add(wS, W);
        wQ = ff_add(wQ, Q);
    });
    wS = support_sum(part[0], wS, nw);
    wQ = support_sum(part[1], wQ, nw);
    // the rest's sum, relative to the row's reference
    FF far = {0.f, 0.f}, wR = {rest, 0.f};
    if (ref != M && rest != 0.f) {
        far = scaled(ref, M);
        wR = ff_mul(wR, exp_table(far));
    }
    const FF sum = ff_add(wR, wS), t0 = a.tail ? rest_of(wQ) : FF{1.f, 0.f};
    // three logs, a lane each
    const FF ln = ln_table(lane == 0 ? sum : lane == 1 ? (a.tail ? t0 : wQ) : FF{rest, 0.f});
    auto lane_of = [&](FF v, int k) -> FF { return {__shfl_sync(0xffffffffu, v.hi, k), __shfl_sync(0xffffffffu, v.lo, k)}; };
    const FF lnS = lane_of(ln, 0), ln1 = lane_of(ln, 1), lnR = lane_of(ln, 2);
    const FF inv_S = ff_div({1.f, 0.f}, sum), inv_Q = a.tail ? FF{1.f, 0.f} : ff_div({1.f, 0.f}, wQ);
    FF loss = {0.f, 0.f};
    bool inf = false;
    each(true, [&](const Entry& x, FF W, FF Q) {
        const FF X = scaled(x.z, M);
        const FF lp = X.hi == -INFINITY ? X : ff_add(X, ff_neg(lnS));
        const FF lt = a.tail ? FF{x.lq, 0.f} : ff_add(scaled(x.lq, mT), ff_neg(ln1)), t = a.tail ? Q : ff_mul(Q, inv_Q);
        const Term r = term_of(a.kind, a.beta, t, lt, ff_mul(W, inv_S), lp);
        loss = ff_add(loss, r.f);
        inf |= r.inf;
    });
    inf = __any_sync(0xffffffffu, inf);
    if (lane == 0) infinite[warp] = inf;
    loss = support_sum(part[2], loss, nw);
    for (int k = 0; k < nw; ++k) inf |= nw > 1 && infinite[k] != 0;
    if (a.tail && rest != 0.f && !((ref - M) * p.inv_t.hi < kRestGone))
        loss = ff_add(loss, term_of(a.kind, a.beta, t0, ln1, ff_mul(wR, inv_S), ff_add(ff_add(far, lnR), ff_neg(lnS))).f);
    if (tid == 0) {
        // (a row of -inf alone has no probabilities)
        a.loss[row] = !(sum.hi > 0.f) ? NAN : inf && loss.hi == loss.hi ? INFINITY : loss.hi + loss.lo;
        if (a.mass) a.mass[row] = (wS.hi + wS.lo) / (sum.hi + sum.lo);
        if (inf || !(fabsf(loss.hi) < INFINITY) || !(sum.hi > 0.f)) set_status(p.status, RL_STATUS_NONFINITE);
    }
}

// ---- the backward alone: gradients from what the forward saved --------------------------------
// One factor times the logits' exponentials, then the support's entries: a stretch of a row a block, all of a thread's loads before
// the look-ups.  HBM bounds it: 2048 fp32 rows of 151,936 371 us (99 % of a copy's rate), 4096 bf16 rows 418 us (88 %, where an
// exponential is half as many bytes).  Stretches of 8 KB: 408 and 466 us; of 32 KB: 369 and 404, but 4096 bf16 rows of 4096 logits
// 18.4 us instead of 14.8.
constexpr int kBwdThreads = 256;
constexpr int kBwdBytes = 16 * 1024;

template <typename T>
__global__ void __launch_bounds__(kBwdThreads) distill_bwd_kernel(const DistArgs p, const DistSaved sv) {
    const rl_distill_args& a = p.a;
    constexpr int E = Pack<T>::E, kStep = kBwdBytes / sizeof(T), kDeep = kStep / kBwdThreads / E;
    const long long row = blockIdx.x;
    const int tid = threadIdx.x, V = static_cast<int>(a.V);
    const int i0 = static_cast<int>(blockIdx.y) * kStep, i1 = min(i0 + kStep, V);
    const T* z = static_cast<const T*>(a.logits) + row * a.row_stride;
    T* d = static_cast<T*>(a.dlogits) + row * a.grad_stride;
    // whole 16 bytes where logits and gradients start alike, the edges by ones
    const uintptr_t x = reinterpret_cast<uintptr_t>(z + i0) & 15, y = reinterpret_cast<uintptr_t>(d + i0) & 15;
    const int head = x == y ? min(static_cast<int>((16 - x) % 16 / sizeof(T)), i1 - i0) : i1 - i0, b0 = i0 + head, packed = (i1 - b0) / E;
    // (all loads are on their way before anything is looked up)
    Pack<T> v[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
        if (u * kBwdThreads + tid < packed) v[u].load(z + b0 + (u * kBwdThreads + tid) * E);
    const float w = a.dloss[row], ref = sv.ref[row], rest = sv.rest[row];
    long long eb = a.offsets[row], ee = a.offsets[row + 1];
    if (eb < 0 || ee < eb || ee > a.nnz) eb = ee = 0;
    const bool zero = w == 0.f || eb == ee;
    const float k = zero ? 0.f : w * rest;
    // one rounding of the argument, as in the pass over the logits
    const float pm = ref * p.c;
    const bool fused = fabsf(pm) < kFusedRef;
    const float k2 = fused ? k * exp2f(-fmaf(ref, p.c, -pm)) : k;
    auto grad = [&](float x) -> float { return k == 0.f ? 0.f : fused ? k2 * exp2_approx(fmaf(x, p.c, -pm)) : k * exp2_approx((x - ref) * p.c); };
    for (int i = i0 + tid; i < b0; i += kBwdThreads) d[i] = from_f32<T>(grad(to_f32(z[i])));
    auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
            const int q = u * kBwdThreads + tid;
            if (q >= packed) break;
            float g[E];
#pragma unroll
            for (int j = 0; j < E; ++j) g[j] = f(to_f32(v[u].t[j]));
            v[u].put(g);
            v[u].store(d + b0 + q * E);
        }
    };
    if (k != 0.f && fused) each([&](float x) { return k2 * exp2_approx(fmaf(x, p.c, -pm)); });
    else each(grad);
    for (int i = b0 + packed * E + tid; i < i1; i += kBwdThreads) d[i] = from_f32<T>(grad(to_f32(z[i])));
    if (zero) return;
    long long lo = eb, hi = ee;                 // first entry with id >= i0
    while (lo < hi) {
        const long long mid = (lo + hi) >> 1;
        if (a.ids[mid] < i0) lo = mid + 1;
        else hi = mid;
    }
    __syncthreads();
    for (long long e = lo + tid; e < ee; e += kBwdThreads) {
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

constexpr int kSliceTarget = 75 * 1024;         // bytes: three blocks a multiprocessor, whose loads, sums and stores overlap
constexpr int kSliceLeast = 4 * 1024;
constexpr int kMiddleSlice = 50 * 1024, kShortSlice = 12 * 1024;
static_assert(kDistillRowBytes <= 8 * (kDistillSliceBytes - 64), "a cluster of eight holds the longest row");

template <typename T, int NT, int kBlocks>
static int distill_launch(const DistArgs& p, const DistSaved& sv, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(distill_kernel<T, NT, kBlocks>, kDistillSliceBytes, done)) return RL_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.a.N * p.cs), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(p.slice) * sizeof(T);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.cs);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    ProfScope prof(RL_PROF_OTHER, stream);
    if (cudaLaunchKernelEx(&cfg, distill_kernel<T, NT, kBlocks>, p, sv) != cudaSuccess) return RL_ERR_CUDA;
    const int rc = launch_after(distill_loss_kernel, dim3(static_cast<unsigned>(p.a.N)), kLossThreads, 0, true, stream, p, sv);
    count_launch(2);
    return rc == RL_OK && cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <typename T>
static int distill_run(DistArgs p, const DistSaved& sv, cudaStream_t stream) {
    const long long bytes = p.a.V * static_cast<long long>(sizeof(T));
    // the fewest blocks a row whose slices leave room for others on the multiprocessor; more of them where
    // there are too few rows to fill the GPU
    int cs = 1;
    while (cs < 8 && (bytes / cs > kSliceTarget || (p.a.N * cs < num_sms() && bytes / cs >= 2 * kSliceLeast))) ++cs;
    const int quantum = 32 / static_cast<int>(sizeof(T));
    p.cs = cs;
    p.slice = static_cast<int>(((p.a.V + 16 / sizeof(T)) + cs * quantum - 1) / (cs * quantum)) * quantum;
    if (p.a.N * cs >= (1ll << 31)) {
        set_last_error("too many rows");
        return RL_ERR_UNSUPPORTED;
    }
    const int own = p.slice * static_cast<int>(sizeof(T));
    return own <= kShortSlice ? distill_launch<T, 128, 8>(p, sv, stream) : own <= kMiddleSlice ? distill_launch<T, 256, 4>(p, sv, stream) : distill_launch<T, 256, 3>(p, sv, stream);
}

template <typename T>
static int distill_bwd_run(const DistArgs& p, const DistSaved& sv, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.a.N), static_cast<unsigned>((p.a.V * static_cast<int64_t>(sizeof(T)) + kBwdBytes - 1) / kBwdBytes), 1);
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
    const DistSaved sv = dist_saved(saved, a->N, a->nnz, nullptr);
    if (pass == kDistillBwd)
        return a->dtype == RL_DTYPE_F32 ? distill_bwd_run<float>(p, sv, stream)
               : a->dtype == RL_DTYPE_BF16 ? distill_bwd_run<__nv_bfloat16>(p, sv, stream) : distill_bwd_run<__half>(p, sv, stream);
    return a->dtype == RL_DTYPE_F32 ? distill_run<float>(p, sv, stream)
           : a->dtype == RL_DTYPE_BF16 ? distill_run<__nv_bfloat16>(p, sv, stream) : distill_run<__half>(p, sv, stream);
}

}  // namespace rl
