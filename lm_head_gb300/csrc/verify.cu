// Verification of drafted tokens against the target's probabilities.
//
// An acceptance u q(x) < p(x) compares two numbers, and almost always they are further apart than
// fp32 sums are wrong; the token after the accepted ones is decided by a cumulative sum over up to the
// whole vocabulary, where fp32 sums would give another one every few hundred requests.  So
//
//  1. chunk_kernel     the only pass over all rows of logits: a warp per 4 KB, its largest logit and the sum of its
//                      weights in fp32.  Rows that no request looks at (a draft's row behind its last draft) are left out.
//  2. decide_kernel    a block a request: puts the rows' totals together and compares; a comparison nearer than the bound
//                      of the fp32 sums' error is taken again with sums that are good to 2^-36.  Draws from support rows.
//  3. sum_kernel       the rows of logits that a request's new token comes from, a step of 512 tokens a warp at a time, every
//                      multiprocessor the same number of them whatever the number of requests: of each part of 128 the sums, as integers
//                      (float-pair weights, see weights.cuh), of the target's weights, or of what is left, max(p - q, 0), where the
//                      draft has logits too.
//  4. pick_kernel      a block a request: adds the parts up, takes a draft's support row off the target's parts, and scans
//                      the part in which the random number falls.
//
// 128 requests of five bf16 rows of 151,936 logits on both sides, 149 us: the pass over 350 MB 62 us (82 % of a copy's rate),
// the decisions 9, the sums 78 and the tokens 16 by themselves, each kernel's start under the one before.  The
// sums read 78 MB that are mostly in L2; what bounds them is the issue of some 50 instructions a weight (two table look-ups,
// two polynomials and three sums in pairs of floats for a token), 2.7 of 4 a cycle.  Sums that stay with a request (a
// cluster of two to eight blocks for each, which scans its own parts) left multiprocessors without blocks: 160 us, one
// request 24 us instead of 20, eight 37 instead of 31.
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "ff.cuh"
#include "internal.h"
#include "weights.cuh"

namespace rl {

constexpr int kVerPart = 128;                  // logits of a part
constexpr int kVerStep = 4;                    // parts that a warp sums up at a time
constexpr int kDecideThreads = 512;            // a row of either side a warp
constexpr int kSumThreads = 1024;
constexpr int kSumBlocks = 1;                  // of them on a multiprocessor
constexpr int kPickThreads = 512;
constexpr int kChunkThreads = 256;
constexpr int kChunkPacks = 8;                 // 16-byte loads of a lane: 4 KB a warp
constexpr int kUsedRows = 32768;               // rows of a step whose use is looked up in shared memory
constexpr int kListedRows = 8192;              // rows of a step of which those that are read are listed
constexpr float kPlainRef = 1900.f;            // |max log2(e) / T| up to which weights need no difference to the maximum

struct VerSide {
    rl_dist d;
    int dtype;
    int nc;             // chunks of a row
    float2* part;       // [T, nc] largest logit, sum of e^((z - it) / T) (T = 0: bits of its first index)
};
struct VerArgs {
    rl_verify_args a;
    VerSide side[2];    // target, draft
    int32_t* status;
    bool sure;          // no draft distribution
    int group;          // chunks that a warp takes one after another
    int steps;          // of a row
    struct VerDraw* draws;      // [R] (NULL: no logits on either side)
    struct VerStep* sums;       // [R, steps]
    int32_t *todo, *n_todo;     // [R] the requests with sums to take, in any order; their number
};

// The row of the distribution that the step's row t has; -1 where there is none.
RL_DEVINL long long row_of(const rl_dist& d, long long t, int& bits) {
    const long long r = d.rows ? d.rows[t] : t;
    if (r < 0 || r >= d.n_rows) {
        bits |= RL_STATUS_OFFSETS;
        return -1;
    }
    return r;
}
RL_DEVINL bool is_support(const rl_dist& d, long long row) { return d.offsets && (!d.logits || d.replayed[row] != 0); }
RL_DEVINL float temperature_of(const rl_dist& d, long long row, int& bits) {      // 0: greedy
    const float T = d.temperature ? d.temperature[row] : 1.f;
    if (T == 0.f) return 0.f;
    if (!(T >= 4.f * FLT_MIN) || !(T <= FLT_MAX)) {
        bits |= RL_STATUS_KNOB;
        return 0.f;
    }
    return T;
}
RL_DEVINL float unit_of(float u, int& bits) {
    if (u >= 0.f && u < 1.f) return u;
    bits |= RL_STATUS_KNOB;
    return u >= 1.f ? 1.f - 5.9604645e-8f : 0.f;
}
RL_DEVINL float logit_at(const rl_dist& d, int dtype, long long row, long long j) {      // NaN and +inf as -inf
    const long long i = row * d.row_stride + j;
    const float z = dtype == RL_DTYPE_F32   ? static_cast<const float*>(d.logits)[i]
                    : dtype == RL_DTYPE_BF16 ? to_f(static_cast<const __nv_bfloat16*>(d.logits)[i])
                                             : to_f(static_cast<const __half*>(d.logits)[i]);
    return z < INFINITY ? z : -INFINITY;
}

// ---- 1. chunks ---------------------------------------------------------------------------
// HBM: 350 MB in 62 us.  A warp's eight 16-byte loads a lane are all on their way before the first is used; 24 warps a
// multiprocessor, 98 KB in flight.
// Places: element i of a row lies at place i + phase, so that 16-byte packs of places are aligned.
template <typename T>
RL_DEVINL float2 chunk_of(const T* row, int V, int chunk, float Tm, bool& bad) {
    constexpr int E = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    const int phase = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int i0 = (chunk * kChunkPacks * 32 + lane) * E - phase;
    uint4 q[kChunkPacks];
    const int first = chunk * kChunkPacks * 32 * E - phase;
    if (first >= 0 && first + kChunkPacks * 32 * E <= V) {
#pragma unroll
        for (int k = 0; k < kChunkPacks; ++k) q[k] = __ldcs(reinterpret_cast<const uint4*>(row + i0 + k * 32 * E));
    } else
#pragma unroll
    for (int k = 0; k < kChunkPacks; ++k) {
        const int i = i0 + k * 32 * E;
        if (i >= 0 && i + E <= V) {
            q[k] = __ldcs(reinterpret_cast<const uint4*>(row + i));
        } else {
            T t[E];
#pragma unroll
            for (int j = 0; j < E; ++j) t[j] = i + j >= 0 && i + j < V ? row[i + j] : static_cast<T>(-INFINITY);
            memcpy(&q[k], t, 16);
        }
    }
    auto get = [&](int k, int j) -> float {
        const uint32_t w = j < E / 4 * 1 ? q[k].x : j < E / 4 * 2 ? q[k].y : j < E / 4 * 3 ? q[k].z : q[k].w;
        if constexpr (sizeof(T) == 4) return __uint_as_float(w);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float((j & 1) ? w & 0xffff0000u : w << 16);
        else return __half2float(__ushort_as_half(static_cast<unsigned short>((j & 1) ? w >> 16 : w & 0xffffu)));
    };
    float m;
    if constexpr (sizeof(T) == 4) {
        m = -INFINITY;
#pragma unroll
        for (int k = 0; k < kChunkPacks; ++k) m = max_nan(max_nan(m, max_nan(get(k, 0), get(k, 1))), max_nan(get(k, 2), get(k, 3)));
    } else {             // two at a time
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 x[kChunkPacks * 4];
        memcpy(x, q, sizeof(x));
        T2 best = x[0];
#pragma unroll
        for (int k = 1; k < kChunkPacks * 4; ++k) best = __hmax2_nan(best, x[k]);
        m = max_nan(__low2float(best), __high2float(best));
    }
    uint32_t key = __reduce_max_sync(0xffffffffu, key_of(m + 0.f));
    if (key >= 0xff800000u) {            // NaN or +inf among them: they count as -inf
        bad = true;
        const uint32_t none = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
        m = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < kChunkPacks; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < kChunkPacks; ++c)
                if (c == k) memcpy(w, &q[c], 16);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int at = sizeof(T) == 4 ? j : j >> 1, sh = sizeof(T) == 4 ? 0 : (j & 1) * 16;
                const uint32_t mask = sizeof(T) == 4 ? 0xffffffffu : 0xffffu;
                T t;
                const uint32_t bitsj = (w[at] >> sh) & mask;
                memcpy(&t, &bitsj, sizeof(T));
                const float z = to_f(t);
                if (!(z < INFINITY)) w[at] = (w[at] & ~(mask << sh)) | (none << sh);
                else m = fmaxf(m, z);
            }
#pragma unroll
            for (int c = 0; c < kChunkPacks; ++c)
                if (c == k) memcpy(&q[c], w, 16);
        }
        key = __reduce_max_sync(0xffffffffu, key_of(m + 0.f));
    }
    m = z_of(key);
    if (!(m > -INFINITY)) return make_float2(m, 0.f);
    if (Tm == 0.f) {
        int at = INT_MAX;
#pragma unroll
        for (int k = kChunkPacks - 1; k >= 0; --k)
#pragma unroll
            for (int j = E - 1; j >= 0; --j)
                if (get(k, j) == m) at = i0 + k * 32 * E + j;
        return make_float2(m, __uint_as_float(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(at))));
    }
    // e^((z - m) / T) as 2^(z c - fl(m c)): one rounding of the argument; the sum is put right for fl(m c) after
    const float c = kLog2eHi / Tm, pm = m * c;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (fabsf(pm) < kFusedRef) {
#pragma unroll
        for (int k = 0; k < kChunkPacks; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) s[j & 3] += exp2_approx(fmaf(get(k, j), c, -pm));
        return make_float2(m, warp_sum((s[0] + s[1]) + (s[2] + s[3])) * exp2f(-fmaf(m, c, -pm)));
    }
#pragma unroll
    for (int k = 0; k < kChunkPacks; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j) s[j & 3] += exp2_approx((get(k, j) - m) * c);
    return make_float2(m, warp_sum((s[0] + s[1]) + (s[2] + s[3])));
}

__global__ void __launch_bounds__(kChunkThreads, 3) chunk_kernel(const __grid_constant__ VerArgs g) {
    __shared__ uint32_t used[2][kUsedRows / 32];
    __shared__ uint16_t list[2 * kListedRows];   // the rows of logits that are read, the target's first
    __shared__ int sums[kChunkThreads / 32];
    const rl_verify_args& a = g.a;
    const int V = static_cast<int>(a.V);
    for (long long t = static_cast<long long>(blockIdx.x) * kChunkThreads + threadIdx.x; t < a.T; t += static_cast<long long>(gridDim.x) * kChunkThreads) {
        a.tokens[t] = -1;
        if (a.logq) a.logq[t] = 0.f;
    }
    if (g.draws && blockIdx.x == 0 && threadIdx.x == 0) *g.n_todo = 0;
    // the rows that requests look at
    const bool known = a.T <= kUsedRows;
    if (known) {
        const int words = static_cast<int>((a.T + 31) / 32);
        for (int i = threadIdx.x; i < words; i += kChunkThreads) used[0][i] = used[1][i] = 0;
        __syncthreads();
        for (long long r = threadIdx.x; r < a.R; r += kChunkThreads) {
            const long long t0 = a.cu_q[r], t1 = a.cu_q[r + 1];
            if (t0 < 0 || t1 < t0 || t1 > a.T) continue;
            for (int t = static_cast<int>(t0); t < t1; ++t) {
                atomicOr(&used[0][t >> 5], 1u << (t & 31));
                if (t + 1 < t1) atomicOr(&used[1][t >> 5], 1u << (t & 31));
            }
        }
        __syncthreads();
    }
    // Where a side may have support rows beside logits, the rows that are read are listed, so that all warps read as many: with 256
    // requests, half of them with support rows, this kernel takes 43 us, 53 without the list.  Making it takes 1.5 us, which steps
    // whose rows are all logits need not spend.
    const bool listed = a.T <= kListedRows && ((g.side[0].d.logits && g.side[0].d.offsets) || (g.side[1].d.logits && g.side[1].d.offsets));
    long long n_rows[2] = {a.T, a.T};
    if (listed) {
        const int T = static_cast<int>(a.T), per = (T + kChunkThreads - 1) / kChunkThreads, t0 = min(static_cast<int>(threadIdx.x) * per, T), t1 = min(t0 + per, T);
        int at = 0;
        for (int side = 0; side < 2; ++side) {
            const rl_dist& d = g.side[side].d;
            auto read = [&](int t) {
                int none = 0;
                if (!d.logits || !((used[side][t >> 5] >> (t & 31)) & 1u)) return false;
                const long long row = row_of(d, t, none);
                return row >= 0 && !is_support(d, row);
            };
            int n = 0;
            for (int t = t0; t < t1; ++t) n += read(t);
            int before = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, before, o);
                if (static_cast<int>(threadIdx.x & 31) >= o) before += x;
            }
            __syncthreads();
            if ((threadIdx.x & 31) == 31) sums[threadIdx.x >> 5] = before;
            __syncthreads();
            before += at - n;
            int total = 0;
            for (int w = 0; w < kChunkThreads / 32; ++w) {
                if (w < static_cast<int>(threadIdx.x >> 5)) before += sums[w];
                total += sums[w];
            }
            for (int t = t0; t < t1 && n > 0; ++t)
                if (read(t)) list[before++] = static_cast<uint16_t>(t);
            n_rows[side] = total;
            at += total;
        }
        __syncthreads();
    }
    // one or two chunks of a row a warp
    const long long warps = static_cast<long long>(gridDim.x) * (kChunkThreads / 32);
    const int groups[2] = {(g.side[0].nc + g.group - 1) / g.group, (g.side[1].nc + g.group - 1) / g.group};
    const long long first = n_rows[0] * groups[0], units = first + n_rows[1] * groups[1];
    int bits = 0;
    bool bad = false;
    for (long long id = static_cast<long long>(blockIdx.x) * (kChunkThreads / 32) + (threadIdx.x >> 5); id < units; id += warps) {
        const int side = id >= first ? 1 : 0;
        const VerSide& s = g.side[side];
        const long long x = side ? id - first : id;
        const long long k = x <= UINT_MAX ? static_cast<uint32_t>(x) / static_cast<uint32_t>(groups[side]) : x / groups[side];
        const int c0 = static_cast<int>(x - k * groups[side]) * g.group, c1 = min(c0 + g.group, s.nc);
        const long long t = listed ? list[(side ? n_rows[0] : 0) + k] : k;
        if (!listed && known && !((used[side][t >> 5] >> (t & 31)) & 1u)) continue;
        int row_bits = 0;
        const long long row = row_of(s.d, t, row_bits);
        if (!listed && (row < 0 || is_support(s.d, row))) continue;
        const float Tm = temperature_of(s.d, row, bits);
        float2 mine = make_float2(0.f, 0.f);
        auto each = [&](auto* p) {
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                const float2 v = chunk_of(p, V, c, Tm, bad);
                if ((threadIdx.x & 31) == c - c0) mine = v;
            }
        };
        if (s.dtype == RL_DTYPE_F32) each(static_cast<const float*>(s.d.logits) + row * s.d.row_stride);
        else if (s.dtype == RL_DTYPE_BF16) each(static_cast<const __nv_bfloat16*>(s.d.logits) + row * s.d.row_stride);
        else each(static_cast<const __half*>(s.d.logits) + row * s.d.row_stride);
        if (static_cast<int>(threadIdx.x & 31) < c1 - c0) s.part[t * s.nc + c0 + (threadIdx.x & 31)] = mine;
    }
    if (bad) bits |= RL_STATUS_NONFINITE;
    set_status(g.status, bits);
    let_next_start();
}

// ---- 2. requests ---------------------------------------------------------------------------
// Latency: a row's parts (75 of 4 KB), its candidate's logit, one comparison (9 us by itself); support rows' draws are
// a block's sums and a scan (256 requests, half of them support rows, 18 us).
enum { kDistNone, kDistDense, kDistPoint, kDistSupport };

// A row's distribution.
struct VerRow {
    int mode, dtype, at;            // kDistPoint: all of it on `at`
    int prec;                       // sums are in units of 2^-prec
    long long row, eb, ee;
    float M, S;                     // largest logit, fp32 sum of e^((z - M) / T)
    FF c;                           // log2(e) / T
    float inv_c, R;                 // weights are 2^(z c - R) where `plain`, else 2^((z - M) c) with R = 0
    int plain, vec;
    unsigned long long total;       // the sum of all weights, once it is counted
};
// 2^lam as it enters the draft's weights: an integer power, a part in steps of 2^-11 in [0, 1) and the rest.
struct Lam {
    int whole;
    float hi, lo;
};
// What a request's new token is drawn from.
struct VerDraw {
    long long t;                    // -1: nothing is left to draw
    float u;
    Lam lam;                        // of two rows of logits: log2 of the draft's total over the target's, as their fp32 sums have it
    VerRow row[2];
};
// The sums of a step, in the rows' units.
struct alignas(16) VerStep {
    unsigned long long part[kVerStep];      // of each part, what the token is drawn from
    float drop[kVerStep];                   // of two rows of logits: the draft's weight where something is left,
    unsigned long long p, q;                // and both totals
};

template <int NT>
struct VerShared {
    float2 tab[2048];
    unsigned long long red[NT / 32];
    unsigned long long red2[NT / 32];
    VerDraw draw;
    VerRow rows[NT / 32];           // the rows of a stretch of the request, target and draft in turn
    float lp[NT / 32];              // log2 of the candidate's probability
    int bits[NT / 32];
    int flag, token;
    float lpx;
    FF lam;                         // log2 of the draft's total over the target's, as they are counted
    float turn;                     // ln 2 times the difference to the fp32 sums'
    unsigned long long unit;
};

// hi + lo (normalised, 0 <= it < 2) in units of 2^-k, k <= 60
RL_DEVINL unsigned long long fixed_of(float hi, float lo, int k) {
    if (!(hi > 0.f)) return 0ull;
    const uint32_t b = __float_as_uint(hi);
    const int sh = static_cast<int>(b >> 23) - 127 - 23 + k;
    const unsigned long long m = (b & 0x7fffffu) | ((b >> 23) ? 0x800000u : 0u);
    const unsigned long long w = sh >= 0 ? m << sh : sh > -25 ? (m + (1ull << (-sh - 1))) >> -sh : 0ull;
    const long long v = static_cast<long long>(w) + __float2ll_rn(lo * power_of_2(k));
    return v > 0 ? static_cast<unsigned long long>(v) : 0ull;
}
// 2^(x c - ref - lam_lo) as a normalised pair, below 2; magic = 6144 - ref with ref in steps of 2^-11 (see weight_pair; with
// lam_lo |r| may be 2^-11, so 2^r - 1 goes to the third power).
template <bool kLow = true>
RL_DEVINL FF weight_off(float x, float xl, FF c, float magic, float lam_lo, const float2* tab) {
    const float t = fmaf(x, c.hi, magic);
    float r = fmaf(x, c.hi, -__fsub_rn(t, magic));
    r = fmaf(x, c.lo, r);
    if (kLow) r = fmaf(xl, c.hi, r);             // (x is not a pair where weights need no difference)
    r -= lam_lo;
    const uint32_t tb = __float_as_uint(t);
    const float2 q = tab[tb & 2047u];
    const float hi = __uint_as_float(__float_as_uint(q.x) + (tb << 12));
    return fast_two_sum(hi, hi * fmaf(r, fmaf(r, fmaf(r, 0.05550410866482158f, 0.24022650695910072f), 0.69314718055994531f), q.y));
}
// The weight of a logit over 2^ref (as in VerRow) times 2^-lam.  ref holds lam's part in steps of 2^-11, lam_lo the rest.
RL_DEVINL FF weight_of(float z, const VerRow& w, float ref, float lam_lo, const float2* tab) {
    const FF d = w.plain ? FF{z, 0.f} : two_sum(z, -w.M);
    return weight_off(d.hi, d.lo, w.c, 6144.f - (w.R + ref), lam_lo, tab);
}
// Its exponent, as a float.
RL_DEVINL float exponent_of(float z, const VerRow& w, float ref) {
    return fmaf(w.plain ? z : two_sum(z, -w.M).hi, w.c.hi, -(w.R + ref));
}
// The logit at which the exponent over 2^ref is e.
RL_DEVINL float logit_of(const VerRow& w, float ref, float e) {
    const float x = (ref + w.R + e) * w.inv_c;
    return w.plain ? x : w.M + x;
}
// max(v - q, 0) of normalised pairs, as a pair that is not in order
RL_DEVINL FF left_of(FF v, FF q) {
    const float d = __fsub_rn(v.hi, q.hi), e = __fadd_rn(__fsub_rn(__fsub_rn(v.hi, d), q.hi), __fsub_rn(v.lo, q.lo));
    return v.hi >= q.hi && __fadd_rn(d, e) > 0.f ? FF{d, e} : FF{0.f, 0.f};
}
RL_DEVINL FF ordered(FF x) { return two_sum(x.hi, x.lo); }

RL_DEVINL const void* logits_of(const rl_dist& d, const VerRow& r) {
    return static_cast<const char*>(d.logits) + ((r.row * d.row_stride) << (r.dtype == RL_DTYPE_F32 ? 2 : 1));
}
// A lane's logits of N parts from element i0 on, four of each, past the row's end -inf.
template <int N>
RL_DEVINL void step_load(const void* logits, const VerRow& r, int V, int i0, float (&z)[N][4]) {
    const int lane = threadIdx.x & 31;
    const bool whole = r.vec && i0 + N * kVerPart <= V;
    if (r.dtype == RL_DTYPE_F32) {
        const float* p = static_cast<const float*>(logits) + i0 + lane * 4;
        if (whole) {
#pragma unroll
            for (int s = 0; s < N; ++s) {
                const float4 q = *reinterpret_cast<const float4*>(p + s * kVerPart);
                z[s][0] = q.x; z[s][1] = q.y; z[s][2] = q.z; z[s][3] = q.w;
            }
        } else {
#pragma unroll
            for (int s = 0; s < N; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) z[s][j] = i0 + s * kVerPart + lane * 4 + j < V ? p[s * kVerPart + j] : -INFINITY;
        }
        return;
    }
    const uint16_t* p = static_cast<const uint16_t*>(logits) + i0 + lane * 4;
    uint2 q[N];
    if (whole) {
#pragma unroll
        for (int s = 0; s < N; ++s) q[s] = *reinterpret_cast<const uint2*>(p + s * kVerPart);
    } else {
        const uint32_t none = r.dtype == RL_DTYPE_BF16 ? 0xff80u : 0xfc00u;
#pragma unroll
        for (int s = 0; s < N; ++s) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = i0 + s * kVerPart + lane * 4 + j < V ? p[s * kVerPart + j] : none;
            q[s] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        }
    }
    if (r.dtype == RL_DTYPE_BF16) {
#pragma unroll
        for (int s = 0; s < N; ++s) {
            z[s][0] = __uint_as_float(q[s].x << 16);
            z[s][1] = __uint_as_float(q[s].x & 0xffff0000u);
            z[s][2] = __uint_as_float(q[s].y << 16);
            z[s][3] = __uint_as_float(q[s].y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int s = 0; s < N; ++s) {
            const __half2 a = *reinterpret_cast<const __half2*>(&q[s].x), b = *reinterpret_cast<const __half2*>(&q[s].y);
            z[s][0] = __low2float(a); z[s][1] = __high2float(a); z[s][2] = __low2float(b); z[s][3] = __high2float(b);
        }
    }
}
// The warp's largest of them; NaN and +inf become -inf.
template <int N>
RL_DEVINL float step_largest(float (&z)[N][4]) {
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < N; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max_nan(m, z[s][j]);
    uint32_t key = __reduce_max_sync(0xffffffffu, key_of(m + 0.f));
    if (key >= 0xff800000u) {
        m = -INFINITY;
#pragma unroll
        for (int s = 0; s < N; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[s][j] = z[s][j] < INFINITY ? z[s][j] : -INFINITY;
                m = fmaxf(m, z[s][j]);
            }
        key = __reduce_max_sync(0xffffffffu, key_of(m + 0.f));
    }
    return z_of(key);
}

// Units of 2^(ref - 50) in units of 2^-prec.
RL_DEVINL unsigned long long in_units(unsigned long long w50, int ref, int prec) {
    const int sh = prec - 50 + ref;
    return sh >= 0 ? w50 << sh : sh > -64 ? (w50 + (1ull << (-sh - 1))) >> -sh : 0ull;
}
// The step that a warp takes after step k: every `stride`-th, or the next that no warp of the block has.
struct Steps {
    int stride;
    int* next;                    // in shared memory; NULL: by stride
    RL_DEVINL int after(int k) const {
        if (!next) return k + stride;
        int x = 0;
        if ((threadIdx.x & 31) == 0) x = atomicAdd(next, 1);
        return __shfl_sync(0xffffffffu, x, 0);
    }
};
// The table by its shared address: a pointer that a call passes would be a generic one, with slower loads.
RL_DEVINL const float2* table_at(uint32_t table) { return static_cast<const float2*>(__cvta_shared_to_generic(table)); }
// Sums of the weights of a row's steps that are numbers base + k, k < end, by a warp that begins with k; the parts' sums
// into `out` where it is given.  Each step is summed relative to its own largest weight.  Lane 0 has the sum.
__device__ __noinline__ unsigned long long sum_steps(const void* logits, const VerRow* row, int V, int base, int end, int& k, Steps by,
                                                     VerStep* out, uint32_t table) {
    const VerRow w = *row;
    const float2* tab = table_at(table);
    const int lane = threadIdx.x & 31;
    unsigned long long mine = 0;
#pragma unroll 1
    for (; k < end; k = by.after(k)) {
        float z[kVerStep][4];
        step_load(logits, w, V, (base + k) * kVerStep * kVerPart, z);
        const float m = step_largest(z);
        const float ex = w.plain ? fmaf(m, w.c.hi, -w.R) : (m - w.M) * w.c.hi;
        unsigned long long sum = 0;
        if (ex > -100.f) {                       // (also not for -inf: below, the step is nothing beside the row)
            const float ref = fminf(ceilf(ex), 1.f), magic = 6144.f - (w.R + ref);
            const float zlow = fmaxf(logit_of(w, ref, kLeastExp), -FLT_MAX);
            uint32_t top = 0;
            int low = 0;
#pragma unroll
            for (int s = 0; s < kVerStep; ++s) {
                LaneSum acc;
                float hi[4], v[4];
                if (w.plain) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) weight_pair(fmaxf(z[s][j], zlow), 0.f, w.c, magic, tab, hi[j], v[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const FF x = two_sum(fmaxf(z[s][j], zlow), -w.M);
                        weight_pair(x.hi, x.lo, w.c, magic, tab, hi[j], v[j]);
                    }
                }
                const float least = fminf(fminf(z[s][0], z[s][1]), fminf(z[s][2], z[s][3]));
                if (__any_sync(0xffffffffu, least < zlow)) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (z[s][j] < zlow) hi[j] = v[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) acc.add(hi[j], v[j]);
                const uint32_t t = acc.warp_top();
                const int l = acc.warp_low();
                if (lane == s) {
                    top = t;
                    low = l;
                }
            }
            sum = in_units(LaneSum::total(top, low), static_cast<int>(ref), w.prec);
        }
        if (lane < kVerStep) {
            if (out) out[base + k].part[lane] = sum;
            mine += sum;
        }
    }
    mine = lane < kVerStep ? mine : 0ull;
    return warp_sum(mine);
}
// Up to 15 weights of at most 1 in a lane, pairs in order (as LaneSum, from 16 on, where the last place is 2^-19 too).
struct LongSum {
    float top = 16.f, low = 0.f;
    RL_DEVINL void add(FF x) {
        const float n = __fadd_rn(top, x.hi);
        low += __fadd_rn(__fsub_rn(x.hi, __fsub_rn(n, top)), x.lo);
        top = n;
    }
    RL_DEVINL uint32_t warp_top() const { return __reduce_add_sync(0xffffffffu, __float_as_uint(top) - 0x41800000u); }
    RL_DEVINL int warp_low() const { return __reduce_add_sync(0xffffffffu, __float2int_rn(low * 0x1p43f)); }
};
// A target's and a draft's rows of logits in one pass: the totals of both, and of each part what is left, max(p - q, 0), with the ratio
// of the totals taken from the fp32 sums (2^lam) - and the draft's weight where something is left, by which the parts are put
// right once the ratio is known: what is left changes by q d(lam) ln 2 there, and the tokens at which p and q change places matter in
// second order (d(lam)^2, below 2^-36).  Three passes (both totals, then what is left) took half as long again.
// The draft's total comes out as 2^-(hi + lo) times itself.
template <bool kPlain>
RL_DEVINL void sum_both_of(const void* zp, const VerRow& w, const void* yp, const VerRow& o, Lam lam, int V, int base, int end, int& at, Steps by,
                           VerStep* out, const float2* tab) {
    constexpr int N = kVerStep / 2;              // half a step at a time, for the registers
    const int lane = threadIdx.x & 31;
    const bool wp = kPlain || w.plain, op = kPlain || o.plain;
    unsigned long long mine = 0;
#pragma unroll 1
    for (int k = 2 * at; at < end;) {
        const int i0 = (2 * base + k) * N * kVerPart;
        unsigned long long sum = 0;
        float d_out = 0.f;
        if (i0 < V) {
            float z[N][4], y[N][4];
            step_load(zp, w, V, i0, z);
            step_load(yp, o, V, i0, y);
            const float mz = step_largest(z), my = step_largest(y);
            const float ez = wp ? fmaf(mz, w.c.hi, -w.R) : (mz - w.M) * w.c.hi, ey = op ? fmaf(my, o.c.hi, -o.R) : (my - o.M) * o.c.hi;
            // (below 2^-100 of its row's largest, or -inf, a side is nothing here)
            const float rz = ez > -100.f ? fminf(ceilf(ez), 1.f) : 0.f, ry = ey > -100.f ? fminf(ceilf(ey), 1.f) : 0.f;
            const float zlow = ez > -100.f ? fmaxf(wp ? (rz + w.R + kLeastExp) * w.inv_c : w.M + (rz + kLeastExp) * w.inv_c, -FLT_MAX) : FLT_MAX;
            const float ylow = ey > -100.f ? fmaxf(op ? (ry + o.R + kLeastExp) * o.inv_c : o.M + (ry + kLeastExp) * o.inv_c, -FLT_MAX) : FLT_MAX;
            const float magic_z = 6144.f - (w.R + rz), magic_y = 6144.f - (o.R + ry + lam.hi);
            const float scale = power_of_2(min(max(static_cast<int>(ry - rz) - lam.whole, -126), 100));
            LongSum sp, sq;
            uint32_t top = 0;
            int low = 0, d_in = 0;
#pragma unroll
            for (int s = 0; s < N; ++s) {
                LaneSum acc;
                float d = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // (a clamped logit's weight is not used, but has to be one)
                    const float a = z[s][j] < zlow ? (wp ? w.R * w.inv_c : w.M) : z[s][j], b = y[s][j] < ylow ? (op ? o.R * o.inv_c : o.M) : y[s][j];
                    const FF da = wp ? FF{a, 0.f} : two_sum(a, -w.M), db = op ? FF{b, 0.f} : two_sum(b, -o.M);
                    FF v = weight_off<!kPlain>(da.hi, da.lo, w.c, magic_z, 0.f, tab), q = weight_off<!kPlain>(db.hi, db.lo, o.c, magic_y, lam.lo, tab);
                    if (z[s][j] < zlow) v = {0.f, 0.f};
                    if (y[s][j] < ylow) q = {0.f, 0.f};
                    sp.add(v);
                    sq.add(q);
                    q = {q.hi * scale, q.lo * scale};
                    v = left_of(v, q);
                    if (v.hi != 0.f || v.lo != 0.f) d += q.hi;
                    acc.add(v.hi, v.lo);
                }
                const uint32_t t = acc.warp_top();
                const int l = acc.warp_low(), e = __reduce_add_sync(0xffffffffu, __float2int_rn(d * 0x1p20f));
                if (lane == s) {
                    top = t;
                    low = l;
                    d_in = e;
                }
            }
            d_out = static_cast<float>(d_in) * power_of_2(static_cast<int>(rz) - 20);
            // lanes 0 .. N - 1 the parts, N the target's total, N + 1 the draft's
            const uint32_t tz = sp.warp_top(), ty = sq.warp_top();
            const int lz = sp.warp_low(), ly = sq.warp_low();
            if (lane >= N) {
                top = lane == N ? tz : ty;
                low = lane == N ? lz : ly;
            }
            sum = in_units(LaneSum::total(top, low), static_cast<int>(lane <= N ? rz : ry), lane <= N ? w.prec : o.prec);
        }
        VerStep& to = out[base + at];
        if (lane < N) {
            to.part[(k & 1) * N + lane] = sum;
            to.drop[(k & 1) * N + lane] = d_out;
        } else {
            mine += sum;
            if (k & 1) {
                if (lane < N + 2) (lane == N ? to.p : to.q) = mine;
                mine = 0;
            }
        }
        if (k & 1) {
            at = by.after(at);
            k = 2 * at;
        } else {
            ++k;
        }
    }
}
__device__ __noinline__ void sum_both(const void* zp, const VerRow* rp, const void* yp, const VerRow* rq, Lam lam, int V, int base, int end,
                                      int& at, Steps by, VerStep* out, uint32_t table) {
    const float2* tab = table_at(table);
    const VerRow w = *rp, o = *rq;               // (in registers: read again after each store the sums took 7 us more of 85)
    if (w.plain && o.plain) sum_both_of<true>(zp, w, yp, o, lam, V, base, end, at, by, out, tab);
    else sum_both_of<false>(zp, w, yp, o, lam, V, base, end, at, by, out, tab);
}

template <int NT>
struct Request {
    static constexpr int kWarps = NT / 32;
    const VerArgs& g;
    VerShared<NT>& s;
    int V, tid, lane, warp;

    RL_DEVINL unsigned long long block_sum(unsigned long long v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) s.red[warp] = v;
        __syncthreads();
        unsigned long long x = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x += s.red[w];
        return x;
    }
    RL_DEVINL unsigned long long block_scan(unsigned long long v) {      // exclusive
        unsigned long long i = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, i, o);
            if (lane >= o) i += x;
        }
        __syncthreads();
        if (lane == 31) s.red[warp] = i;
        __syncthreads();
        unsigned long long p = 0;
        for (int w = 0; w < warp; ++w) p += s.red[w];
        return p + i - v;
    }

    // One warp: the step's row t on one side, its fp32 total put together.
    RL_DEVINL VerRow row_at(int side, long long t, int& bits) {
        VerRow x{};
        const VerSide& sd = g.side[side];
        x.dtype = sd.dtype;
        if (side == 1 && g.sure) {
            x.mode = kDistPoint;
            x.at = t + 1 < g.a.T ? g.a.step_tokens[t + 1] : -1;
            return x;
        }
        x.row = row_of(sd.d, t, bits);
        if (x.row < 0) return x;
        if (is_support(sd.d, x.row)) {
            x.eb = sd.d.offsets[x.row];
            x.ee = sd.d.offsets[x.row + 1];
            if (x.eb < 0 || x.ee < x.eb || x.ee > sd.d.nnz) {
                bits |= RL_STATUS_OFFSETS;
                return x;
            }
            x.mode = kDistSupport;
            return x;
        }
        const float T = temperature_of(sd.d, x.row, bits);
        const float2* part = sd.part + t * sd.nc;
        // (most rows' parts stay in registers)
        constexpr int kKept = 6;
        float2 v[kKept];
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            v[k] = k * 32 + lane < sd.nc ? part[k * 32 + lane] : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, v[k].x);
        }
        for (int i = kKept * 32 + lane; i < sd.nc; i += 32) M = fmaxf(M, part[i].x);
        M = z_of(__reduce_max_sync(0xffffffffu, key_of(M + 0.f)));
        if (!(M > -INFINITY)) return x;
        x.M = M;
        if (T == 0.f) {
            unsigned at = UINT_MAX;
            for (int i = lane; i < sd.nc; i += 32)
                if (part[i].x == M) at = min(at, __float_as_uint(part[i].y));
            x.at = static_cast<int>(__reduce_min_sync(0xffffffffu, at));
            x.mode = kDistPoint;
            return x;
        }
        x.c = scale_of(T);
        x.inv_c = 1.f / x.c.hi;
        float S = 0.f;
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            if (v[k].x > -INFINITY) S += v[k].y * exp2f((v[k].x - M) * x.c.hi);
        for (int i = kKept * 32 + lane; i < sd.nc; i += 32) {
            const float2 y = part[i];
            if (y.x > -INFINITY) S += y.y * exp2f((y.x - M) * x.c.hi);
        }
        x.S = warp_sum(S);
        x.mode = kDistDense;
        const float pm = __fmul_rn(M, x.c.hi);
        x.plain = fabsf(pm) < kPlainRef;
        x.R = x.plain ? ceilf(pm) : 0.f;
        // S < 2^e, the sum below 2^61 units
        const int e = static_cast<int>(__float_as_uint(x.S * 1.01f) >> 23) - 126;
        x.prec = min(54, 61 - max(e, 1));
        const uintptr_t mask = x.dtype == RL_DTYPE_F32 ? 15 : 7, size = x.dtype == RL_DTYPE_F32 ? 4 : 2;
        x.vec = ((reinterpret_cast<uintptr_t>(sd.d.logits) + static_cast<uintptr_t>(x.row * sd.d.row_stride) * size) & mask) == 0;
        return x;
    }
    // log2 of token j's probability, to fp32 sums; -inf: none
    RL_DEVINL float log2_prob(int side, const VerRow& x, int j, int& bits) {
        if (x.mode == kDistPoint) return j == x.at ? 0.f : -INFINITY;
        if (x.mode == kDistDense) {
            const float z = logit_at(g.side[side].d, x.dtype, x.row, j);
            if (!(z > -INFINITY)) return -INFINITY;
            const FF d = two_sum(z, -x.M);
            const float e = fmaf(d.hi, x.c.hi, fmaf(d.lo, x.c.hi, d.hi * x.c.lo));
            return e > -INFINITY ? e - log2f(x.S) : -INFINITY;       // (a product past the range of floats, or two of them: NaN)
        }
        return support_at(side, x, j, bits) * kLog2e;
    }
    // a support row's log-probability of token j
    RL_DEVINL float support_at(int side, const VerRow& x, int j, int& bits) {
        if (x.mode != kDistSupport) return -INFINITY;
        const rl_dist& d = g.side[side].d;
        long long lo = x.eb, hi = x.ee;
        while (lo < hi) {
            const long long mid = (lo + hi) >> 1;
            if (d.ids[mid] < j) lo = mid + 1;
            else hi = mid;
        }
        if (lo < x.ee && d.ids[lo] == j) {
            const float q = d.logq[lo];
            if (!(q <= 1e-6f)) bits |= RL_STATUS_LOGQ;
            return q < INFINITY ? q : -INFINITY;
        }
        return -INFINITY;
    }
    // ln of token j's probability, in 64 bits (a dense row's total has been counted)
    RL_DEVINL double ln_prob(int side, const VerRow& x, int j, int& bits) {
        if (x.mode == kDistPoint) return j == x.at ? 0.0 : -INFINITY;
        if (x.mode == kDistDense) {
            const float z = logit_at(g.side[side].d, x.dtype, x.row, j);
            if (!(z > -INFINITY) || x.total == 0) return -INFINITY;
            const double c = static_cast<double>(x.c.hi) + static_cast<double>(x.c.lo);
            const double e = x.plain ? z * c : (static_cast<double>(z) - x.M) * c;
            return 0.69314718055994530942 * (e - x.R - (log2(static_cast<double>(x.total)) - x.prec));
        }
        return support_at(side, x, j, bits);
    }
    // A draft's probability of token j as a pair (a dense row's total has been counted, ln_total its log).
    RL_DEVINL FF prob_pair(const VerRow& x, int j, FF ln_total, int& bits) {
        if (x.mode == kDistPoint) return {j == x.at ? 1.f : 0.f, 0.f};
        if (x.mode == kDistDense) {
            const float z = logit_at(g.side[1].d, x.dtype, x.row, j);
            if (!(exponent_of(z, x, 0.f) > -200.f)) return {0.f, 0.f};       // (-inf, or a product past the range of floats)
            const FF d = x.plain ? FF{z, 0.f} : two_sum(z, -x.M);
            // e = d c - R in log2 units, then to natural ones less the total's log
            FF e = ff_add(ff_mul(d, x.c), {-x.R, 0.f});
            e = ff_add(ff_mul(e, {0.693147182464599609375f, -1.90465429995775e-09f}), ff_neg(ln_total));
            return exp_table(e);
        }
        const float q = support_at(1, x, j, bits);
        return q > -INFINITY ? exp_table({q, 0.f}) : FF{0.f, 0.f};
    }
    // ln of a counted total, in the unit 2^R (2^0) of its weights
    static RL_DEVINL FF ln_of(unsigned long long total, int prec) {
        const float th = __ull2float_rz(total);
        const float tl = static_cast<float>(static_cast<long long>(total - static_cast<unsigned long long>(th)));
        return ln_pair(fast_two_sum(th * power_of_2(-prec), tl * power_of_2(-prec)));
    }

    RL_DEVINL void finish(long long t, int token, float l, int& bits) {
        if (token < 0) bits |= RL_STATUS_EMPTY_ROW;
        g.a.tokens[t] = token;
        if (g.a.logq) g.a.logq[t] = token < 0 ? -INFINITY : l;
    }
    // A draw from a support row, by one block.  Sums in units of 2^-52.
    RL_DEVINL void draw_support(long long t, float u, int& bits) {
        const VerRow p = s.draw.row[0], q = s.draw.row[1];
        const rl_dist& d = g.side[0].d;
        const long long n = p.ee - p.eb;
        const FF lq = q.mode == kDistDense ? ln_of(q.total, q.prec) : FF{0.f, 0.f};
        bool whole = q.mode == kDistNone;
        auto left = [&](long long i) -> unsigned long long {
            const int j = d.ids[p.eb + i];
            const float l = d.logq[p.eb + i];
            if (j < 0 || j >= V) {
                bits |= RL_STATUS_ID_RANGE;
                return 0ull;
            }
            if (i > 0 && d.ids[p.eb + i - 1] >= j) bits |= RL_STATUS_ROW_ORDER;
            if (!(l <= 1e-6f)) bits |= RL_STATUS_LOGQ;
            if (!(l < INFINITY) || !(l > -INFINITY)) return 0ull;
            FF v = exp_table({l, 0.f});
            if (!whole) v = ordered(left_of(v, prob_pair(q, j, lq, bits)));
            return fixed_of(v.hi, v.lo, 52);
        };
        // a stretch of the row a thread
        const long long per = (n + NT - 1) / NT, i0 = min(tid * per, n), i1 = min(i0 + per, n);
        unsigned long long mine = 0, total = 0;
        for (int tries = 0; tries < 2; ++tries) {
            mine = 0;
            for (long long i = i0; i < i1; ++i) mine += left(i);
            total = block_sum(mine);
            if (total > 0 || whole) break;
            whole = true;
        }
        const unsigned long long before = block_scan(mine), target = fraction_of(u, total);
        if (tid == 0) s.token = -1;
        __syncthreads();
        if (total > 0 && mine > 0 && before <= target && target < before + mine) {
            unsigned long long c = before;
            for (long long i = i0; i < i1; ++i) {
                c += left(i);
                if (c > target) {
                    s.token = d.ids[p.eb + i];
                    s.lpx = d.logq[p.eb + i];
                    break;
                }
            }
        }
        __syncthreads();
        if (tid == 0) finish(t, s.token, s.lpx, bits);
    }
};

// log2 of the draft's total over the target's, by the fp32 sums, in the rows' units: S e^(M / T) over 2^R.
RL_DEVINL Lam rough_ratio(const VerRow& p, const VerRow& q) {
    auto rough = [](const VerRow& w) -> FF {
        const FF l = {log2f(w.S), 0.f};
        return w.plain ? ff_add(l, ff_add(ff_mul({w.M, 0.f}, w.c), {-w.R, 0.f})) : l;
    };
    const FF lam = ff_add(rough(q), ff_neg(rough(p)));
    const float whole = floorf(lam.hi);
    const FF f = ff_add(lam, {-whole, 0.f});
    Lam x;
    x.whole = static_cast<int>(whole);
    x.hi = floorf(f.hi * 2048.f) * (1.f / 2048.f);
    x.lo = __fadd_rn(__fsub_rn(f.hi, x.hi), f.lo);
    return x;
}

// A block a request: what is accepted, and the new token where no row of logits has to be summed up for it.
__global__ void __launch_bounds__(kDecideThreads, 2) decide_kernel(const __grid_constant__ VerArgs g) {
    extern __shared__ __align__(16) uint8_t raw[];
    VerShared<kDecideThreads>& s = *reinterpret_cast<VerShared<kDecideThreads>*>(raw);
    const rl_verify_args& a = g.a;
    const long long r = blockIdx.x;
    const int tid = threadIdx.x, V = static_cast<int>(a.V);
    Request<kDecideThreads> q{g, s, V, tid, tid & 31, tid >> 5};
    constexpr int kRows = kDecideThreads / 64;
    int bits = 0;
    bool table = false;
    wait_for_previous();
    let_next_start();
    long long t0 = a.cu_q[r], t1 = a.cu_q[r + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.T) {
        bits |= RL_STATUS_LENGTHS;
        t0 = t1 = 0;
    }
    // Row k of a stretch of the request: a warp its target, the next its draft (the last row has none).
    long long t = t0;
    bool going = t1 > t0;
    int at = 0;                                  // the row that the new token is drawn from, in the stretch
    while (going) {
        const long long mine = t + (q.warp >> 1);
        const int side = q.warp & 1;
        __syncthreads();
        if (mine < t1) {
            VerRow x{};
            int rb = 0;
            float lp = -INFINITY;
            const bool candidate = mine + 1 < t1;
            if (candidate || side == 0) {
                const int token = candidate ? a.step_tokens[mine + 1] : -1;
                x = q.row_at(side, mine, rb);
                if (candidate) {
                    if (x.mode == kDistNone) rb |= RL_STATUS_EMPTY_ROW;
                    if (token < 0 || token >= V) rb |= RL_STATUS_ID_RANGE;
                    else lp = q.log2_prob(side, x, token, rb);
                }
            }
            if (q.lane == 0) {
                s.rows[q.warp] = x;
                s.lp[q.warp] = lp;
                s.bits[q.warp] = rb;
            }
        }
        __syncthreads();
        const int n = static_cast<int>(min(static_cast<long long>(kRows), t1 - t));
        int k = 0;
        for (; k < n; ++k) {
            if (t + k + 1 >= t1) {               // the last row
                going = false;
                bits |= s.bits[2 * k];
                break;
            }
            bits |= s.bits[2 * k] | s.bits[2 * k + 1];
            const int x = a.step_tokens[t + k + 1];
            const float u = unit_of(a.u[t + k], bits), lp = s.lp[2 * k], lu = log2f(u) + s.lp[2 * k + 1];
            // The bound of the difference's error: two totals of fp32 exponentials (2^-22 each, arguments' roundings, 60 additions)
            // and the logs' own roundings
            const float bound = 0x1p-15f + 0x1p-21f * (fabsf(lp) + fabsf(lu));
            float l = lp * kLn2;
            int res;
            if (lp == -INFINITY) res = 1;
            else if (lu == -INFINITY) res = 0;
            else res = lu < lp - bound ? 0 : lu > lp + bound ? 1 : 2;
            if (res == 2) {                      // too near: with counted totals and 64-bit logs
                if (!table) fill_table(s.tab, tid, kDecideThreads);
                table = true;
                const int steps = (V + kVerStep * kVerPart - 1) / (kVerStep * kVerPart);
                for (int sd = 0; sd < 2; ++sd) {
                    VerRow& w = s.rows[2 * k + sd];
                    if (w.mode != kDistDense) continue;
                    __syncthreads();
                    int first = q.warp;
                    const unsigned long long sum = sum_steps(logits_of(g.side[sd].d, w), &w, V, 0, steps, first, {kDecideThreads / 32, nullptr}, nullptr, smem_addr(s.tab));
                    const unsigned long long total = q.block_sum(q.lane == 0 ? sum : 0ull);
                    if (tid == 0) w.total = total;
                }
                __syncthreads();
                if (tid == 0) {
                    const double dp = q.ln_prob(0, s.rows[2 * k], x, bits), dq = q.ln_prob(1, s.rows[2 * k + 1], x, bits);
                    s.flag = static_cast<double>(u) * exp(dq) < exp(dp) ? 0 : 1;
                    s.lpx = static_cast<float>(dp);
                }
                __syncthreads();
                res = s.flag;
                l = s.lpx;
            }
            if (res != 0) {
                going = false;
                break;
            }
            if (tid == 0) {
                a.tokens[t + k] = x;
                if (a.logq) a.logq[t + k] = l;
            }
        }
        t += k;
        at = k;
    }
    if (tid == 0) {
        a.accepted[r] = static_cast<int>(t - t0);
        if (a.keep_lens) a.keep_lens[r] = (a.ctx_lens ? a.ctx_lens[r] : 0) + static_cast<int>(t1 > t0 ? t - t0 + 1 : 0);
    }
    bool rest = false;
    if (t1 > t0) {
        const float u = unit_of(a.u_next[r], bits);
        const bool refused = t + 1 < t1;
        if (tid == 0) {
            s.draw.t = t;
            s.draw.u = u;
            s.draw.row[0] = s.rows[2 * at];
            s.draw.row[1] = s.rows[2 * at + 1];
            if (!refused) s.draw.row[1].mode = kDistNone;
            if (s.draw.row[0].mode == kDistDense && s.draw.row[1].mode == kDistDense) s.draw.lam = rough_ratio(s.draw.row[0], s.draw.row[1]);
        }
        __syncthreads();
        const int p = s.draw.row[0].mode, d = s.draw.row[1].mode;
        if (p == kDistDense || (p == kDistSupport && d == kDistDense)) rest = true;
        else if (p == kDistSupport) q.draw_support(t, u, bits);
        // (all of the target on one token: it is what is left, or what there is)
        else if (tid == 0) q.finish(t, p == kDistPoint ? s.draw.row[0].at : -1, 0.f, bits);
    }
    if (g.draws) {
        __syncthreads();
        if (rest) {
            const int words = static_cast<int>(sizeof(VerDraw) / 8);
            if (tid < words) reinterpret_cast<unsigned long long*>(g.draws + r)[tid] = reinterpret_cast<const unsigned long long*>(&s.draw)[tid];
            if (tid == 0) g.todo[atomicAdd(g.n_todo, 1)] = static_cast<int>(r);      // (whose order no result depends on)
        } else if (tid == 0) {
            g.draws[r].t = -1;
        }
    }
    set_status(g.status, bits);
}

// ---- 3. sums ---------------------------------------------------------------------------------
// A block takes as many steps as another, its warps one after another as they get done (with the same number of steps for each warp,
// 128 requests take 3 us longer: a multiprocessor's warps do not end together).  One block of 1024 threads (64 registers) a
// multiprocessor; of 768 1 us longer, two of 512 6 us longer.
__global__ void __launch_bounds__(kSumThreads, kSumBlocks) sum_kernel(const __grid_constant__ VerArgs g) {
    __shared__ float2 tab[2048];
    __shared__ int next;
    const int V = static_cast<int>(g.a.V), steps = g.steps;
    fill_table(tab, threadIdx.x, kSumThreads);
    if (threadIdx.x == 0) next = kSumThreads / 32;
    __syncthreads();
    wait_for_previous();
    let_next_start();
    const long long units = static_cast<long long>(*g.n_todo) * steps, first = units * blockIdx.x / gridDim.x;
    const int n = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - first);
    for (int k = threadIdx.x >> 5; k < n;) {
        const long long i = (first + k) / steps;
        const int base = static_cast<int>(first - i * steps), end = min(n, steps - base), r = g.todo[i];      // (the request's step 0 is -base of the block's)
        const VerDraw& d = g.draws[r];
        VerStep* out = g.sums + static_cast<long long>(r) * steps;
        const bool p = d.row[0].mode == kDistDense, q = d.row[1].mode == kDistDense;
        if (p && q) sum_both(logits_of(g.side[0].d, d.row[0]), &d.row[0], logits_of(g.side[1].d, d.row[1]), &d.row[1], d.lam, V, base, end, k, {0, &next}, out, smem_addr(tab));
        else sum_steps(logits_of(g.side[p ? 0 : 1].d, d.row[p ? 0 : 1]), &d.row[p ? 0 : 1], V, base, end, k, {0, &next}, out, smem_addr(tab));
    }
}

// ---- 4. the token ----------------------------------------------------------------------------
// Latency: the parts' sums of a row of 151,936 are 19 KB, and loads, block sums, two logs and the scan of one part follow on one
// another (16 us by itself, some 7 of them after the sums).
// A block a request: the new token from rows of logits.
struct Pick : Request<kPickThreads> {
    unsigned long long* cs;       // sums of the row's parts
    VerStep* sums;                // of its steps
    int steps;

    // The parts' sums into cs; returns the total.
    RL_DEVINL unsigned long long take_parts() {
        unsigned long long v = 0;
        for (int k = tid; k < steps; k += kPickThreads) {
            const ulonglong2* x = reinterpret_cast<const ulonglong2*>(sums[k].part);
            const ulonglong2 a = x[0], b = x[1];
            ulonglong2* to = reinterpret_cast<ulonglong2*>(cs + k * kVerStep);
            to[0] = a;
            to[1] = b;
            v += (a.x + a.y) + (b.x + b.y);
        }
        return block_sum(v);
    }
    // What is left of a token of a dense target, z its logit and y the draft's, in the target's units.
    RL_DEVINL unsigned long long left_at(float z, float y, int j, bool whole, int& bits) {
        const VerRow& p = s.draw.row[0];
        const VerRow& q = s.draw.row[1];
        // (by exponents: where the logits' spacing is worth several of them, their bounds as logits would be rounded past a logit)
        if (!(exponent_of(z, p, 0.f) >= kLeastExp)) return 0ull;
        FF v = weight_of(z, p, 0.f, 0.f, s.tab);
        if (!whole && q.mode == kDistDense) {
            const float lam_hi = rintf(s.lam.hi * 2048.f) * (1.f / 2048.f), lam_lo = (s.lam.hi - lam_hi) + s.lam.lo;
            const float e = exponent_of(y, q, lam_hi);
            if (e > 0.75f) return 0ull;          // (the target's weight is at most 1)
            if (e >= kLeastExp) v = ordered(left_of(v, weight_of(y, q, lam_hi, lam_lo, s.tab)));
            return fixed_of(v.hi, v.lo, p.prec);
        }
        const unsigned long long w = fixed_of(v.hi, v.lo, p.prec);
        if (whole || q.mode == kDistNone) return w;
        return w - taken(w, q.mode == kDistPoint ? (j == q.at ? 0.f : -INFINITY) : support_at(1, q, j, bits));
    }
    // What a draft's probability e^lq takes off a weight w: the smaller of the two.
    RL_DEVINL unsigned long long taken(unsigned long long w, float lq) {
        if (!(lq > -INFINITY)) return 0ull;
        const FF e = exp_table({lq, 0.f});
        const double x = (static_cast<double>(e.hi) + static_cast<double>(e.lo)) * static_cast<double>(s.draw.row[0].total);
        return x >= static_cast<double>(w) ? w : static_cast<unsigned long long>(__double2ll_rn(x));
    }

    // What is left of a dense target beside a dense draft, by parts in cs; returns the total, and sets both rows' totals.
    RL_DEVINL unsigned long long left_of_rows() {
        VerRow& p = s.draw.row[0];
        VerRow& q = s.draw.row[1];
        ulonglong2 x = make_ulonglong2(0, 0);
        for (int k = tid; k < steps; k += kPickThreads) {
            x.x += sums[k].p;
            x.y += sums[k].q;
        }
        x.x = warp_sum(x.x);
        x.y = warp_sum(x.y);
        if (lane == 0) {
            s.red[warp] = x.x;
            s.red2[warp] = x.y;
        }
        __syncthreads();
        if (warp == 0) {
            x = make_ulonglong2(0, 0);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                x.x += s.red[k];
                x.y += s.red2[k];
            }
            // the logs of both, a lane each, in the rows' units; log2 of the draft's total over the target's as a pair
            const Lam lam = s.draw.lam;
            const FF l = ln_of(lane == 0 ? x.x : x.y, lane == 0 ? p.prec : q.prec);
            const FF lq = {__shfl_sync(0xffffffffu, l.hi, 1), __shfl_sync(0xffffffffu, l.lo, 1)};
            if (lane == 0) {
                FF d = ff_add(ff_mul(ff_add(lq, ff_neg(l)), {kLog2eHi, kLog2eLo}), {lam.hi, lam.lo});        // log2 and the part that the sum left out
                s.lam = d;
                d = ff_add(d, {-static_cast<float>(lam.whole), 0.f});
                d = ff_add(d, {-lam.hi, -lam.lo});
                s.turn = (d.hi + d.lo) * kLn2;
                p.total = x.x;
                q.total = x.y;                   // (less that part: only the ratio is read of it)
            }
        }
        __syncthreads();
        const float turn = s.turn * power_of_2(p.prec);
        unsigned long long v = 0;
        for (int k = tid; k < steps; k += kPickThreads)
#pragma unroll
            for (int j = 0; j < kVerStep; ++j) {
                const long long y = static_cast<long long>(sums[k].part[j]) + __float2ll_rn(sums[k].drop[j] * turn);
                cs[k * kVerStep + j] = y > 0 ? static_cast<unsigned long long>(y) : 0ull;
                v += cs[k * kVerStep + j];
            }
        return block_sum(v);
    }

    RL_DEVINL void draw_dense(long long t, float u, int& bits) {
        const VerRow& p = s.draw.row[0];
        const VerRow& q = s.draw.row[1];
        const rl_dist& dp = g.side[0].d;
        const rl_dist& dq = g.side[1].d;
        bool whole = q.mode == kDistNone;
        unsigned long long total;
        if (q.mode == kDistDense) {
            total = left_of_rows();
        } else {
            total = take_parts();
            if (tid == 0) s.draw.row[0].total = total;
            __syncthreads();
        }
        if (q.mode == kDistPoint || q.mode == kDistSupport) {
            // the draft's tokens off their parts
            const long long n = q.mode == kDistPoint ? 1 : q.ee - q.eb;
            for (long long i = tid; i < n; i += kPickThreads) {
                const int j = q.mode == kDistPoint ? q.at : dq.ids[q.eb + i];
                if (j < 0 || j >= V) {
                    if (q.mode == kDistSupport) bits |= RL_STATUS_ID_RANGE;
                    continue;
                }
                float lq = 0.f;
                if (q.mode == kDistSupport) {
                    lq = dq.logq[q.eb + i];
                    if (!(lq <= 1e-6f)) bits |= RL_STATUS_LOGQ;
                    if (!(lq < INFINITY)) lq = -INFINITY;
                    if (i > 0 && dq.ids[q.eb + i - 1] >= j) bits |= RL_STATUS_ROW_ORDER;
                }
                const unsigned long long w = left_at(logit_at(dp, p.dtype, p.row, j), 0.f, j, true, bits);
                atomicAdd(&cs[j / kVerPart], 0ull - taken(w, lq));
            }
            __syncthreads();
            // (a part's sum and its tokens' weights are rounded apart)
            unsigned long long v = 0;
            for (int i = tid; i < steps * kVerStep; i += kPickThreads) {
                if (static_cast<long long>(cs[i]) < 0) cs[i] = 0;
                v += cs[i];
            }
            total = block_sum(v);
        }
        if (total > 0 && !whole) {
            if (search(t, fraction_of(u, total), false, bits)) return;
            total = 0;
        }
        if (!whole) {                            // nothing is left: from the target
            whole = true;
            int first = warp;
            sum_steps(logits_of(dp, p), &s.draw.row[0], V, 0, steps, first, {kWarps, nullptr}, sums, smem_addr(s.tab));
            __syncthreads();
            total = take_parts();
        }
        if (total > 0) search(t, fraction_of(u, total), true, bits);
        else if (tid == 0) finish(t, -1, 0.f, bits);
    }
    // The part in which the number falls, then its token.  False if nothing is left of any token of the part: what was summed up
    // is the sums' own error (p and q are the same to their accuracy).
    RL_DEVINL bool search(long long t, unsigned long long want, bool whole, int& bits) {
        const int n = steps * kVerStep, per = (n + kPickThreads - 1) / kPickThreads;
        unsigned long long v = 0;
        if (tid == 0) s.flag = 1;
        __syncthreads();
        for (int j = 0; j < per; ++j) v += tid * per + j < n ? cs[tid * per + j] : 0ull;
        unsigned long long c = block_scan(v);
        if (c <= want && want < c + v)
            for (int j = 0; j < per; ++j) {
                const unsigned long long x = cs[tid * per + j];
                if (want < c + x) {
                    s.token = tid * per + j;
                    s.unit = want - c;
                    break;
                }
                c += x;
            }
        __syncthreads();
        if (warp == 0) token_of(t, whole, bits);
        __syncthreads();
        return s.flag != 0;
    }
    RL_DEVINL void token_of(long long t, bool whole, int& bits) {
        const int i0 = s.token * kVerPart + lane * 4;
        const unsigned long long rest = s.unit;
        const VerRow& p = s.draw.row[0];
        const VerRow& q = s.draw.row[1];
        unsigned long long w[4], mine = 0;
        int last = -1, likely = -1;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const float z = i0 + j < V ? logit_at(g.side[0].d, p.dtype, p.row, i0 + j) : -INFINITY;
            const float y = i0 + j < V && !whole && q.mode == kDistDense ? logit_at(g.side[1].d, q.dtype, q.row, i0 + j) : -INFINITY;
            w[j] = z > -INFINITY ? left_at(z, y, i0 + j, whole, bits) : 0ull;
            mine += w[j];
            if (w[j] > 0) last = j;
            if (z > -INFINITY) likely = j;
        }
        unsigned long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, incl > rest), some = __ballot_sync(0xffffffffu, last >= 0),
                       any = __ballot_sync(0xffffffffu, likely >= 0);
        if (!whole && !some) {
            if (lane == 0) s.flag = 0;
            return;
        }
        int at = last >= 0 ? last : likely;
        int src;
        if (hit) {
            src = __ffs(hit) - 1;
            unsigned long long c2 = incl - mine;
            bool got = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                c2 += w[j];
                if (!got && c2 > rest) {
                    got = true;
                    at = j;
                }
            }
        } else {                // the number met the part's sum to the last place
            src = 31 - __clz(some ? some : any | 1u);
        }
        if (lane == src) {
            const int token = i0 + max(at, 0);
            finish(t, token, static_cast<float>(ln_prob(0, p, token, bits)), bits);
        }
    }
};

__global__ void __launch_bounds__(kPickThreads, 2) pick_kernel(const __grid_constant__ VerArgs g) {
    extern __shared__ __align__(16) uint8_t raw[];
    VerShared<kPickThreads>& s = *reinterpret_cast<VerShared<kPickThreads>*>(raw);
    const long long r = blockIdx.x;
    const int tid = threadIdx.x, V = static_cast<int>(g.a.V);
    Pick q{{g, s, V, tid, tid & 31, tid >> 5}, reinterpret_cast<unsigned long long*>(raw + (sizeof(VerShared<kPickThreads>) + 15) / 16 * 16), g.sums + r * g.steps, g.steps};
    int bits = 0;
    fill_table(s.tab, tid, kPickThreads);
    wait_for_previous();
    const int words = static_cast<int>(sizeof(VerDraw) / 8);
    if (tid < words) reinterpret_cast<unsigned long long*>(&s.draw)[tid] = reinterpret_cast<const unsigned long long*>(g.draws + r)[tid];
    __syncthreads();
    if (s.draw.t < 0) return;
    if (s.draw.row[0].mode == kDistDense) {
        q.draw_dense(s.draw.t, s.draw.u, bits);
    } else {
        const unsigned long long total = q.take_parts();
        if (tid == 0) s.draw.row[1].total = total;
        __syncthreads();
        q.draw_support(s.draw.t, s.draw.u, bits);
    }
    set_status(g.status, bits);
}

// ---- host ------------------------------------------------------------------------------------
static VerArgs verify_view(void* ws, const rl_verify_args* a, int32_t* status, size_t* bytes) {
    VerArgs g{};
    g.a = *a;
    g.status = status;
    g.sure = !a->draft.logits && !a->draft.offsets;
    g.side[0].d = a->target;
    g.side[0].dtype = a->target_dtype;
    g.side[1].d = a->draft;
    g.side[1].dtype = a->draft_dtype;
    Carve cv(ws);
    for (auto& s : g.side)
        if (s.d.logits) {
            const int64_t e = s.dtype == RL_DTYPE_F32 ? 4 : 8, chunk = kChunkPacks * 32 * e;
            s.nc = static_cast<int>((a->V + e - 1 + chunk - 1) / chunk);
            s.part = cv.take<float2>(static_cast<size_t>(a->T) * s.nc);
        }
    g.steps = static_cast<int>((a->V + kVerStep * kVerPart - 1) / (kVerStep * kVerPart));
    if (a->target.logits || a->draft.logits) {
        g.draws = cv.take<VerDraw>(static_cast<size_t>(a->R));
        g.sums = cv.take<VerStep>(static_cast<size_t>(a->R) * g.steps);
        g.todo = cv.take<int32_t>(static_cast<size_t>(a->R));
        g.n_todo = cv.take<int32_t>(1);
    }
    if (bytes) *bytes = align_up(cv.off, 256);
    return g;
}

size_t verify_ws_bytes(const rl_verify_args* a) {
    size_t b = 0;
    verify_view(nullptr, a, nullptr, &b);
    return b;
}

int verify_impl(const rl_verify_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    VerArgs g = verify_view(ws, a, status, nullptr);
    ProfScope prof(RL_PROF_OTHER, stream);
    int launches = 0;
    if (a->T > 0) {
        // (two chunks share the look-up of their row, 8 us less for 128 requests; of few rows each warp gets one)
        const long long cap = 3ll * num_sms(), chunks = a->T * (g.side[0].nc + g.side[1].nc);
        g.group = chunks > cap * (kChunkThreads / 32) ? 2 : 1;
        const long long units = a->T * ((g.side[0].nc + g.group - 1) / g.group + (g.side[1].nc + g.group - 1) / g.group), fill = (a->T + kChunkThreads - 1) / kChunkThreads;
        long long blocks = (units + kChunkThreads / 32 - 1) / (kChunkThreads / 32);
        if (blocks < fill) blocks = fill;
        if (blocks > cap) blocks = cap;
        chunk_kernel<<<static_cast<unsigned>(blocks), kChunkThreads, 0, stream>>>(g);
        ++launches;
    }
    if (a->R > 0) {
        static std::atomic<uint64_t> decide{0}, pick{0};
        const int smem = static_cast<int>(sizeof(VerShared<kDecideThreads>));
        if (!allow_smem(decide_kernel, smem, decide)) return RL_ERR_CUDA;
        int rc = launch_after(decide_kernel, dim3(static_cast<unsigned>(a->R)), kDecideThreads, static_cast<size_t>(smem), launches > 0, stream, g);
        if (rc != RL_OK) return rc;
        ++launches;
        if (g.draws && a->T > 0) {
            const long long most = static_cast<long long>(kSumBlocks) * num_sms(), units = a->R * g.steps;
            rc = launch_after(sum_kernel, dim3(static_cast<unsigned>(units < most ? units : most)), kSumThreads, 0, true, stream, g);
            if (rc != RL_OK) return rc;
            const size_t fixed = (sizeof(VerShared<kPickThreads>) + 15) / 16 * 16, longest = ((size_t(1) << 20) / kVerPart + kVerStep) * 8;
            if (!allow_smem(pick_kernel, static_cast<int>(fixed + longest), pick)) return RL_ERR_CUDA;
            rc = launch_after(pick_kernel, dim3(static_cast<unsigned>(a->R)), kPickThreads, fixed + static_cast<size_t>(g.steps) * kVerStep * 8, true, stream, g);
            if (rc != RL_OK) return rc;
            launches += 2;
        }
    }
    count_launch(launches);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // namespace rl
