// Sampling with temperature, top-k, top-p and min-p from given random numbers, and the
// sampler support as CSR rows (the head's rl_support).
//
// The token of a draw u is the first whose cumulative weight, in index order, passes u times
// the total: a sum over up to the whole vocabulary decides which of two neighbours it is, so
// fp32 sums would give another token every few thousand draws.  Weights and sums are therefore
// carried to about 2^-37 of the largest weight:
//   w = 2^p, p = (z - ref) log2(e) / T as a float pair (p, e);  p = n + j/2048 + r, exactly;
//   2^(j/2048) = hi (1 + rho) from a table, 2^r - 1 = r ln2 + (r ln2)^2 / 2 (the next term is
//   below 2^-40), so w = 2^n hi (1 + rho + ...) is the unevaluated pair (2^n hi, v).
// fp64 would do the same at a fiftieth of the rate on this part.
//
//  1. stats_kernel   one warp per 1024 logits: the largest of each 128, and where a row needs
//                    it the sum of weights, with a reference of the chunk's own so that no
//                    pass for the row's maximum comes first.  The only pass over all logits.
//  2. select_kernel  one block a row: the kept set as a threshold (key, index), by collecting
//                    the candidates into shared memory and sorting them when a bound from the
//                    128-wide maxima shows that few can matter, else after a histogram that
//                    brackets the border; then the weights of each chunk's kept tokens, and
//                    each draw by a search over the chunks and a scan of one chunk.
//                    Whole rows (no cut) take the chunk sums of 1.  Sums over chunks of kept
//                    tokens are integers (units of 2^-50): their order does not matter.
//  3. emit_kernel    the support rows, one warp a chunk.
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "ff.cuh"
#include "internal.h"

#include <cuda_fp16.h>

namespace rl {

constexpr int kChunk = 1024;               // logits of one warp step
constexpr int kSub = 128;                  // ... of one 32-lane load
constexpr int kSubs = kChunk / kSub;
constexpr int kListCap = 4096;             // candidates sorted in shared memory
constexpr int kBins = 2048;
constexpr float kWholeRef = 1900.f;        // |max * log2(e) / T| up to which a chunk needs no reference
constexpr float kLog2eHi = 1.44269502162933349609f, kLog2eLo = 1.92596299112661746887e-8f;
constexpr double kUnit = 1125899906842624.0;   // 2^50

// 2^(i/2048), i = 0..31, as float pairs
static __device__ __constant__ float kFine2Hi[32] = {
    1.000000000e+00f, 1.000338554e+00f, 1.000677109e+00f, 1.001015902e+00f, 1.001354694e+00f, 1.001693726e+00f,
    1.002032757e+00f, 1.002371907e+00f, 1.002711296e+00f, 1.003050685e+00f, 1.003390193e+00f, 1.003729939e+00f,
    1.004069686e+00f, 1.004409552e+00f, 1.004749537e+00f, 1.005089641e+00f, 1.005429864e+00f, 1.005770206e+00f,
    1.006110668e+00f, 1.006451249e+00f, 1.006791949e+00f, 1.007132769e+00f, 1.007473707e+00f, 1.007814765e+00f,
    1.008155942e+00f, 1.008497119e+00f, 1.008838534e+00f, 1.009180069e+00f, 1.009521723e+00f, 1.009863377e+00f,
    1.010205269e+00f, 1.010547161e+00f};
static __device__ __constant__ float kFine2Lo[32] = {
    0.000000000e+00f, -4.632964234e-08f, 2.192841819e-08f, -3.360561251e-08f, 2.552565270e-08f, -3.905755364e-08f,
    1.110217429e-08f, 5.683439142e-08f, -2.103134022e-08f, 1.596242782e-08f, 4.864528691e-08f, -4.215315741e-08f,
    -1.797542026e-08f, 2.008129441e-09f, 1.783642567e-08f, 2.954841349e-08f, 3.718305308e-08f, 4.077931948e-08f,
    4.037620016e-08f, 3.601268972e-08f, 2.772780583e-08f, 1.556056972e-08f, -4.499763340e-10f, -2.026478008e-08f,
    -4.384477847e-08f, 4.805839993e-08f, 1.706526653e-08f, -1.757578438e-08f, -5.582563389e-08f, 2.156413892e-08f,
    -2.378589947e-08f, 4.658198804e-08f};

struct ChunkStat {
    float max;
    int ref;            // the sum is in units of 2^ref; INT_MIN: of the weight of `max`
    double sum;
};
struct RowRec {
    float M;            // the row's largest logit
    FF inv_t;           // 1 / T
    FF ln_w;            // ln of the kept weights' sum, relative to M's
    uint32_t key;       // kept: key(z) > key, or equal and index <= tie
    int tie;
    int mode;
};
enum { kRowEmpty = 0, kRowWhole = 1, kRowCut = 2 };

struct SampleArgs {
    rl_sample_args a;
    int32_t* status;
    int nc, ns;              // chunks, 128-wide parts of a row
    ChunkStat* stat;         // [N, nc]
    float* submax;           // [N, ns]
    int* ccnt;               // [N, nc] kept tokens of each chunk
    int* count;              // [N] entries of the support row
    RowRec* rec;             // [N]
    unsigned* done;          // rows finished (back to zero at the end of a call)
};

struct Knobs {
    float T, p, mp;
    int k;                   // 0 < k < V, or V
    bool greedy, cut, total; // total: the sum over all logits is needed
    int bits;
};
RL_DEVINL Knobs load_knobs(const rl_sample_args& a, long long r) {
    Knobs q;
    q.bits = 0;
    q.T = a.temperature ? a.temperature[r] : 1.f;
    q.p = a.top_p ? a.top_p[r] : 1.f;
    q.mp = a.min_p ? a.min_p[r] : 0.f;
    q.k = a.top_k ? a.top_k[r] : 0;
    if (q.k <= 0 || q.k > a.V) q.k = static_cast<int>(a.V);
    q.greedy = q.T == 0.f;
    if (!(q.T >= 0.f) || !(q.T <= FLT_MAX) || (q.T > 0.f && q.T < 4.f * FLT_MIN)) {
        q.greedy = true;
        q.bits |= RL_STATUS_KNOB;
    }
    if (q.p != q.p || q.mp != q.mp) {
        q.bits |= RL_STATUS_KNOB;
        if (q.p != q.p) q.p = 1.f;
        if (q.mp != q.mp) q.mp = 0.f;
    }
    q.mp = fminf(fmaxf(q.mp, 0.f), 1.f);
    q.cut = q.greedy || q.k < a.V || q.p < 1.f || q.mp > 0.f;
    q.total = !q.greedy && q.k == a.V && q.mp == 0.f;
    return q;
}

// log2(e) / T as a float pair
RL_DEVINL FF scale_of(float T) {
    const float h = kLog2eHi / T;
    return {h, (fmaf(-h, T, kLog2eHi) + kLog2eLo) / T};
}
RL_DEVINL FF inv_of(float T) {
    const float h = 1.f / T;
    return {h, fmaf(-h, T, 1.f) / T};
}

// Order of floats as unsigned numbers (-0 does not occur: loads add +0).
RL_DEVINL uint32_t key_of(float z) {
    const uint32_t b = __float_as_uint(z);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
RL_DEVINL float z_of(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

RL_DEVINL float to_f(float x) { return x; }
RL_DEVINL float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
RL_DEVINL float to_f(__half x) { return __half2float(x); }

// Four logits from element i on; past the row's end -inf.  NaN and +inf become -inf (`bad`).
template <typename T, bool kVec>
RL_DEVINL void load4(const T* row, int i, int V, float (&z)[4], bool& bad) {
    if (kVec && i + 4 <= V) {
        if constexpr (sizeof(T) == 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(row + i));
            z[0] = q.x; z[1] = q.y; z[2] = q.z; z[3] = q.w;
        } else {
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + i));
            T t[4];
            memcpy(t, &q, 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = to_f(t[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = i + j < V ? to_f(row[i + j]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (!(z[j] < INFINITY)) {
            bad = true;
            z[j] = -INFINITY;
        }
        z[j] += 0.f;
    }
}

// Table entry j: bits of 2^(j/2048) less j << 12 (so that adding the phase's bits gives the
// scaled value), and the relative error of that float.
RL_DEVINL void fill_table(float2* tab, int tid, int threads) {
    for (int j = tid; j < 2048; j += threads) {
        const FF v = ff_mul({kExp2Hi[j >> 5], kExp2Lo[j >> 5]}, {kFine2Hi[j & 31], kFine2Lo[j & 31]});
        tab[j] = make_float2(__uint_as_float(__float_as_uint(v.hi) - (static_cast<uint32_t>(j) << 12)), v.lo / v.hi);
    }
}
// 2^(p + e - ref) as hi + v, for p - ref in [-66, 1] and magic = 6144 - ref: 6144 + x has
// 2^-11 as its last place, so the sum's bits are 0x45C00000 + 2048 n + j.
RL_DEVINL void weight_pair(float p, float e, float magic, const float2* tab, float& hi, float& v) {
    const float t = __fadd_rn(p, magic);
    const float r = __fadd_rn(__fsub_rn(p, __fsub_rn(t, magic)), e);
    const uint32_t tb = __float_as_uint(t);
    const float2 q = tab[tb & 2047u];
    hi = __uint_as_float(__float_as_uint(q.x) + (tb << 12));
    v = hi * fmaf(r, fmaf(r, 0.24022650695910072f, 0.69314718055994531f), q.y);
}
// p, e of (z - m) * c
RL_DEVINL void phase_rel(float z, float m, FF c, float& p, float& e) {
    const FF d = two_sum(z, -m);
    p = __fmul_rn(d.hi, c.hi);
    e = fmaf(d.lo, c.hi, fmaf(d.hi, c.lo, fmaf(d.hi, c.hi, -p)));
}
// The weight of z relative to M in units of 2^-50; `zlow` = M - 64 / c, at least
// -FLT_MAX: below it the weight is 0 (M itself where the difference is lost).
RL_DEVINL unsigned long long weight_fixed(float z, float M, FF c, float zlow, const float2* tab) {
    if (!(z >= zlow)) return 0ull;
    float p, e, hi, v;
    phase_rel(z, M, c, p, e);
    weight_pair(p, e, 6144.f, tab, hi, v);
    const float wh = __fadd_rn(hi, v), wl = __fsub_rn(v, __fsub_rn(wh, hi));
    if (!(wh < 2.f)) return 0ull;             // differences past the range of floats
    const uint32_t b = __float_as_uint(wh);
    const int sh = static_cast<int>(b >> 23) - 127 - 23 + 50;          // the 24-bit significand times 2^sh
    const unsigned long long m = (b & 0x7fffffu) | 0x800000u;
    const unsigned long long w = sh >= 0 ? m << sh : (sh > -25 ? (m + (1ull << (-sh - 1))) >> -sh : 0ull);
    return w + static_cast<long long>(__float2int_rn(wl * 1125899906842624.f));
}
// ln q of a token
RL_DEVINL float log_q(float z, const RowRec& r) {
    const FF d = two_sum(z, -r.M);
    const FF p = two_prod(d.hi, r.inv_t.hi);
    const float e = fmaf(d.lo, r.inv_t.hi, fmaf(d.hi, r.inv_t.lo, p.lo));
    const FF s = two_sum(p.hi, -r.ln_w.hi);
    return s.hi + (s.lo + (e - r.ln_w.lo));
}

// ---- 1. chunk statistics -------------------------------------------------------------
constexpr int kStatThreads = 256;

template <typename T, bool kVec>
__global__ void __launch_bounds__(kStatThreads) stats_kernel(const SampleArgs g) {
    __shared__ float2 tab[2048];
    const rl_sample_args& a = g.a;
    fill_table(tab, threadIdx.x, kStatThreads);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int V = static_cast<int>(a.V);
    const long long warps = static_cast<long long>(gridDim.x) * (kStatThreads / 32);
    const long long units = a.N * g.nc;
    bool bad = false;
    for (long long id = static_cast<long long>(blockIdx.x) * (kStatThreads / 32) + (threadIdx.x >> 5); id < units; id += warps) {
        const long long r = id / g.nc;
        const int c = static_cast<int>(id - r * g.nc);
        const T* row = static_cast<const T*>(a.logits) + r * a.row_stride;
        float z[kSubs][4];
#pragma unroll
        for (int s = 0; s < kSubs; ++s) load4<T, kVec>(row, c * kChunk + s * kSub + lane * 4, V, z[s], bad);
        uint32_t cmax = 0, mine = 0;
#pragma unroll
        for (int s = 0; s < kSubs; ++s) {
            const float m = fmaxf(fmaxf(z[s][0], z[s][1]), fmaxf(z[s][2], z[s][3]));
            const uint32_t k = __reduce_max_sync(0xffffffffu, key_of(m));
            cmax = max(cmax, k);
            if (lane == s) mine = k;
        }
        if (lane < kSubs && c * kSubs + lane < g.ns) g.submax[r * g.ns + c * kSubs + lane] = z_of(mine);
        const float m = z_of(cmax);
        const Knobs q = load_knobs(a, r);
        ChunkStat st{m, 0, 0.0};
        if (q.total && m > -INFINITY) {
            const FF cs = scale_of(q.T);
            const float pm = m * cs.hi;
            uint32_t top_sum = 0;
            int low_sum = 0;
            float S = 0.f, L = 0.f;
            // hi part on a grid of 2^-18 (sums of 32 values up to 1 are exact), the rest apart
            auto add = [&](float hi, float v) {
                const float wh = __fadd_rn(hi, v), wl = __fsub_rn(v, __fsub_rn(wh, hi));
                const float top = __fsub_rn(__fadd_rn(wh, 48.f), 48.f);
                S += top;
                L += __fsub_rn(wh, top);
                L += wl;
            };
            if (fabsf(pm) < kWholeRef) {
                const float ref = ceilf(pm), magic = 6144.f - ref, zlow = fmaxf((ref - 64.f) / cs.hi, -FLT_MAX);
                st.ref = static_cast<int>(ref);
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = fmaxf(z[s][j], zlow);
                        const float p = __fmul_rn(x, cs.hi);
                        const float e = fmaf(x, cs.lo, fmaf(x, cs.hi, -p));
                        float hi, v;
                        weight_pair(p, e, magic, tab, hi, v);
                        const bool in = z[s][j] >= zlow;
                        add(in ? hi : 0.f, in ? v : 0.f);
                    }
            } else {
                const float zlow = fmaxf(m - 64.f / cs.hi, -FLT_MAX);
                st.ref = INT_MIN;
#pragma unroll
                for (int s = 0; s < kSubs; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = z[s][j] >= zlow;
                        float p, e, hi, v;
                        phase_rel(in ? z[s][j] : m, m, cs, p, e);
                        weight_pair(p, e, 6144.f, tab, hi, v);
                        add(in ? hi : 0.f, in ? v : 0.f);
                    }
            }
            top_sum = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(S * 262144.f));
            low_sum = __reduce_add_sync(0xffffffffu, __float2int_rn(L * 549755813888.f));
            st.sum = static_cast<double>(top_sum) * 3.814697265625e-06 + static_cast<double>(low_sum) * 1.8189894035458565e-12;
        }
        if (lane == 0) g.stat[r * g.nc + c] = st;
    }
    if (bad) set_status(g.status, RL_STATUS_NONFINITE);
}

// ---- 2. selection and draws ------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// How a logit lies to the bracket: above it, in it, or below.
struct Bracket {
    int mode;               // 0: everything in; 1: everything above; 2: linear bin b; 3: key >> shift == b
    float hi, scale;
    int shift;
    uint32_t b;
};
RL_DEVINL int linear_bin(float z, float hi, float scale) {
    return static_cast<int>(fminf((hi - z) * scale, static_cast<float>(kBins - 1)));
}
RL_DEVINL int place(const Bracket& k, float z, uint32_t key) {   // > 0 above, 0 in, < 0 below
    if (k.mode == 0) return 0;
    if (k.mode == 1) return 1;
    if (k.mode == 2) return static_cast<int>(k.b) - linear_bin(z, k.hi, k.scale);
    const uint32_t x = k.shift < 32 ? key >> k.shift : 0;
    return x > k.b ? 1 : x == k.b ? 0 : -1;
}

struct SelShared {
    unsigned long long red[kSelWarps];
    double redd[kSelWarps];
    float2 tab[2048];
    unsigned long long comp[kListCap];     // candidates: key << 32 | ~index
    unsigned long long wt[kListCap];       // their weights; the histogram before that
    unsigned n_list, bin_lo;
    unsigned long long bin_before, bin_inside;
    int pick;
    float fpick;
    RowRec rec;
    // then: unsigned long long / double cs[nc], int cnt[nc], int in[nc]
};

template <typename T>
RL_DEVINL T block_sum(T v, T* red) {                    // every thread gets the sum, in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T s = red[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; ++w) s += red[w];
    return s;
}
RL_DEVINL unsigned long long block_max(unsigned long long v, unsigned long long* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    unsigned long long s = red[0];
#pragma unroll
    for (int w = 1; w < kSelWarps; ++w) s = max(s, red[w]);
    return s;
}
// Exclusive block scan of one value a thread.
template <typename T>
RL_DEVINL T block_scan(T v, T* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T i = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T x = __shfl_up_sync(0xffffffffu, i, o);
        if (lane >= o) i += x;
    }
    __syncthreads();
    if (lane == 31) red[warp] = i;
    __syncthreads();
    T p = 0;
    for (int w = 0; w < warp; ++w) p += red[w];
    return p + i - v;
}

template <typename T, bool kVec>
struct Row {
    const SampleArgs& g;
    SelShared& s;
    unsigned long long* cs;      // [nc] kept weight of each chunk (units of 2^-50)
    int* cnt;                    // [nc] kept tokens
    int* in;                     // [nc] tokens in the bracket
    const T* row;
    const float* submax;
    int V, tid, lane, warp;
    float M, zlow;               // zlow: weights are 0 from here down
    FF c;
    uint32_t bkey;               // the set that selection starts from: key > bkey, or equal and
    int btie;                    // index <= btie

    RL_DEVINL unsigned long long weight(float z) const { return weight_fixed(z, M, c, zlow, s.tab); }

    // f(z, index) for every logit >= lo, a warp a chunk; after(chunk) once a chunk, by all lanes
    template <typename F, typename G>
    RL_DEVINL void each(float lo, F f, G after) {
        bool bad = false;
        for (int ch = warp; ch < g.nc; ch += kSelWarps) {
            const int n = min(kSubs, g.ns - ch * kSubs);
            for (int q = 0; q < n; ++q) {
                if (submax[ch * kSubs + q] < lo) continue;
                float z[4];
                const int i = ch * kChunk + q * kSub + lane * 4;
                load4<T, kVec>(row, i, V, z, bad);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (z[j] >= lo && z[j] > -INFINITY) f(z[j], i + j);
            }
            after(ch);
        }
    }
    RL_DEVINL bool in_base(uint32_t key, int i) const { return key > bkey || (key == bkey && i <= btie); }

    // One pass: weight and number of the logits above the bracket by chunk, those in it listed.
    RL_DEVINL void collect(const Bracket& k, float lo) {
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        unsigned long long acc = 0;
        int n = 0, inside = 0;
        each(lo, [&](float z, int i) {
                const uint32_t key = key_of(z);
                if (!in_base(key, i)) return;
                const int pl = place(k, z, key);
                if (pl > 0) {
                    acc += weight(z);
                    ++n;
                } else if (pl == 0) {
                    ++inside;
                    const unsigned at = atomicAdd(&s.n_list, 1u);
                    if (at < kListCap) s.comp[at] = (static_cast<unsigned long long>(key) << 32) | static_cast<uint32_t>(~i);
                }
            },
            [&](int ch) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
                n = __reduce_add_sync(0xffffffffu, n);
                inside = __reduce_add_sync(0xffffffffu, inside);
                if (lane == 0) {
                    cs[ch] = acc;
                    cnt[ch] = n;
                    in[ch] = inside;
                }
                acc = 0;
                n = inside = 0;
            });
        __syncthreads();
    }
    RL_DEVINL double sum_weight() {
        double v = 0.0;
        for (int ch = tid; ch < g.nc; ch += kSelThreads) v += static_cast<double>(cs[ch]);
        return block_sum(v, s.redd);
    }
    RL_DEVINL long long sum_int(const int* x) {
        long long v = 0;
        for (int ch = tid; ch < g.nc; ch += kSelThreads) v += x[ch];
        return static_cast<long long>(block_sum(static_cast<unsigned long long>(v), s.red));
    }
    // The list in descending order (ties: the lower index first), and its weights.
    RL_DEVINL void sort_list(int n) {
        int m = 32;
        while (m < n) m <<= 1;
        for (int i = n + tid; i < m; i += kSelThreads) s.comp[i] = 0;
        __syncthreads();
        for (int size = 2; size <= m; size <<= 1)
            for (int step = size >> 1; step > 0; step >>= 1) {
                for (int t = tid; t < m / 2; t += kSelThreads) {
                    const int i = 2 * t - (t & (step - 1)), j = i + step;
                    const unsigned long long x = s.comp[i], y = s.comp[j];
                    if ((x < y) == ((i & size) == 0)) {
                        s.comp[i] = y;
                        s.comp[j] = x;
                    }
                }
                __syncthreads();
            }
        for (int i = tid; i < n; i += kSelThreads) s.wt[i] = weight(z_of(static_cast<uint32_t>(s.comp[i] >> 32)));
        __syncthreads();
    }
    // How many of the sorted list come before the sum (above + those before) reaches target.
    RL_DEVINL int keep_by_weight(int n, double above, double target, double& all) {
        constexpr int kPer = kListCap / kSelThreads;
        unsigned long long v[kPer], t = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            v[j] = i < n ? s.wt[i] : 0;
            t += v[j];
        }
        unsigned long long p = block_scan(t, s.red);
        unsigned long long keep = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            if (i < n && above + static_cast<double>(p) < target) ++keep;
            p += v[j];
        }
        const unsigned long long k = block_sum(keep, s.red);
        all = above + static_cast<double>(block_sum(t, s.red));
        return static_cast<int>(k);
    }
    // The first `keep` of the sorted list join the kept tokens; the border becomes the base.
    RL_DEVINL void close_list(int n, int keep) {
        for (int i = tid; i < keep; i += kSelThreads) {
            const int ch = static_cast<int>(~static_cast<uint32_t>(s.comp[i])) / kChunk;
            atomicAdd(&cs[ch], s.wt[i]);
            atomicAdd(&cnt[ch], 1);
        }
        if (n > 0) {
            const unsigned long long e = s.comp[keep > 0 ? keep - 1 : 0];
            bkey = static_cast<uint32_t>(e >> 32);
            btie = keep > 0 ? static_cast<int>(~static_cast<uint32_t>(e)) : -1;
        }
        __syncthreads();
    }
    // The first bin at which the cumulative histogram reaches target (else the last filled one).
    template <typename H>
    RL_DEVINL void find_bin(const H* hist, unsigned long long target, int bins, unsigned& bin,
                            unsigned long long& before, unsigned long long& inside) {
        constexpr int kPer = kBins / kSelThreads;
        unsigned long long v[kPer], t = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int i = tid * kPer + j;
            v[j] = i < bins ? hist[i] : 0;
            t += v[j];
        }
        const unsigned long long p0 = block_scan(t, s.red);
        const unsigned long long total = block_sum(t, s.red);
        const unsigned long long want = min(max(target, 1ull), total);
        unsigned long long p = p0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (p < want && p + v[j] >= want) {
                s.bin_lo = tid * kPer + j;
                s.bin_before = p;
                s.bin_inside = v[j];
            }
            p += v[j];
        }
        __syncthreads();
        bin = s.bin_lo;
        before = s.bin_before;
        inside = s.bin_inside;
        __syncthreads();
    }

    // Cuts the base set (of logits >= lo) to its first `k` tokens (by_count) or to the shortest
    // prefix whose weight reaches `target`; cs / cnt then hold the kept ones, bkey / btie the
    // border.  `mass`: the base set's weight (for the histogram by weight).  True: the sorted list
    // begins with the whole kept set.
    RL_DEVINL bool cut(bool by_count, long long k, double target, double mass, float lo, bool few) {
        Bracket b{0, 0.f, 0.f, 0, 0};
        if (few) {                                  // likely few enough to list them all
            collect(b, lo);
            if (s.n_list <= kListCap) {
                finish(by_count, k, target, b);
                return true;
            }
        }
        uint32_t* h32 = reinterpret_cast<uint32_t*>(s.wt);
        unsigned long long* h64 = s.wt;
        unsigned bin = 0;
        unsigned long long before = 0, inside = 0;
        b.mode = 2;
        b.hi = M;
        b.scale = static_cast<float>(kBins) / (M - lo);      // inf - the range is one value - or 0 end in mode 3
        if (b.scale > 0.f && b.scale <= FLT_MAX) {
            for (int i = tid; i < kBins; i += kSelThreads) h32[i] = 0;
            __syncthreads();
            const float q = static_cast<float>(2147483648.0 / (mass / kUnit));
            each(lo, [&](float z, int i) {
                    if (!in_base(key_of(z), i)) return;
                    // a rounded weight: this only says where to look
                    const uint32_t w = by_count ? 1u : __float2uint_rn(exp2_approx((z - M) * c.hi) * q);
                    if (w) atomicAdd(&h32[linear_bin(z, b.hi, b.scale)], w);
                },
                [](int) {});
            __syncthreads();
            find_bin(h32, by_count ? static_cast<unsigned long long>(k)
                                   : static_cast<unsigned long long>(fmin(target / mass, 1.0) * 2147483648.0),
                     kBins, bin, before, inside);
            b.b = bin;
            for (int tries = 0; tries < kBins; ++tries) {
                collect(b, lo);
                if (s.n_list > kListCap) break;
                // the border may lie a bin further, by the rounding of the histogram's weights
                if (by_count) break;
                const double above = sum_weight();
                if (above >= target && b.b > 0) {
                    --b.b;
                    continue;
                }
                unsigned long long t = 0;
                const int n = static_cast<int>(s.n_list);
                for (int i = tid; i < n; i += kSelThreads) t += weight(z_of(static_cast<uint32_t>(s.comp[i] >> 32)));
                const double all = above + static_cast<double>(block_sum(t, s.red));
                if (all < target && b.b < kBins - 1) {
                    ++b.b;
                    continue;
                }
                break;
            }
            if (s.n_list <= kListCap) {
                finish(by_count, k, target, b);
                return false;
            }
        }
        // digits of the key, 11 + 11 + 10 bits, weights in units of 2^-40
        b.mode = 3;
        unsigned long long rest = by_count ? static_cast<unsigned long long>(k)
                                           : static_cast<unsigned long long>(fmax(ceil(target / 1024.0), 1.0));
        uint32_t prefix = 0;
        for (int level = 0; level < 3; ++level) {
            const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kSelThreads) h64[i] = 0;
            __syncthreads();
            each(lo, [&](float z, int i) {
                    const uint32_t key = key_of(z);
                    if (!in_base(key, i)) return;
                    if (level > 0 && (key >> (shift + bits)) != prefix) return;
                    // descending order: bin 0 holds the largest digit
                    const uint32_t d = (1u << bits) - 1u - ((key >> shift) & ((1u << bits) - 1u));
                    atomicAdd(&h64[d], by_count ? 1ull : weight(z) >> 10);
                },
                [](int) {});
            __syncthreads();
            find_bin(h64, rest, 1 << bits, bin, before, inside);
            rest = rest > before ? rest - before : 1;
            prefix = (prefix << bits) | ((1u << bits) - 1u - bin);
            b.shift = shift;
            b.b = prefix;
            __syncthreads();
            collect(b, lo);
            if (s.n_list <= kListCap) break;
        }
        finish(by_count, k, target, b);
        return false;
    }
    // After a collect: how many of the bracket's tokens stay, and the border.
    RL_DEVINL void finish(bool by_count, long long k, double target, const Bracket& b) {
        const long long n_above = sum_int(cnt);
        const double above = sum_weight();
        const long long n = s.n_list;
        __syncthreads();
        if (n <= kListCap) {
            sort_list(static_cast<int>(n));
            double all;
            long long keep = by_count ? min(max(k - n_above, 0ll), n) : keep_by_weight(static_cast<int>(n), above, target, all);
            if (keep == 0 && n_above == 0 && n > 0) keep = 1;
            close_list(static_cast<int>(n), static_cast<int>(keep));
            return;
        }
        // more equal logits than the list holds (the bracket is one key): the lowest indices stay
        const uint32_t key = b.b;
        const unsigned long long w = weight(z_of(key));
        long long keep = by_count ? k - n_above : (w == 0 ? n : static_cast<long long>(ceil(fmax(target - above, 0.0) / static_cast<double>(w))));
        keep = min(max(keep, n_above == 0 ? 1ll : 0ll), n);
        if (tid == 0) {
            s.pick = -1;
            long long left = keep;
            for (int ch = 0; ch < g.nc; ++ch) {
                const int t = static_cast<int>(min(left, static_cast<long long>(in[ch])));
                cs[ch] += w * static_cast<unsigned long long>(t);
                cnt[ch] += t;
                if (t > 0 && left <= in[ch]) {       // the last kept one is the left-th of this chunk
                    s.pick = ch;
                    s.bin_lo = static_cast<unsigned>(left);
                    break;
                }
                left -= t;
            }
        }
        __syncthreads();
        const int ch = s.pick;
        __syncthreads();
        if (ch >= 0 && warp == 0) {
            int want = static_cast<int>(s.bin_lo), at = -1;
            bool bad = false;
            for (int q = 0; q < min(kSubs, g.ns - ch * kSubs) && at < 0; ++q) {
                float z[4];
                const int i0 = ch * kChunk + q * kSub + lane * 4;
                load4<T, kVec>(row, i0, V, z, bad);
                int m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) m += (z[j] > -INFINITY && key_of(z[j]) == key && in_base(key, i0 + j)) ? 1 : 0;
                int incl = m;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                int found = -1, left = want - (incl - m);
                if (left >= 1 && left <= m) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (z[j] > -INFINITY && key_of(z[j]) == key && in_base(key, i0 + j) && --left == 0) found = i0 + j;
                }
                at = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(found + 1))) - 1;
                want -= __shfl_sync(0xffffffffu, incl, 31);
            }
            if (lane == 0) s.pick = at;
        }
        __syncthreads();
        bkey = key;
        btie = s.pick;
        __syncthreads();
    }

    // One draw by one warp; cs holds the inclusive sums of the chunks' weights, as doubles.
    RL_DEVINL void draw(long long r, int d, double total) {
        auto pre = [&](int ch) { return __longlong_as_double(static_cast<long long>(cs[ch])); };
        float u = g.a.u[r * g.a.K + d];
        if (!(u >= 0.f) || !(u < 1.f)) {
            if (lane == 0) set_status(g.status, RL_STATUS_KNOB);
            u = u >= 1.f ? 1.f - 5.9604645e-8f : 0.f;
        }
        const double target = static_cast<double>(u) * total;
        int lo = 0, hi = g.nc - 1;                   // first chunk whose inclusive sum passes the target
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre(mid) > target) hi = mid;
            else lo = mid + 1;
        }
        const double rest = target - (lo > 0 ? pre(lo - 1) : 0.0);
        const unsigned long long want = rest > 0.0 ? static_cast<unsigned long long>(rest) : 0ull;
        unsigned long long run = 0;
        int at = -1, last = -1;
        float zat = 0.f, zlast = 0.f;
        bool bad = false;
        for (int q = 0; q < min(kSubs, g.ns - lo * kSubs) && at < 0; ++q) {
            float z[4];
            const int i0 = lo * kChunk + q * kSub + lane * 4;
            load4<T, kVec>(row, i0, V, z, bad);
            unsigned long long w[4], mine = 0;
            int my_last = -1;
            float my_z = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = z[j] > -INFINITY && in_base(key_of(z[j]), i0 + j) ? weight(z[j]) : 0ull;
                mine += w[j];
                if (z[j] > -INFINITY && in_base(key_of(z[j]), i0 + j)) {
                    my_last = i0 + j;
                    my_z = z[j];
                }
            }
            unsigned long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, run + incl > want);
            if (hit) {
                const int src = __ffs(hit) - 1;
                unsigned long long p = run + incl - mine;
                int f = 0;
                bool got = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p += w[j];
                    if (!got && p > want) {
                        got = true;
                        f = j;
                    }
                }
                const float zf = f == 0 ? z[0] : f == 1 ? z[1] : f == 2 ? z[2] : z[3];
                at = __shfl_sync(0xffffffffu, i0 + f, src);
                zat = __shfl_sync(0xffffffffu, zf, src);
            }
            const unsigned any = __ballot_sync(0xffffffffu, my_last >= 0);
            if (any) {
                const int src = 31 - __clz(any);
                last = __shfl_sync(0xffffffffu, my_last, src);
                zlast = __shfl_sync(0xffffffffu, my_z, src);
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (at < 0) {           // the target met the chunk's sum to the last place
            at = last;
            zat = zlast;
        }
        if (lane == 0) {
            g.a.tokens[r * g.a.K + d] = at;
            if (g.a.logq) g.a.logq[r * g.a.K + d] = log_q(zat, s.rec);
        }
    }
};

// k-th largest of the row's 128-wide maxima (k <= ns): a bound that at least k logits reach.
RL_DEVINL uint32_t kth_submax(SelShared& s, const float* submax, int ns, int k) {
    uint32_t* h = reinterpret_cast<uint32_t*>(s.wt);
    uint32_t prefix = 0;
    unsigned rest = k;
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) h[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < ns; i += kSelThreads) {
            const uint32_t key = key_of(submax[i] + 0.f);
            if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&h[255 - ((key >> shift) & 255)], 1u);
        }
        __syncthreads();
        const unsigned v = threadIdx.x < 256 ? h[threadIdx.x] : 0;
        const unsigned p = static_cast<unsigned>(block_scan(static_cast<unsigned long long>(v), s.red));
        if (p < rest && p + v >= rest) {
            s.pick = 255 - threadIdx.x;
            s.bin_lo = p;
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(s.pick);
        rest -= s.bin_lo;
        __syncthreads();
    }
    return prefix;
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SampleArgs g) {
    extern __shared__ __align__(16) uint8_t raw[];
    SelShared& s = *reinterpret_cast<SelShared*>(raw);
    const rl_sample_args& a = g.a;
    const long long r = blockIdx.x;
    const int tid = threadIdx.x;
    const int V = static_cast<int>(a.V);
    unsigned long long* cs = reinterpret_cast<unsigned long long*>(raw + sizeof(SelShared));
    int* cnt = reinterpret_cast<int*>(cs + g.nc);
    Row<T, kVec> w{g, s, cs, cnt, cnt + g.nc, static_cast<const T*>(a.logits) + r * a.row_stride, g.submax + r * g.ns, V,
                   tid, tid & 31, tid >> 5, 0.f, 0.f, {0.f, 0.f}, 0u, INT_MAX};
    const ChunkStat* stat = g.stat + r * g.nc;
    const Knobs q = load_knobs(a, r);
    fill_table(s.tab, tid, kSelThreads);
    unsigned long long mk = 0;
    for (int ch = tid; ch < g.nc; ch += kSelThreads) mk = max(mk, static_cast<unsigned long long>(key_of(stat[ch].max)));
    const float M = z_of(static_cast<uint32_t>(block_max(mk, s.red)));
    w.M = M;
    int count = 0, mode = kRowEmpty, bits = tid == 0 ? q.bits : 0;
    double total = 0.0;

    if (!(M > -INFINITY)) {
        for (int d = tid; d < a.K; d += kSelThreads) {
            a.tokens[r * a.K + d] = -1;
            if (a.logq) a.logq[r * a.K + d] = -INFINITY;
        }
        for (int ch = tid; ch < g.nc; ch += kSelThreads) cnt[ch] = 0;
        bits |= tid == 0 ? RL_STATUS_EMPTY_ROW : 0;
        if (tid == 0) s.rec = RowRec{M, {1.f, 0.f}, {0.f, 0.f}, 0u, -1, kRowEmpty};
    } else if (q.greedy) {
        // the lowest index of the largest logit
        unsigned long long first = 0;
        for (int i = tid; i < g.ns; i += kSelThreads)
            if (w.submax[i] == M) {
                first = ~static_cast<unsigned long long>(i);
                break;
            }
        const int sub = static_cast<int>(~block_max(first, s.red));
        if (w.warp == 0) {
            float z[4];
            bool bad = false;
            load4<T, kVec>(w.row, sub * kSub + w.lane * 4, V, z, bad);
            int at = INT_MAX;
#pragma unroll
            for (int j = 3; j >= 0; --j)
                if (z[j] == M) at = sub * kSub + w.lane * 4 + j;
            at = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(at)));
            if (w.lane == 0) s.pick = at;
        }
        for (int ch = tid; ch < g.nc; ch += kSelThreads) cnt[ch] = 0;
        __syncthreads();
        const int at = s.pick;
        for (int d = tid; d < a.K; d += kSelThreads) {
            a.tokens[r * a.K + d] = at;
            if (a.logq) a.logq[r * a.K + d] = 0.f;
        }
        if (tid == 0) {
            cnt[at / kChunk] = 1;
            s.rec = RowRec{M, {1.f, 0.f}, {0.f, 0.f}, key_of(M), at, kRowCut};
        }
        count = 1;
        mode = kRowCut;
        __syncthreads();
    } else {
        w.c = scale_of(q.T);
        w.zlow = fmaxf(M - 64.f / w.c.hi, -FLT_MAX);
        // the least logit whose weight is at least min_p and 2^-100
        if (tid == 0) {
            const double lim = static_cast<double>(M) + static_cast<double>(q.T) * log(fmax(static_cast<double>(q.mp), 0x1p-100));
            float f = __double2float_ru(lim);
            s.fpick = fminf(fmaxf(f, -FLT_MAX), M) + 0.f;
        }
        __syncthreads();
        const float zmin = s.fpick;
        w.bkey = key_of(zmin);
        w.btie = INT_MAX;
        bool fixed = true;                              // cs in units of 2^-50, else (whole rows) weights
        if (q.total) {
            // the chunks' sums relative to M's weight
            const double cd = 1.4426950408889634 / static_cast<double>(q.T);
            const double pm = static_cast<double>(M) * cd;
            const bool plain = fabsf(M * w.c.hi) < kWholeRef;
            const double ref = ceil(static_cast<double>(M * w.c.hi));
            const double f = plain ? exp2(ref - pm) : 1.0;
            double v = 0.0;
            for (int ch = tid; ch < g.nc; ch += kSelThreads) {
                const ChunkStat st = stat[ch];
                double x = 0.0;
                if (st.sum > 0.0) {
                    if (plain && st.ref != INT_MIN) {
                        const int n = st.ref - static_cast<int>(ref);
                        x = n < -200 ? 0.0 : st.sum * f * __longlong_as_double(static_cast<long long>(1023 + n) << 52);
                    } else {
                        x = st.sum * exp2(st.ref == INT_MIN ? (static_cast<double>(st.max) - M) * cd : st.ref - pm);
                    }
                }
                x = x < 0x1p-52 ? 0.0 : x * kUnit;       // below what a draw can tell from nothing
                cs[ch] = static_cast<unsigned long long>(__double_as_longlong(x));
                v += x;
            }
            total = block_sum(v, s.redd);
            fixed = false;
        }
        if (!q.cut) {
            mode = kRowWhole;
            count = a.K - 1;
        } else {
            mode = kRowCut;
            double mass = total;
            float lo = zmin;
            bool done = false, listed = false;
            if (q.k < V) {
                bool few = false;
                if (q.k <= g.ns) {
                    lo = fmaxf(lo, z_of(kth_submax(s, w.submax, g.ns, q.k)));
                    few = q.k <= kListCap / 2;
                }
                listed = w.cut(true, q.k, 0.0, 0.0, lo, few);
                done = true;
            } else if (!q.total) {                      // min_p alone so far: all of its tokens
                unsigned long long hit = 0;
                for (int i = tid; i < g.ns; i += kSelThreads) hit += w.submax[i] >= lo ? 1 : 0;
                const bool few = block_sum(hit, s.red) * 10 < static_cast<unsigned long long>(g.ns) * 9;
                Bracket b{few ? 0 : 1, 0.f, 0.f, 0, 0};
                w.collect(b, lo);
                if (few && s.n_list > kListCap) {
                    b.mode = 1;
                    __syncthreads();
                    w.collect(b, lo);
                }
                if (b.mode == 0) w.finish(true, V, 0.0, b);
                listed = b.mode == 0;
                done = true;
            }
            if (done) mass = w.sum_weight();
            if (q.p < 1.f) {
                const double target = static_cast<double>(q.p) * mass;
                if (listed) {
                    // the whole set is the sorted list's head
                    const int n = static_cast<int>(w.sum_int(w.cnt));
                    double all;
                    int keep = w.keep_by_weight(n, 0.0, target, all);
                    keep = max(keep, 1);
                    for (int ch = tid; ch < g.nc; ch += kSelThreads) {
                        cs[ch] = 0;
                        cnt[ch] = 0;
                    }
                    __syncthreads();
                    w.close_list(n, keep);
                } else {
                    // a logit whose weight is below (1 - p) mass / V cannot be needed
                    if (tid == 0) {
                        const double rest = (1.0 - fmax(static_cast<double>(q.p), 0.0)) * (mass / kUnit) / static_cast<double>(V) * 0.999;
                        const double lim = static_cast<double>(M) + static_cast<double>(q.T) * log(fmin(fmax(rest, 0x1p-100), 1.0));
                        s.fpick = fminf(fmaxf(__double2float_rd(lim), -FLT_MAX), M) + 0.f;
                    }
                    __syncthreads();
                    lo = fmaxf(lo, s.fpick);
                    unsigned long long hit = 0;
                    for (int i = tid; i < g.ns; i += kSelThreads) hit += w.submax[i] >= lo ? 1 : 0;
                    const bool few = block_sum(hit, s.red) * 10 < static_cast<unsigned long long>(g.ns) * 9;
                    w.cut(false, 0, target, mass, lo, few);
                }
            }
            fixed = true;
            count = static_cast<int>(w.sum_int(w.cnt));
        }
        // inclusive sums over the chunks (in place: a thread's own consecutive chunks, then a scan)
        const int per = (g.nc + kSelThreads - 1) / kSelThreads;
        double t = 0.0;
        for (int j = 0; j < per; ++j) {
            const int ch = tid * per + j;
            if (ch < g.nc) {
                t += fixed ? static_cast<double>(cs[ch]) : __longlong_as_double(static_cast<long long>(cs[ch]));
                cs[ch] = static_cast<unsigned long long>(__double_as_longlong(t));
            }
        }
        const double before = block_scan(t, s.redd);
        for (int j = 0; j < per; ++j) {
            const int ch = tid * per + j;
            if (ch < g.nc)
                cs[ch] = static_cast<unsigned long long>(
                    __double_as_longlong(__longlong_as_double(static_cast<long long>(cs[ch])) + before));
        }
        __syncthreads();
        total = __longlong_as_double(static_cast<long long>(cs[g.nc - 1]));
        if (tid == 0) {
            const double lw = log(total / kUnit);
            const float h = static_cast<float>(lw);
            s.rec = RowRec{M, inv_of(q.T), {h, static_cast<float>(lw - h)}, w.bkey, w.btie, mode};
        }
        __syncthreads();
        for (int d = w.warp; d < a.K; d += kSelWarps) w.draw(r, d, total);
    }
    __syncthreads();
    if (a.replayed && tid == 0) a.replayed[r] = q.cut ? 1 : 0;
    if (a.offsets) {
        if (mode == kRowCut)
            for (int ch = tid; ch < g.nc; ch += kSelThreads) g.ccnt[r * g.nc + ch] = cnt[ch];
        if (tid == 0) {
            g.count[r] = count;
            g.rec[r] = s.rec;
        }
        // the last block to finish turns the counts into offsets
        __threadfence();
        __syncthreads();
        if (tid == 0) s.pick = atomicAdd(g.done, 1u) == gridDim.x - 1 ? 1 : 0;
        __syncthreads();
        if (s.pick) {
            __threadfence();
            long long base = 0;
            for (long long b0 = 0; b0 < a.N; b0 += kSelThreads * 4) {
                unsigned long long v[4], t = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const long long i = b0 + tid * 4 + j;
                    v[j] = i < a.N ? static_cast<unsigned long long>(__ldcg(g.count + i)) : 0;
                    t += v[j];
                }
                unsigned long long p = base + block_scan(t, s.red);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const long long i = b0 + tid * 4 + j;
                    if (i < a.N) a.offsets[i] = static_cast<int64_t>(p);
                    p += v[j];
                }
                base += static_cast<long long>(block_sum(t, s.red));
            }
            if (tid == 0) {
                a.offsets[a.N] = base;
                if (base > a.capacity) bits |= RL_STATUS_CAPACITY;
                *g.done = 0;
            }
        }
    }
    set_status(g.status, bits);
}

// ---- 3. the support rows --------------------------------------------------------------
constexpr int kEmitThreads = 256;

template <typename T, bool kVec>
__global__ void __launch_bounds__(kEmitThreads) emit_kernel(const SampleArgs g) {
    __shared__ int sorted[1024];
    const rl_sample_args& a = g.a;
    const int lane = threadIdx.x & 31;
    const int parts = gridDim.x;
    const int V = static_cast<int>(a.V);
    bool bad = false;
    for (long long r = blockIdx.y; r < a.N; r += gridDim.y) {
        const RowRec rec = g.rec[r];
        const T* row = static_cast<const T*>(a.logits) + r * a.row_stride;
        const long long base = a.offsets[r];
        if (rec.mode == kRowWhole) {
            if (blockIdx.x != 0 || a.K < 2) continue;
            int m = 32;
            while (m < a.K - 1) m <<= 1;
            for (int i = threadIdx.x; i < m; i += kEmitThreads) sorted[i] = i < a.K - 1 ? a.tokens[r * a.K + 1 + i] : INT_MAX;
            __syncthreads();
            for (int size = 2; size <= m; size <<= 1)
                for (int step = size >> 1; step > 0; step >>= 1) {
                    for (int t = threadIdx.x; t < m / 2; t += kEmitThreads) {
                        const int i = 2 * t - (t & (step - 1)), j = i + step;
                        const int x = sorted[i], y = sorted[j];
                        if ((x > y) == ((i & size) == 0)) {
                            sorted[i] = y;
                            sorted[j] = x;
                        }
                    }
                    __syncthreads();
                }
            for (int i = threadIdx.x; i < a.K - 1; i += kEmitThreads)
                if (base + i < a.capacity) {
                    a.ids[base + i] = sorted[i];
                    a.support_logq[base + i] = log_q(to_f(row[sorted[i]]), rec);
                }
            __syncthreads();
        } else if (rec.mode == kRowCut) {
            const int* ccnt = g.ccnt + r * g.nc;
            for (int ch = blockIdx.x * (kEmitThreads / 32) + (threadIdx.x >> 5); ch < g.nc; ch += parts * (kEmitThreads / 32)) {
                const int n = ccnt[ch];
                if (n == 0) continue;
                int before = 0;
                for (int i = lane; i < ch; i += 32) before += ccnt[i];
                long long at = base + __reduce_add_sync(0xffffffffu, before);
                int left = n;
                for (int q = 0; q < min(kSubs, g.ns - ch * kSubs) && left > 0; ++q) {
                    if (key_of(g.submax[r * g.ns + ch * kSubs + q] + 0.f) < rec.key) continue;
                    float z[4];
                    const int i0 = ch * kChunk + q * kSub + lane * 4;
                    load4<T, kVec>(row, i0, V, z, bad);
                    bool keep[4];
                    int m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t k = key_of(z[j]);
                        keep[j] = z[j] > -INFINITY && (k > rec.key || (k == rec.key && i0 + j <= rec.tie));
                        m += keep[j] ? 1 : 0;
                    }
                    int incl = m;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int x = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += x;
                    }
                    long long p = at + incl - m;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (keep[j]) {
                            if (p < a.capacity) {
                                a.ids[p] = i0 + j;
                                a.support_logq[p] = log_q(z[j], rec);
                            }
                            ++p;
                        }
                    const int all = __shfl_sync(0xffffffffu, incl, 31);
                    at += all;
                    left -= all;
                }
            }
        }
    }
}

// ---- host ------------------------------------------------------------------------------
static SampleArgs sample_view(void* ws, const rl_sample_args* a, size_t* bytes) {
    SampleArgs g{};
    g.nc = static_cast<int>((a->V + kChunk - 1) / kChunk);
    g.ns = static_cast<int>((a->V + kSub - 1) / kSub);
    Carve cv(ws);
    g.done = cv.take<unsigned>(64);
    g.stat = cv.take<ChunkStat>(static_cast<size_t>(a->N) * g.nc);
    g.submax = cv.take<float>(static_cast<size_t>(a->N) * g.ns);
    g.ccnt = cv.take<int>(static_cast<size_t>(a->N) * g.nc);
    g.count = cv.take<int>(static_cast<size_t>(a->N));
    g.rec = cv.take<RowRec>(static_cast<size_t>(a->N));
    if (bytes) *bytes = align_up(cv.off, 256);
    return g;
}

size_t sample_ws_bytes(int64_t N, int64_t V) {
    rl_sample_args a{};
    a.N = N;
    a.V = V;
    size_t b = 0;
    sample_view(nullptr, &a, &b);
    return b;
}

template <typename T, bool kVec>
static int sample_run(const SampleArgs& g, cudaStream_t stream) {
    const long long units = g.a.N * g.nc;
    long long blocks = (units + kStatThreads / 32 - 1) / (kStatThreads / 32);
    const long long cap = 4ll * num_sms();
    if (blocks > cap) blocks = cap;
    const size_t smem = sizeof(SelShared) + static_cast<size_t>(g.nc) * (sizeof(unsigned long long) + 2 * sizeof(int));
    if (cudaFuncSetAttribute(select_kernel<T, kVec>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return RL_ERR_CUDA;
    ProfScope prof(RL_PROF_OTHER, stream);
    stats_kernel<T, kVec><<<static_cast<unsigned>(blocks), kStatThreads, 0, stream>>>(g);
    select_kernel<T, kVec><<<static_cast<unsigned>(g.a.N), kSelThreads, smem, stream>>>(g);
    int launches = 2;
    if (g.a.offsets) {
        // a block takes eight chunks a step; rows beyond the grid's share are looped over
        const int parts = static_cast<int>((g.nc + 31) / 32);
        const dim3 grid(static_cast<unsigned>(parts), static_cast<unsigned>(g.a.N < 16384 ? g.a.N : 16384), 1);
        emit_kernel<T, kVec><<<grid, kEmitThreads, 0, stream>>>(g);
        ++launches;
    }
    count_launch(launches);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

template <typename T>
static int sample_typed(const SampleArgs& g, cudaStream_t stream) {
    const uintptr_t mask = 4 * sizeof(T) - 1;
    const bool vec = (reinterpret_cast<uintptr_t>(g.a.logits) & mask) == 0 && (g.a.N == 1 || g.a.row_stride % 4 == 0);
    return vec ? sample_run<T, true>(g, stream) : sample_run<T, false>(g, stream);
}

int sample_impl(const rl_sample_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    SampleArgs g = sample_view(ws, a, nullptr);
    g.a = *a;
    g.status = status;
    if (a->dtype == RL_DTYPE_F32) return sample_typed<float>(g, stream);
    if (a->dtype == RL_DTYPE_BF16) return sample_typed<__nv_bfloat16>(g, stream);
    return sample_typed<__half>(g, stream);
}

}  // namespace rl
