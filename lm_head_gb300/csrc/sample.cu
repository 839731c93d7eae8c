// Sampling with temperature, top-k, top-p and min-p from given random numbers, and the
// sampler support as CSR rows (the head's rl_support).
//
// The token of a draw u is the first whose cumulative weight, in index order, passes u times
// the total: a sum over up to the whole vocabulary decides which of two neighbours it is, so
// fp32 sums would give another token every few thousand draws.  Weights and sums are therefore
// carried to about 2^-36 of their row's total:
//   w = 2^p, p = z log2(e) / T - ref with the factor as two floats;  p = n + j/2048 + r;
//   2^(j/2048) = hi (1 + rho) from a table, 2^r - 1 = r ln2 + (r ln2)^2 / 2 (the next term is
//   below 2^-40), so w = 2^n hi (1 + rho + ...) is the unevaluated pair (2^n hi, v).
// fp64 would do the same at a fiftieth of the rate on this part.
//
//  1. stats_kernel   one warp per 1024 logits: the largest of each 128, and where a row needs
//                    them the sums of weights of each 128, with a reference of the chunk's own so
//                    that no pass for the row's maximum comes first.  The only pass over all logits.
//  2. select_kernel  one block a row: the kept set as a threshold (key, index), by collecting
//                    the candidates into shared memory and sorting them when a bound from the
//                    128-wide maxima shows that few can matter, else after a histogram that
//                    brackets the border; then the weight of each part's kept tokens, and each
//                    draw by a search over the parts and a scan of one.  Whole rows (no cut)
//                    take the sums of 1.  Sums are integers in a unit of the row's, the
//                    finest 2^-p of the largest weight (p from 42 to 54) in which its total is sure
//                    to fit: their order does not matter.
//  3. emit_kernel    the support rows, one warp a part.
//
// Measured (one GB300, rows of 151,936 logits, device time):
//   stats   64 us for 256 fp32 rows (2.4 TB/s): bound by instruction issue, some 40 a logit where
//           sums are taken; the float-pair sum is what equality with exact arithmetic costs.
//   select  17 us for 128 whole rows with 17 draws (latency: barriers and one part a draw);
//           203 us for 256 rows whose nucleus is some 20,000 tokens: two passes over the row by one
//           block, bound by issue and the instruction cache.  Clusters of 2, 4 and 8 blocks that
//           share the passes were slower (the whole call 533 to 1036 us against 356 then): the
//           others wait while the first sorts, scans and draws.  So was a block of 1024 threads
//           alone on its multiprocessor for such rows (451 us against 317).
//   emit    70 us for the 5 million entries of those rows.
#include <cfloat>
#include <climits>
#include <cmath>

#include "common.cuh"
#include "ff.cuh"
#include "internal.h"
#include "weights.cuh"

namespace rl {

constexpr int kChunk = 1024;               // logits of one warp step
constexpr int kSub = 128;                  // ... of one 32-lane load
constexpr int kSubs = kChunk / kSub;
constexpr int kListCap = 4096;             // candidates sorted in shared memory
constexpr int kBins = 2048;
constexpr float kWholeRef = 1900.f;        // |max * log2(e) / T| up to which a chunk needs no reference

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
    int nc, ns;                    // chunks of 1024, parts of 128 of a row
    float* submax;                 // [N, ns] largest logit of a part
    unsigned long long* subsum;    // [N, ns] sum of its weights in units of 2^(ref - 50)
    int* ref;                      // [N, nc] the chunk's ref; INT_MIN: the weight of its largest logit
    int* cpre;                     // [N, ns] kept tokens of the parts before
    int* count;                    // [N] entries of the support row
    RowRec* rec;                   // [N]
    unsigned* done;                // rows finished (the call's first kernel clears it)
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

// Four logits as they lie in memory.
template <typename T>
struct Quad {
    T t[4];
    template <bool kVec>
    RL_DEVINL void load(const T* row, int i, int V) {         // from element i on; past the row's end -inf
        if (kVec && i + 4 <= V) {
            if constexpr (sizeof(T) == 4) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(row + i));
                memcpy(t, &q, 16);
            } else {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(row + i));
                memcpy(t, &q, 8);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = i + j < V ? row[i + j] : static_cast<T>(-INFINITY);
        }
    }
    RL_DEVINL void get(float (&z)[4]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = to_f(t[j]);
    }
};
template <typename T, bool kVec>
RL_DEVINL void load4_raw(const T* row, int i, int V, float (&z)[4]) {
    Quad<T> q;
    q.template load<kVec>(row, i, V);
    q.get(z);
}
// Four logits with NaN and +inf as -inf, and no -0.
template <typename T, bool kVec>
RL_DEVINL void load4(const T* row, int i, int V, float (&z)[4]) {
    load4_raw<T, kVec>(row, i, V, z);
#pragma unroll
    for (int j = 0; j < 4; ++j) z[j] = (z[j] < INFINITY ? z[j] : -INFINITY) + 0.f;
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
__global__ void __launch_bounds__(kStatThreads, 2) stats_kernel(const SampleArgs g) {
    __shared__ float2 tab[2048];
    const rl_sample_args& a = g.a;
    if (blockIdx.x == 0 && threadIdx.x == 0) *g.done = 0;
    fill_table(tab, threadIdx.x, kStatThreads);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int V = static_cast<int>(a.V);
    const long long warps = static_cast<long long>(gridDim.x) * (kStatThreads / 32);
    const long long units = a.N * g.nc;
    bool bad = false;
    // a chunk's logits as they lie in memory, the next chunk's on their way while one is worked on
    Quad<T> raw[kSubs], ahead[kSubs];
    Knobs q, q_ahead;
    auto fetch = [&](long long id) {
        const long long r = id / g.nc;
        const T* row = static_cast<const T*>(a.logits) + r * a.row_stride;
        q_ahead = load_knobs(a, r);
#pragma unroll
        for (int s = 0; s < kSubs; ++s) ahead[s].template load<kVec>(row, static_cast<int>(id - r * g.nc) * kChunk + s * kSub + lane * 4, V);
    };
    long long id = static_cast<long long>(blockIdx.x) * (kStatThreads / 32) + (threadIdx.x >> 5);
    if (id < units) fetch(id);
    for (; id < units; id += warps) {
        const long long r = id / g.nc;
        const int c = static_cast<int>(id - r * g.nc);
#pragma unroll
        for (int s = 0; s < kSubs; ++s) raw[s] = ahead[s];
        q = q_ahead;
        if (id + warps < units) fetch(id + warps);
        float z[kSubs][4];
#pragma unroll
        for (int s = 0; s < kSubs; ++s) raw[s].get(z[s]);
        uint32_t cmax = 0, mine = 0;
#pragma unroll
        for (int s = 0; s < kSubs; ++s) {
            float m = max_nan(max_nan(z[s][0], z[s][1]), max_nan(z[s][2], z[s][3]));
            uint32_t k = __reduce_max_sync(0xffffffffu, key_of(m));
            if (k >= 0xff800000u) {                   // NaN or +inf among them
                bad = true;
#pragma unroll
                for (int j = 0; j < 4; ++j) z[s][j] = z[s][j] < INFINITY ? z[s][j] : -INFINITY;
                m = fmaxf(fmaxf(z[s][0], z[s][1]), fmaxf(z[s][2], z[s][3]));
                k = __reduce_max_sync(0xffffffffu, key_of(m));
            }
            cmax = max(cmax, k);
            if (lane == s) mine = k;
        }
        if (lane < kSubs && c * kSubs + lane < g.ns) g.submax[r * g.ns + c * kSubs + lane] = z_of(mine);
        const float m = z_of(cmax);
        if (!q.total) continue;
        uint32_t part_top = 0;
        int part_low = 0, ref_out = 0;
        if (m > -INFINITY) {
            const FF cs = scale_of(q.T);
            const float pm = m * cs.hi;
            if (fabsf(pm) < kWholeRef) {
                const float ref = ceilf(pm), magic = 6144.f - ref, zlow = fmaxf((ref + kLeastExp) / cs.hi, -FLT_MAX);
                ref_out = static_cast<int>(ref);
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    LaneSum acc;
                    float hi[4], v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        weight_pair(fmaxf(z[s][j], zlow), 0.f, cs, magic, tab, hi[j], v[j]);
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
                        part_top = t;
                        part_low = l;
                    }
                }
            } else {
                const float zlow = fmaxf(m + kLeastExp / cs.hi, -FLT_MAX);
                ref_out = INT_MIN;
#pragma unroll
                for (int s = 0; s < kSubs; ++s) {
                    LaneSum acc;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = z[s][j] >= zlow;
                        float hi, v;
                        const FF d = two_sum(in ? z[s][j] : m, -m);
                        weight_pair(d.hi, d.lo, cs, 6144.f, tab, hi, v);
                        acc.add(in ? hi : 0.f, in ? v : 0.f);
                    }
                    const uint32_t t = acc.warp_top();
                    const int l = acc.warp_low();
                    if (lane == s) {
                        part_top = t;
                        part_low = l;
                    }
                }
            }
        }
        if (lane < kSubs && c * kSubs + lane < g.ns) g.subsum[r * g.ns + c * kSubs + lane] = LaneSum::total(part_top, part_low);
        if (lane == 0) g.ref[r * g.nc + c] = ref_out;
    }
    if (bad) set_status(g.status, RL_STATUS_NONFINITE);
    let_next_start();
}

// ---- 2. selection and draws ------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// How a logit lies to the bracket: above it, in it, or below.
struct Bracket {
    int mode;               // 0: everything in; 1: everything above; 2: bin b of (hi - z) scale; 3: key >> shift == b
    float hi, scale;
    int shift;
    uint32_t b;
};
RL_DEVINL int place(const Bracket& k, uint32_t key) {            // modes 0, 1, 3: > 0 above, 0 in, < 0 below
    if (k.mode == 0) return 0;
    if (k.mode == 1) return 1;
    const uint32_t x = k.shift < 32 ? key >> k.shift : 0;
    return x > k.b ? 1 : x == k.b ? 0 : -1;
}

struct SelShared {
    unsigned long long red[kSelWarps];
    float2 tab[2048];
    unsigned long long comp[kListCap];     // candidates: key << 32 | ~index
    unsigned long long wt[kListCap];       // their weights; the histogram before that
    unsigned long long bin_before, bin_inside;
    unsigned long long unit;               // 2^62 over the weight of M in its chunk's units
    unsigned n_list, n_sub, bin_lo;
    int pick;
    float fpick;
    RowRec rec;
    // then: unsigned long long cs[ns]; int cnt[ns], in[ns]; uint16_t subs[ns]
};
constexpr size_t kMaxParts = (1 << 20) / kSub;      // V <= 2^20
constexpr size_t kSelPart = sizeof(unsigned long long) + 2 * sizeof(int) + sizeof(uint16_t);

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
    unsigned long long* cs;      // [ns] kept weight of each part (units of 2^-prec)
    int* cnt;                    // [ns] kept tokens
    int* in;                     // [ns] tokens in the bracket
    uint16_t* subs;              // the parts that a pass reads
    const T* row;
    const float* submax;
    int V, tid, lane, warp;
    float M, zlow;               // zlow: weights are 0 below
    FF c;
    int prec;                    // sums are in units of 2^-prec of M's weight
    uint32_t bkey;               // the set that selection starts from: key > bkey, or equal and
    int btie;                    // index <= btie

    RL_DEVINL unsigned long long weight(float z) const { return weight_fixed(z, M, c, zlow, prec, s.tab); }
    // What LaneSum gives for weights relative to 2^ref of M's, in the row's unit.
    RL_DEVINL unsigned long long in_unit(unsigned long long w50, int ref) const {
        const int sh = prec - 50 + ref;
        return sh >= 0 ? w50 << sh : sh > -64 ? (w50 + (1ull << (-sh - 1))) >> -sh : 0ull;
    }
    RL_DEVINL bool in_base(uint32_t key, int i) const { return key > bkey || (key == bkey && i <= btie); }

    // Lists the parts with a logit >= lo, and clears the sums; returns how many there are.
    RL_DEVINL int list_parts(float lo) {
        __syncthreads();
        if (tid == 0) s.n_sub = 0;
        __syncthreads();
        for (int i0 = 0; i0 < g.ns; i0 += kSelThreads) {
            const int i = i0 + tid;
            const bool hit = i < g.ns && submax[i] >= lo;
            const unsigned m = __ballot_sync(0xffffffffu, hit);
            unsigned at = 0;
            if (lane == 0 && m) at = atomicAdd(&s.n_sub, __popc(m));
            at = __shfl_sync(0xffffffffu, at, 0);
            if (hit) subs[at + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(i);
            if (i < g.ns) {
                cs[i] = 0;
                cnt[i] = 0;
                in[i] = 0;
            }
        }
        __syncthreads();
        return static_cast<int>(s.n_sub);
    }
    // f(z[4], first index, part) for the logits of the listed parts, by all lanes together, a warp a
    // part, the next two parts' logits on their way.  (Four parts at a time, unrolled, ran out of
    // the instruction cache.)
    template <typename F>
    RL_DEVINL void each(F f) {
        const int n = static_cast<int>(s.n_sub);
        Quad<T> ahead[2];
        int part[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int i = warp + q * kSelWarps;
            part[q] = i < n ? subs[i] : -1;
            if (part[q] >= 0) ahead[q].template load<kVec>(row, part[q] * kSub + lane * 4, V);
        }
#pragma unroll 1
        for (int i = warp; i < n; i += kSelWarps) {
            float z[4];
            ahead[0].get(z);
            const int now = part[0];
            ahead[0] = ahead[1];
            part[0] = part[1];
            const int next = i + 2 * kSelWarps;
            part[1] = next < n ? subs[next] : -1;
            if (part[1] >= 0) ahead[1].template load<kVec>(row, part[1] * kSub + lane * 4, V);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = (z[j] < INFINITY ? z[j] : -INFINITY) + 0.f;
            f(z, now * kSub + lane * 4, now);
        }
    }

    // One pass: weight and number of the logits above the bracket by part, those in it listed.
    RL_DEVINL void collect(const Bracket& k, float lo) {
        list_parts(lo);
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        const float fb = static_cast<float>(k.b);
        const bool all_base = btie == INT_MAX && key_of(lo) >= bkey;
        each([&](const float(&z)[4], int i0, int part) {
            const float ref = ceilf((submax[part] - M) * c.hi);
            bool up[4], mid[4], any_up = false, any_mid = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (k.mode == 2) {
                    const float x = fminf((k.hi - z[j]) * k.scale, static_cast<float>(kBins - 1));
                    up[j] = x < fb;
                    mid[j] = !up[j] && x < fb + 1.f;
                } else {
                    const int pl = place(k, key_of(z[j]));
                    up[j] = pl > 0;
                    mid[j] = pl == 0;
                }
                const bool in_set = z[j] >= lo && z[j] > -INFINITY && (all_base || in_base(key_of(z[j]), i0 + j));
                up[j] = up[j] && in_set;
                mid[j] = mid[j] && in_set;
                any_up |= up[j];
                any_mid |= mid[j];
            }
            if (__any_sync(0xffffffffu, any_up)) {
                // those above one after another in shared memory, so that few of them cost few weights
                float* dense = reinterpret_cast<float*>(s.wt) + warp * kSub;      // the list has no weights yet
                int n = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned m = __ballot_sync(0xffffffffu, up[j]);
                    if (up[j]) dense[n + __popc(m & ((1u << lane) - 1u))] = z[j];
                    n += __popc(m);
                }
                __syncwarp();
                LaneSum acc;
                for (int i = lane; i < n; i += 32) {
                    const float x = dense[i];
                    const FF d = two_sum(fmaxf(x, zlow), -M);
                    float hi, v;
                    weight_pair(d.hi, d.lo, c, 6144.f - ref, s.tab, hi, v);
                    if (x >= zlow) acc.add(hi, v);
                }
                __syncwarp();
                const uint32_t wt = acc.warp_top();
                const int wl = acc.warp_low();
                if (lane == 0) {
                    cs[part] = LaneSum::total(wt, wl);
                    cnt[part] = n;
                }
            }
            if (__any_sync(0xffffffffu, any_mid)) {
                int inside = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (mid[j]) {
                        ++inside;
                        const unsigned at = atomicAdd(&s.n_list, 1u);
                        if (at < kListCap)
                            s.comp[at] = (static_cast<unsigned long long>(key_of(z[j])) << 32) | static_cast<uint32_t>(~(i0 + j));
                    }
                inside = __reduce_add_sync(0xffffffffu, inside);
                if (lane == 0) in[part] = inside;
            }
        });
        __syncthreads();
        // the sums into the row's unit (a part a thread: 330 us for 256 flat nuclei, and 336 within the pass)
        for (int i = tid; i < g.ns; i += kSelThreads)
            if (cs[i]) cs[i] = in_unit(cs[i], static_cast<int>(ceilf((submax[i] - M) * c.hi)));
        __syncthreads();
    }
    // Totals over the parts: weight, numbers.
    RL_DEVINL unsigned long long sum_weight() {
        unsigned long long v = 0;
        for (int i = tid; i < g.ns; i += kSelThreads) v += cs[i];
        return block_sum(v, s.red);
    }
    RL_DEVINL long long sum_int(const int* x) {
        unsigned long long v = 0;
        for (int i = tid; i < g.ns; i += kSelThreads) v += static_cast<unsigned>(x[i]);
        return static_cast<long long>(block_sum(v, s.red));
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
                // with one pair a thread, pairs up to 32 apart stay within a warp's 64 entries
                const int next = step > 1 ? step >> 1 : size;
                if (step > 32 || next > 32 || m > kSelThreads * 2) __syncthreads();
                else __syncwarp();
            }
        __syncthreads();
        for (int i = tid; i < n; i += kSelThreads) s.wt[i] = weight(z_of(static_cast<uint32_t>(s.comp[i] >> 32)));
        __syncthreads();
    }
    // How many of the sorted list come before the sum (above + those before) reaches target.
    RL_DEVINL int keep_by_weight(int n, unsigned long long above, unsigned long long target) {
        const unsigned long long lim = target > above ? target - above : 0ull;
        constexpr int kPer = kListCap / kSelThreads;
        const int per = (n + kSelThreads - 1) / kSelThreads;
        unsigned long long t = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per && tid * per + j < n) t += s.wt[tid * per + j];
        unsigned long long p = block_scan(t, s.red);
        unsigned long long keep = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j < per && tid * per + j < n) {
                if (p < lim) ++keep;
                p += s.wt[tid * per + j];
            }
        return static_cast<int>(block_sum(keep, s.red));
    }
    // The first `keep` of the sorted list join the kept tokens; the border becomes the base.
    RL_DEVINL void close_list(int n, int keep) {
        for (int i = tid; i < keep; i += kSelThreads) {
            const int part = static_cast<int>(~static_cast<uint32_t>(s.comp[i])) / kSub;
            atomicAdd(&cs[part], s.wt[i]);
            atomicAdd(&cnt[part], 1);
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

    // Cuts the base set (of logits >= lo) to its first `k` tokens (k > 0) or to the shortest prefix
    // whose weight reaches `top_p` of `mass` (the base set's weight); cs / cnt then
    // hold the kept ones, bkey / btie the border.  True: the sorted list begins with the whole
    // kept set.
    RL_DEVINL bool cut(long long k, float top_p, unsigned long long mass, float lo, bool few) {
        const bool by_count = k > 0;
        const unsigned long long target = by_count ? 0ull : fraction_of(fmaxf(top_p, 0.f), mass);
        Bracket b{0, 0.f, 0.f, 0, 0};
        if (few) {                                  // likely few enough to list them all
            collect(b, lo);
            if (s.n_list <= kListCap) {
                finish(k, target, b);
                return true;
            }
        }
        uint32_t* h32 = reinterpret_cast<uint32_t*>(s.wt);
        unsigned long long* h64 = s.wt;
        unsigned bin = 0;
        unsigned long long before = 0, inside = 0;
        b.mode = 2;
        b.hi = M;
        b.scale = static_cast<float>(kBins) / (M - lo);      // inf (one value) and 0 (too wide) end in mode 3
        if (b.scale > 0.f && b.scale <= FLT_MAX) {
            list_parts(lo);
            for (int i = tid; i < kBins; i += kSelThreads) h32[i] = 0;
            __syncthreads();
            const float q = 2147483648.f / (static_cast<float>(mass) * power_of_2(-prec));
            const bool all_base = btie == INT_MAX && key_of(lo) >= bkey;
            each([&](const float(&z)[4], int i0, int) {
                // a rounded weight: this only says where to look
                uint32_t w[4];
                int bin_of[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = by_count ? 1u : __float2uint_rn(exp2_approx((z[j] - M) * c.hi) * q);
                    bin_of[j] = static_cast<int>(fminf((b.hi - z[j]) * b.scale, static_cast<float>(kBins - 1)));
                    if (!(z[j] >= lo && z[j] > -INFINITY) || !(all_base || in_base(key_of(z[j]), i0 + j))) w[j] = 0;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (w[j]) atomicAdd(&h32[bin_of[j]], w[j]);
            });
            __syncthreads();
            find_bin(h32, by_count ? static_cast<unsigned long long>(k) : static_cast<unsigned long long>(fmaxf(top_p, 0.f) * 2147483648.f),
                     kBins, bin, before, inside);
            b.b = bin;
            int way = 0;
            for (int tries = 0; tries < kBins; ++tries) {
                collect(b, lo);
                if (s.n_list > kListCap) break;
                // the border may lie a bin further, by the rounding of the histogram's weights; it is passed once (a
                // target within the sums' rounding of a bin's edge is in neither of its bins)
                if (by_count) break;
                const unsigned long long above = sum_weight();
                if (above >= target && b.b > 0) {
                    if (way > 0) break;
                    way = -1;
                    --b.b;
                    continue;
                }
                unsigned long long t = 0;
                const int n = static_cast<int>(s.n_list);
                for (int i = tid; i < n; i += kSelThreads) t += weight(z_of(static_cast<uint32_t>(s.comp[i] >> 32)));
                if (above + block_sum(t, s.red) < target && b.b < kBins - 1 && way >= 0) {
                    way = 1;
                    ++b.b;
                    continue;
                }
                break;
            }
            if (s.n_list <= kListCap) {
                finish(k, target, b);
                return false;
            }
        }
        // digits of the key, 11 + 11 + 10 bits
        b.mode = 3;
        unsigned long long rest = by_count ? static_cast<unsigned long long>(k) : max(target, 1ull);
        uint32_t prefix = 0;
        for (int level = 0; level < 3; ++level) {
            const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
            list_parts(lo);
            for (int i = tid; i < kBins; i += kSelThreads) h64[i] = 0;
            __syncthreads();
            each([&](const float(&z)[4], int i0, int) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t key = key_of(z[j]);
                    if (!(z[j] >= lo && z[j] > -INFINITY) || !in_base(key, i0 + j)) continue;
                    if (level > 0 && (key >> (shift + bits)) != prefix) continue;
                    // descending order: bin 0 holds the largest digit
                    const uint32_t d = (1u << bits) - 1u - ((key >> shift) & ((1u << bits) - 1u));
                    atomicAdd(&h64[d], by_count ? 1ull : weight(z[j]));
                }
            });
            __syncthreads();
            find_bin(h64, rest, 1 << bits, bin, before, inside);
            rest = rest > before ? rest - before : 1;
            prefix = (prefix << bits) | ((1u << bits) - 1u - bin);
            b.shift = shift;
            b.b = prefix;
            collect(b, lo);
            if (s.n_list <= kListCap) break;
        }
        finish(k, target, b);
        return false;
    }
    // After a collect: how many of the bracket's tokens stay, and the border.
    RL_DEVINL void finish(long long k, unsigned long long target, const Bracket& b) {
        const bool by_count = k > 0;
        const bool all_in = b.mode == 0;
        const long long n_above = all_in ? 0 : sum_int(cnt);
        const unsigned long long above = all_in ? 0 : sum_weight();
        const long long n = s.n_list;
        __syncthreads();
        if (n <= kListCap) {
            sort_list(static_cast<int>(n));
            long long keep = by_count ? min(max(k - n_above, 0ll), n) : keep_by_weight(static_cast<int>(n), above, target);
            if (keep == 0 && n_above == 0 && n > 0) keep = 1;
            close_list(static_cast<int>(n), static_cast<int>(keep));
            return;
        }
        // more equal logits than the list holds (the bracket is one key): the lowest indices stay.  Their
        // number by the weight in 64 bits: a rounding of it to the row's unit would count once a token.
        const uint32_t key = b.b;
        const float zk = z_of(key);
        double w = 0.0;
        if (zk >= zlow) {
            float hi, v;
            const FF d = two_sum(zk, -M);
            weight_pair(d.hi, d.lo, c, 6144.f, s.tab, hi, v);
            if (hi < 2.f) w = static_cast<double>(hi) + static_cast<double>(v);      // (differences past the range of floats)
        }
        long long keep = by_count ? k - n_above : n;
        if (!by_count && w > 0.0) {
            const double few = static_cast<double>(target > above ? target - above : 0ull) * static_cast<double>(power_of_2(-prec)) / w;
            if (few < static_cast<double>(n)) keep = static_cast<long long>(ceil(few));
        }
        keep = min(max(keep, n_above == 0 ? 1ll : 0ll), n);
        if (tid == 0) s.pick = -1;
        const int per = (g.ns + kSelThreads - 1) / kSelThreads;
        unsigned long long mine = 0;
        for (int j = 0; j < per; ++j) {
            const int i = tid * per + j;
            if (i < g.ns) mine += static_cast<unsigned>(in[i]);
        }
        long long before = static_cast<long long>(block_scan(mine, s.red));
        for (int j = 0; j < per; ++j) {
            const int i = tid * per + j;
            if (i < g.ns && in[i] > 0 && before < keep) {
                const int t = static_cast<int>(min(keep - before, static_cast<long long>(in[i])));
                cs[i] += __double2ull_rn(w * t * static_cast<double>(power_of_2(prec)));
                cnt[i] += t;
                if (before + in[i] >= keep) {        // the last kept one is the t-th of this part
                    s.pick = i;
                    s.bin_lo = static_cast<unsigned>(t);
                }
                before += in[i];
            }
        }
        __syncthreads();
        const int part = s.pick;
        __syncthreads();
        if (part >= 0 && warp == 0) {
            float z[4];
            const int i0 = part * kSub + lane * 4;
            load4<T, kVec>(row, i0, V, z);
            bool is[4];
            int m = 0, left = static_cast<int>(s.bin_lo), at = -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                is[j] = z[j] > -INFINITY && key_of(z[j]) == key && in_base(key, i0 + j);
                const unsigned bal = __ballot_sync(0xffffffffu, is[j]);
                left -= __popc(bal & ((1u << lane) - 1u));
                m += is[j] ? 1 : 0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (is[j] && --left == 0) at = i0 + j;
            at = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(at + 1))) - 1;
            if (lane == 0) s.pick = at;
        }
        __syncthreads();
        bkey = key;
        btie = s.pick;
        __syncthreads();
    }

    // One draw by one warp; cs holds the inclusive sums of the parts' weights.
    RL_DEVINL void draw(long long r, int d, unsigned long long total) {
        float u = g.a.u[r * g.a.K + d];
        if (!(u >= 0.f) || !(u < 1.f)) {
            if (lane == 0) set_status(g.status, RL_STATUS_KNOB);
            u = u >= 1.f ? 1.f - 5.9604645e-8f : 0.f;
        }
        const unsigned long long target = fraction_of(u, total);
        int lo = 0, hi = g.ns - 1;                   // first part whose inclusive sum passes the target
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cs[mid] > target) hi = mid;
            else lo = mid + 1;
        }
        const unsigned long long before = lo > 0 ? cs[lo - 1] : 0ull;
        const unsigned long long want = target > before ? target - before : 0ull;
        float z[4];
        const int i0 = lo * kSub + lane * 4;
        load4<T, kVec>(row, i0, V, z);
        unsigned long long w[4], mine = 0;
        int my_last = -1;
        float my_z = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in_set = z[j] > -INFINITY && in_base(key_of(z[j]), i0 + j);
            w[j] = in_set ? weight(z[j]) : 0ull;
            mine += w[j];
            if (in_set) {
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
        const unsigned hit = __ballot_sync(0xffffffffu, incl > want);
        int at = my_last;
        float zat = my_z;
        int src;
        if (hit) {
            src = __ffs(hit) - 1;
            unsigned long long p = incl - mine;
            bool got = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p += w[j];
                if (!got && p > want) {
                    got = true;
                    at = i0 + j;
                    zat = z[j];
                }
            }
        } else {                // the target met the part's sum to the last place
            src = 31 - __clz(__ballot_sync(0xffffffffu, my_last >= 0) | 1u);
        }
        if (lane == src) {
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
__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const SampleArgs g) {
    extern __shared__ __align__(16) uint8_t raw[];
    SelShared& s = *reinterpret_cast<SelShared*>(raw);
    const rl_sample_args& a = g.a;
    const long long r = blockIdx.x;
    const int tid = threadIdx.x;
    const int V = static_cast<int>(a.V);
    unsigned long long* cs = reinterpret_cast<unsigned long long*>(raw + sizeof(SelShared));
    int* cnt = reinterpret_cast<int*>(cs + g.ns);
    Row<T, kVec> w{g, s, cs, cnt, cnt + g.ns, reinterpret_cast<uint16_t*>(cnt + 2 * g.ns),
                   static_cast<const T*>(a.logits) + r * a.row_stride, g.submax + r * g.ns, V,
                   tid, tid & 31, tid >> 5, 0.f, 0.f, {0.f, 0.f}, 0, 0u, INT_MAX};
    const Knobs q = load_knobs(a, r);
    fill_table(s.tab, tid, kSelThreads);
    wait_for_previous();
    unsigned long long mk = 0;
    for (int i = tid; i < g.ns; i += kSelThreads) mk = max(mk, static_cast<unsigned long long>(key_of(w.submax[i] + 0.f)));
    const float M = z_of(static_cast<uint32_t>(block_max(mk, s.red)));
    w.M = M;
    int count = 0, mode = kRowEmpty, bits = tid == 0 ? q.bits : 0;

    if (!(M > -INFINITY)) {
        for (int d = tid; d < a.K; d += kSelThreads) {
            a.tokens[r * a.K + d] = -1;
            if (a.logq) a.logq[r * a.K + d] = -INFINITY;
        }
        for (int i = tid; i < g.ns; i += kSelThreads) cnt[i] = 0;
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
            load4<T, kVec>(w.row, sub * kSub + w.lane * 4, V, z);
            int at = INT_MAX;
#pragma unroll
            for (int j = 3; j >= 0; --j)
                if (z[j] == M) at = sub * kSub + w.lane * 4 + j;
            at = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(at)));
            if (w.lane == 0) s.pick = at;
        }
        for (int i = tid; i < g.ns; i += kSelThreads) cnt[i] = 0;
        __syncthreads();
        const int at = s.pick;
        for (int d = tid; d < a.K; d += kSelThreads) {
            a.tokens[r * a.K + d] = at;
            if (a.logq) a.logq[r * a.K + d] = 0.f;
        }
        if (tid == 0) {
            cnt[at / kSub] = 1;
            s.rec = RowRec{M, {1.f, 0.f}, {0.f, 0.f}, key_of(M), at, kRowCut};
        }
        count = 1;
        mode = kRowCut;
        __syncthreads();
        if (a.offsets)
            for (int i = tid; i < g.ns; i += kSelThreads) g.cpre[r * g.ns + i] = i > at / kSub ? 1 : 0;
    } else {
        w.c = scale_of(q.T);
        w.zlow = fmaxf(M + kLeastExp / w.c.hi, -FLT_MAX);
        // the least logit whose weight is at least min_p and 2^-100: M + T ln(...), rounded up
        if (tid == 0) {
            FF lim = q.mp > 0.f ? ln_pair({fmaxf(q.mp, 7.888609e-31f), 0.f}) : FF{-69.31472016f, 1.5413417e-06f};
            lim = ff_add(ff_mul(lim, {q.T, 0.f}), {M, 0.f});
            const float f = lim.lo > 0.f ? nextafterf(lim.hi, INFINITY) : lim.hi;
            s.fpick = fminf(fmaxf(f, -FLT_MAX), M) + 0.f;
            // 2^(ref - p) for M's phase p: what turns its chunk's units into M's weight
            const float pm = __fmul_rn(M, w.c.hi);
            if (fabsf(pm) < kWholeRef) {
                float hi, v;
                weight_pair(-M, 0.f, w.c, 6144.f + ceilf(pm), s.tab, hi, v);
                s.unit = (static_cast<unsigned long long>(hi * 8388608.f) << 39) + static_cast<long long>(v * 0x1p62f);
            }
        }
        // the unit of the row's sums: with S the sum of the parts' largest weights, from 1 to 8192, the
        // total is at most 128 S, below 2^62 units of 2^-(54 - floor(log2 S))
        float likely = 0.f;
        for (int i = tid; i < g.ns; i += kSelThreads) likely += exp2_approx(fmaxf(w.submax[i] - M, -FLT_MAX) * w.c.hi);
        likely = block_sum(likely, reinterpret_cast<float*>(s.red));
        w.prec = 54 - min(max(static_cast<int>(__float_as_uint(likely) >> 23) - 127, 0), 13);
        const float zmin = s.fpick;
        w.bkey = key_of(zmin);
        w.btie = INT_MAX;
        unsigned long long mass = 0;
        if (q.total) {
            // the parts' sums relative to M's weight
            const float pm = __fmul_rn(M, w.c.hi);
            const bool plain = fabsf(pm) < kWholeRef;
            const int ref = plain ? static_cast<int>(ceilf(pm)) : 0;
            const unsigned long long unit = s.unit;
            unsigned long long v = 0;
            for (int i = tid; i < g.ns; i += kSelThreads) {
                unsigned long long x = g.subsum[r * g.ns + i];
                const int rc = g.ref[r * g.nc + i / kSubs];
                if (x) {
                    if (plain && rc != INT_MIN) {
                        const int n = ref - rc + 54 - w.prec;          // at most 2^57 in, times 2^4 units of 2^-54
                        x = n < 64 ? __umul64hi(x << 6, unit) >> n : 0ull;
                    } else {                            // very large logits: the slow way
                        const double cd = 1.4426950408889634 / static_cast<double>(q.T);
                        float cm = -INFINITY;
                        for (int j = i / kSubs * kSubs; j < min(i / kSubs * kSubs + kSubs, g.ns); ++j) cm = fmaxf(cm, w.submax[j]);
                        const double d = rc == INT_MIN ? (static_cast<double>(cm) - M) * cd : rc - M * cd;
                        x = static_cast<unsigned long long>(static_cast<double>(x) * exp2(d + (w.prec - 50)));
                    }
                }
                cs[i] = x;
                v += x;
            }
            if (q.cut) mass = block_sum(v, s.red);
            else __syncthreads();
        }
        if (!q.cut) {
            mode = kRowWhole;
            count = a.K - 1;
        } else {
            mode = kRowCut;
            float lo = zmin;
            bool listed = false;
            if (q.k < V) {
                bool few = false;
                if (q.k <= g.ns) {
                    lo = fmaxf(lo, z_of(kth_submax(s, w.submax, g.ns, q.k)));
                    few = q.k <= kListCap / 2;
                }
                listed = w.cut(q.k, 0.f, 0ull, lo, few);
            } else if (!q.total) {                      // min_p alone so far: all of its tokens
                const bool few = w.list_parts(lo) * 10 < g.ns * 9;
                Bracket b{few ? 0 : 1, 0.f, 0.f, 0, 0};
                w.collect(b, lo);
                if (few && s.n_list > kListCap) {
                    b.mode = 1;
                    w.collect(b, lo);
                }
                if (b.mode == 0) w.finish(V, 0ull, b);
                listed = b.mode == 0;
            }
            if (!q.total && q.p < 1.f) mass = w.sum_weight();
            if (q.p < 1.f) {
                if (listed) {
                    // the whole set is the sorted list's head
                    const int n = static_cast<int>(w.sum_int(w.cnt));
                    const int keep = max(w.keep_by_weight(n, 0ull, fraction_of(fmaxf(q.p, 0.f), mass)), 1);
                    for (int i = tid; i < g.ns; i += kSelThreads) {
                        cs[i] = 0;
                        cnt[i] = 0;
                    }
                    __syncthreads();
                    w.close_list(n, keep);
                } else {
                    // a logit whose weight is below (1 - p) mass / V cannot be needed
                    const float rest = (1.f - fmaxf(q.p, 0.f)) * (static_cast<float>(mass) * power_of_2(-w.prec)) / static_cast<float>(V) * 0.999f;
                    const float need = M + q.T * fminf(logf(fmaxf(rest, 7.9e-31f)), 0.f);
                    lo = fmaxf(lo, fminf(need - 0x1p-18f * (q.T + fabsf(M)), M));
                    w.cut(0, q.p, mass, lo, w.list_parts(lo) * 10 < g.ns * 9);
                }
            }
        }
        // inclusive sums over the parts, of weights (in place) and of the kept tokens
        const int per = (g.ns + kSelThreads - 1) / kSelThreads;
        unsigned long long t = 0, tn = 0;
        for (int j = 0; j < per; ++j) {
            const int i = tid * per + j;
            if (i < g.ns) {
                t += cs[i];
                cs[i] = t;
                if (mode == kRowCut) tn += static_cast<unsigned>(cnt[i]);
            }
        }
        const unsigned long long before = block_scan(t, s.red);
        for (int j = 0; j < per; ++j) {
            const int i = tid * per + j;
            if (i < g.ns) cs[i] += before;
        }
        if (mode == kRowCut) {
            unsigned long long p = block_scan(tn, s.red);
            if (a.offsets)
                for (int j = 0; j < per; ++j) {
                    const int i = tid * per + j;
                    if (i < g.ns) {
                        g.cpre[r * g.ns + i] = static_cast<int>(p);
                        p += static_cast<unsigned>(cnt[i]);
                    }
                }
            count = static_cast<int>(block_sum(tn, s.red));
        }
        __syncthreads();
        const unsigned long long total = cs[g.ns - 1];
        if (tid == 0) {
            // the total as a float pair
            const float th = __ull2float_rz(total);
            const float tl = static_cast<float>(static_cast<long long>(total - static_cast<unsigned long long>(th)));
            s.rec = RowRec{M, inv_of(q.T), ln_pair(fast_two_sum(th * power_of_2(-w.prec), tl * power_of_2(-w.prec))), w.bkey, w.btie, mode};
        }
        __syncthreads();
        for (int d = w.warp; d < a.K; d += kSelWarps) w.draw(r, d, total);
    }
    __syncthreads();
    let_next_start();
    if (a.replayed && tid == 0) a.replayed[r] = q.cut ? 1 : 0;
    if (a.offsets) {
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
    __shared__ float kept_z[kEmitThreads / 32][kSub];
    __shared__ uint8_t kept_i[kEmitThreads / 32][kSub];
    const rl_sample_args& a = g.a;
    const int lane = threadIdx.x & 31;
    const int parts = gridDim.x;
    const int V = static_cast<int>(a.V);
    wait_for_previous();
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
                    a.support_logq[base + i] = log_q(to_f(row[max(sorted[i], 0)]) + 0.f, rec);
                }
            __syncthreads();
        } else if (rec.mode == kRowCut) {
            const int* cpre = g.cpre + r * g.ns;
            float* kz = kept_z[threadIdx.x >> 5];
            uint8_t* ki = kept_i[threadIdx.x >> 5];
            const float zk = z_of(rec.key);
            const int total = static_cast<int>(min(static_cast<long long>(a.offsets[r + 1]) - base, static_cast<long long>(INT_MAX)));
            // 32 parts a warp and step
            for (int p0 = (blockIdx.x * (kEmitThreads / 32) + (threadIdx.x >> 5)) * 32; p0 < g.ns; p0 += parts * kEmitThreads) {
                const int mine = p0 + lane;
                const int from = mine < g.ns ? cpre[mine] : 0;
                const int to = mine < g.ns ? (mine + 1 < g.ns ? cpre[mine + 1] : total) : 0;
                unsigned todo = __ballot_sync(0xffffffffu, to > from);
                // one part after another, the next two parts' logits on their way
                Quad<T> ahead[2];
                int part[2];
                auto fetch = [&](int q) {
                    part[q] = todo ? __ffs(todo) - 1 : -1;
                    todo &= todo - 1u;
                    if (part[q] >= 0) ahead[q].template load<kVec>(row, (p0 + part[q]) * kSub + lane * 4, V);
                };
                fetch(0);
                fetch(1);
#pragma unroll 1
                while (part[0] >= 0) {
                    float z[4];
                    ahead[0].get(z);
                    const int now = part[0];
                    ahead[0] = ahead[1];
                    part[0] = part[1];
                    fetch(1);
                    // the part's kept logits one after another in shared memory, then dense arithmetic
                    const int i0 = (p0 + now) * kSub + lane * 4;
                    int have = 0, at = 0;              // index order: a lane's four logits are neighbours
                    unsigned keeps = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool keep = (z[j] > zk && z[j] < INFINITY) || (z[j] == zk && i0 + j <= rec.tie);
                        const unsigned m = __ballot_sync(0xffffffffu, keep);
                        at += __popc(m & ((1u << lane) - 1u));
                        have += __popc(m);
                        keeps |= (keep ? 1u : 0u) << j;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if ((keeps >> j) & 1u) {
                            kz[at] = z[j] + 0.f;
                            ki[at] = static_cast<uint8_t>(lane * 4 + j);
                            ++at;
                        }
                    __syncwarp();
                    const long long to_at = base + __shfl_sync(0xffffffffu, from, now);
                    for (int i = lane; i < have; i += 32) {
                        if (to_at + i >= a.capacity) break;
                        a.ids[to_at + i] = (p0 + now) * kSub + ki[i];
                        a.support_logq[to_at + i] = log_q(kz[i], rec);
                    }
                    __syncwarp();
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
    g.submax = cv.take<float>(static_cast<size_t>(a->N) * g.ns);
    g.subsum = cv.take<unsigned long long>(static_cast<size_t>(a->N) * g.ns);
    g.ref = cv.take<int>(static_cast<size_t>(a->N) * g.nc);
    g.cpre = cv.take<int>(static_cast<size_t>(a->N) * g.ns);
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
    const long long cap = 2ll * num_sms();
    if (blocks > cap) blocks = cap;
    const size_t smem = sizeof(SelShared) + static_cast<size_t>(g.ns) * kSelPart;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(select_kernel<T, kVec>, static_cast<int>(sizeof(SelShared) + kMaxParts * kSelPart), done)) return RL_ERR_CUDA;
    ProfScope prof(RL_PROF_OTHER, stream);
    stats_kernel<T, kVec><<<static_cast<unsigned>(blocks), kStatThreads, 0, stream>>>(g);
    int launches = 2;
    int rc = launch_after(select_kernel<T, kVec>, dim3(static_cast<unsigned>(g.a.N)), kSelThreads, smem, true, stream, g);
    if (rc != RL_OK) return rc;
    if (g.a.offsets) {
        // a block takes 256 parts a step; rows beyond the grid's share are looped over
        const int parts = static_cast<int>((g.ns + kEmitThreads - 1) / kEmitThreads);
        const dim3 grid(static_cast<unsigned>(parts), static_cast<unsigned>(g.a.N < 16384 ? g.a.N : 16384), 1);
        rc = launch_after(emit_kernel<T, kVec>, grid, kEmitThreads, 0, true, stream, g);
        if (rc != RL_OK) return rc;
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
