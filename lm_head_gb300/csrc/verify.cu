// Verification of drafted tokens against the target's probabilities.
//
//  rows_kernel     one block a row of logits: its largest logit and the sum of its weights
//  request_kernel  one block a request: the accepted drafts, then the token drawn from what is left of the
//                  target at the first that is not, or from its last row
#include <cfloat>
#include <climits>
#include <cmath>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace rl {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;

struct VerRow {
    float M;            // the row's largest logit (-inf: none)
    int at;             // its first index
    double S;           // sum of e^((z - M) / T)
};
struct VerSide {
    rl_dist d;
    int dtype;
    VerRow* rec;        // [T] of the step's rows
};
struct VerArgs {
    rl_verify_args a;
    VerSide side[2];    // target, draft
    int32_t* status;
    bool sure;          // no draft distribution
};

RL_DEVINL float logit_at(const rl_dist& d, int dtype, long long row, long long j) {
    const long long i = row * d.row_stride + j;
    float z;
    if (dtype == RL_DTYPE_F32) z = static_cast<const float*>(d.logits)[i];
    else if (dtype == RL_DTYPE_BF16) z = __bfloat162float(static_cast<const __nv_bfloat16*>(d.logits)[i]);
    else z = __half2float(static_cast<const __half*>(d.logits)[i]);
    return z;
}
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

template <typename T>
RL_DEVINL T vblock_sum(T v, T* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    T s = red[0];
    for (int w = 1; w < kVerWarps; ++w) s += red[w];
    return s;
}

__global__ void __launch_bounds__(kVerThreads) rows_kernel(const VerArgs g) {
    __shared__ double red[kVerWarps];
    __shared__ unsigned long long redk[kVerWarps];
    const long long t = blockIdx.x;
    const VerSide& s = g.side[blockIdx.y];
    const int V = static_cast<int>(g.a.V);
    int bits = 0;
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        g.a.tokens[t] = -1;
        if (g.a.logq) g.a.logq[t] = 0.f;
    }
    if (!s.d.logits) return;
    const long long row = row_of(s.d, t, bits);
    if (row < 0 || is_support(s.d, row)) return;
    const float T = temperature_of(s.d, row, bits);
    unsigned long long best = 0;             // key of the logit, then the lower index
    for (int j = threadIdx.x; j < V; j += kVerThreads) {
        float z = logit_at(s.d, s.dtype, row, j);
        if (!(z < INFINITY)) {
            bits |= RL_STATUS_NONFINITE;
            z = -INFINITY;
        }
        const uint32_t b = __float_as_uint(z + 0.f);
        const uint32_t k = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
        best = max(best, (static_cast<unsigned long long>(k) << 32) | static_cast<uint32_t>(~j));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    if ((threadIdx.x & 31) == 0) redk[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kVerWarps; ++w) best = max(best, redk[w]);
    const uint32_t k = static_cast<uint32_t>(best >> 32);
    const float M = __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
    double S = 0.0;
    if (M > -INFINITY && T > 0.f)
        for (int j = threadIdx.x; j < V; j += kVerThreads) {
            const float z = logit_at(s.d, s.dtype, row, j);
            if (z < INFINITY && z > -INFINITY) S += exp((static_cast<double>(z) - M) / T);
        }
    S = vblock_sum(S, red);
    if (threadIdx.x == 0) s.rec[t] = VerRow{M, static_cast<int>(~static_cast<uint32_t>(best)), S};
    set_status(g.status, bits);
}

// A row's distribution, as a block sees it.
struct VerDist {
    enum { kNone, kDense, kPoint, kSupport };
    int mode, dtype, at;                // kPoint: all of it on `at`
    const rl_dist* d;
    long long row, eb, ee;
    float M, T;
    double S;
};
RL_DEVINL VerDist dist_at(const VerArgs& g, int side, long long t, int& bits) {
    VerDist x{};
    const VerSide& s = g.side[side];
    x.d = &s.d;
    x.dtype = s.dtype;
    if (side == 1 && g.sure) {
        x.mode = VerDist::kPoint;
        x.at = t + 1 < g.a.T ? g.a.step_tokens[t + 1] : -1;
        return x;
    }
    x.row = row_of(s.d, t, bits);
    if (x.row < 0) return x;
    if (is_support(s.d, x.row)) {
        x.eb = s.d.offsets[x.row];
        x.ee = s.d.offsets[x.row + 1];
        if (x.eb < 0 || x.ee < x.eb || x.ee > s.d.nnz) {
            bits |= RL_STATUS_OFFSETS;
            return x;
        }
        x.mode = VerDist::kSupport;
        return x;
    }
    const VerRow r = s.rec[t];
    if (!(r.M > -INFINITY)) return x;
    x.T = temperature_of(s.d, x.row, bits);
    x.M = r.M;
    x.S = r.S;
    x.at = r.at;
    x.mode = x.T > 0.f ? VerDist::kDense : VerDist::kPoint;
    return x;
}
// ln of the probability of token j (0 <= j < V); -inf: none
RL_DEVINL double log_prob(const VerDist& x, int j, int& bits) {
    if (x.mode == VerDist::kPoint) return j == x.at ? 0.0 : -INFINITY;
    if (x.mode == VerDist::kDense) {
        const float z = logit_at(*x.d, x.dtype, x.row, j);
        return z < INFINITY && z > -INFINITY ? (static_cast<double>(z) - x.M) / x.T - log(x.S) : -INFINITY;
    }
    if (x.mode == VerDist::kSupport) {
        long long lo = x.eb, hi = x.ee;
        while (lo < hi) {
            const long long mid = (lo + hi) >> 1;
            if (x.d->ids[mid] < j) lo = mid + 1;
            else hi = mid;
        }
        if (lo < x.ee && x.d->ids[lo] == j) {
            const float q = x.d->logq[lo];
            if (!(q <= 1e-6f)) bits |= RL_STATUS_LOGQ;
            return q < INFINITY ? static_cast<double>(q) : -INFINITY;
        }
    }
    return -INFINITY;
}

__global__ void __launch_bounds__(kVerThreads) request_kernel(const VerArgs g) {
    __shared__ double red[kVerWarps];
    __shared__ int s_token;
    const rl_verify_args& a = g.a;
    const long long r = blockIdx.x;
    const int tid = threadIdx.x, V = static_cast<int>(a.V);
    int bits = 0;
    long long t0 = a.cu_q[r], t1 = a.cu_q[r + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.T) {
        bits |= RL_STATUS_LENGTHS;
        t0 = t1 = 0;
    }
    long long t = t0;
    for (; t + 1 < t1; ++t) {
        const int x = a.step_tokens[t + 1];
        const VerDist p = dist_at(g, 0, t, bits), q = dist_at(g, 1, t, bits);
        if (p.mode == VerDist::kNone || q.mode == VerDist::kNone) bits |= RL_STATUS_EMPTY_ROW;
        if (x < 0 || x >= V) {
            bits |= RL_STATUS_ID_RANGE;
            break;
        }
        const double lp = log_prob(p, x, bits), lq = log_prob(q, x, bits);
        const float u = unit_of(a.u[t], bits);
        if (!(static_cast<double>(u) * exp(lq) < exp(lp))) break;
        if (tid == 0) {
            a.tokens[t] = x;
            if (a.logq) a.logq[t] = static_cast<float>(lp);
        }
    }
    const long long accepted = t - t0;
    if (tid == 0) {
        a.accepted[r] = static_cast<int>(accepted);
        if (a.keep_lens) a.keep_lens[r] = (a.ctx_lens ? a.ctx_lens[r] : 0) + static_cast<int>(t1 > t0 ? accepted + 1 : 0);
    }
    if (t1 > t0) {
        const bool refused = t + 1 < t1;
        const VerDist p = dist_at(g, 0, t, bits);
        VerDist q{};
        if (refused) q = dist_at(g, 1, t, bits);
        const float u = unit_of(a.u_next[r], bits);
        const bool listed = p.mode == VerDist::kSupport;
        const long long n = listed ? p.ee - p.eb : V;
        auto token = [&](long long i) -> int { return listed ? p.d->ids[p.eb + i] : static_cast<int>(i); };
        // what is left of the i-th token; with `whole` all of it
        auto left = [&](long long i, bool whole) -> double {
            const int j = token(i);
            if (j < 0 || j >= V) {
                bits |= RL_STATUS_ID_RANGE;
                return 0.0;
            }
            double lp;
            if (listed) {
                const float l = p.d->logq[p.eb + i];
                if (!(l <= 1e-6f)) bits |= RL_STATUS_LOGQ;
                if (i > 0 && p.d->ids[p.eb + i - 1] >= j) bits |= RL_STATUS_ROW_ORDER;
                lp = l < INFINITY ? static_cast<double>(l) : -INFINITY;
            } else {
                lp = log_prob(p, j, bits);
            }
            const double v = exp(lp) - (whole ? 0.0 : exp(log_prob(q, j, bits)));
            return v > 0.0 ? v : 0.0;
        };
        bool whole = q.mode == VerDist::kNone;
        double total = 0.0;
        if (p.mode != VerDist::kNone) {
            for (int pass = 0; pass < 2; ++pass) {
                double v = 0.0;
                for (long long i = tid; i < n; i += kVerThreads) v += left(i, whole);
                total = vblock_sum(v, red);
                if (total > 0.0 || whole) break;
                whole = true;
            }
        }
        if (tid == 0) s_token = -1;
        __syncthreads();
        if (total > 0.0) {
            const double target = static_cast<double>(u) * total;
            double before = 0.0;
            for (long long i0 = 0; i0 < n; i0 += kVerThreads) {
                const long long i = i0 + tid;
                const double v = i < n ? left(i, whole) : 0.0;
                double c = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, c, o);
                    if ((tid & 31) >= o) c += y;
                }
                __syncthreads();
                if ((tid & 31) == 31) red[tid >> 5] = c;
                __syncthreads();
                double base = before;
                for (int w = 0; w < kVerWarps; ++w) {
                    if (w < (tid >> 5)) base += red[w];
                    before += red[w];
                }
                // (the last token with anything left, where rounding keeps the sum below the target)
                if (v > 0.0 && base + c - v <= target) atomicMax(&s_token, static_cast<int>(i));
            }
            __syncthreads();
        }
        if (tid == 0) {
            const int i = s_token;
            int y = -1;
            float l = -INFINITY;
            if (i >= 0) {
                y = token(i);
                l = static_cast<float>(listed ? static_cast<double>(p.d->logq[p.eb + i]) : log_prob(p, y, bits));
            } else {
                bits |= RL_STATUS_EMPTY_ROW;
            }
            a.tokens[t] = y;
            if (a.logq) a.logq[t] = l;
        }
    }
    set_status(g.status, bits);
}

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
        if (s.d.logits) s.rec = cv.take<VerRow>(static_cast<size_t>(a->T));
    if (bytes) *bytes = align_up(cv.off, 256);
    return g;
}

size_t verify_ws_bytes(const rl_verify_args* a) {
    size_t b = 0;
    verify_view(nullptr, a, nullptr, &b);
    return b;
}

int verify_impl(const rl_verify_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    const VerArgs g = verify_view(ws, a, status, nullptr);
    ProfScope prof(RL_PROF_OTHER, stream);
    int launches = 0;
    if (a->T > 0) {
        rows_kernel<<<dim3(static_cast<unsigned>(a->T), g.side[1].d.logits ? 2u : 1u, 1), kVerThreads, 0, stream>>>(g);
        ++launches;
    }
    if (a->R > 0) {
        request_kernel<<<static_cast<unsigned>(a->R), kVerThreads, 0, stream>>>(g);
        ++launches;
    }
    count_launch(launches);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // namespace rl
