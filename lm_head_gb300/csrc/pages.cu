// Page plans and cache writes of the generation path.
//
//  page_plan_kernel   one launch: every block covers a stretch of the step's tokens, and scans
//                     the requests' lengths (tiles of 2048 in shared memory) up to the end of its
//                     stretch; block b also writes the per-request outputs of tiles b,
//                     b + grid, ...  A new page's table entry is written with the first token in it
//                     (every new page has one).  No second launch, no block waits for another.
//                     26 us for 8192 requests with 2.1M tokens (25 MB written, 0.96 TB/s: every block
//                     scans the lengths up to its tokens), 8 us for 128 requests of one token (a
//                     chain of dependent loads and barriers in one block).
//  kv_append_kernel   16 bytes a thread and step, four loads in flight.  65,536 tokens of 8 heads of
//                     128 in 91.5 us: 5.9 TB/s, 88 % of a plain copy; 128 tokens of 4 heads in 3.1 us.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace rl {

constexpr int kPlanThreads = 256;
constexpr int kPlanItems = 8;                           // consecutive requests of one thread
constexpr int kPlanTile = kPlanThreads * kPlanItems;
constexpr int kPlanGroups = 1024;                       // groups held in shared memory: 8 KB, as much as a tile's lengths

// Exclusive block scan of two 64-bit sums; returns the thread's prefix, totals in (ta, tb).
struct Scan2 {
    long long a, b;
};
RL_DEVINL Scan2 block_scan2(long long a, long long b, long long* warp_a, long long* warp_b, long long& ta,
                            long long& tb) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += xa;
            ib += xb;
        }
    }
    __syncthreads();      // warp_a / warp_b of the previous tile have been read
    if (lane == 31) {
        warp_a[warp] = ia;
        warp_b[warp] = ib;
    }
    __syncthreads();
    long long pa = 0, pb = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) {
            pa = ta;
            pb = tb;
        }
        ta += warp_a[w];
        tb += warp_b[w];
    }
    return {pa + ia - a, pb + ib - b};
}

// pages that x tokens take
RL_DEVINL uint32_t pages_of(uint32_t x, int shift, uint32_t mask) { return (x >> shift) + ((x & mask) ? 1u : 0u); }

struct PlanArgs {
    rl_page_plan_args a;
    int32_t* status;
    long long tokens_per_block;
    int shift;           // log2(page_size)
};

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanArgs p) {
    // first token and first new page of each request, relative to the tile's; the request's
    // cached tokens; its prefix length
    __shared__ int s_q[kPlanTile + 1], s_n[kPlanTile + 1], s_ctx[kPlanTile], s_pre[kPlanTile];
    __shared__ long long warp_a[kPlanThreads / 32], warp_b[kPlanThreads / 32];
    __shared__ int s_go[kPlanGroups + 1], s_pl[kPlanGroups];     // the groups, where they fit
    const rl_page_plan_args& a = p.a;
    const bool grouped = a.group_offsets && a.G > 0 && a.positions;
    const bool go_shared = grouped && a.G <= kPlanGroups;
    if (go_shared)
        for (int i = threadIdx.x; i <= a.G; i += kPlanThreads) {
            s_go[i] = a.group_offsets[i];
            if (i < a.G) s_pl[i] = a.prefix_lens[i];
        }
    const int* go = go_shared ? s_go : a.group_offsets;
    const int* pl = go_shared ? s_pl : a.prefix_lens;            // read after the scan's barriers
    const long long used = a.free_used ? max(*a.free_used, 0) : 0;
    const uint32_t W = static_cast<uint32_t>(a.table_width);
    const uint32_t mask = static_cast<uint32_t>(a.page_size) - 1u;
    const long long t0 = min(blockIdx.x * p.tokens_per_block, static_cast<long long>(a.T));
    const long long t1 = min(t0 + p.tokens_per_block, static_cast<long long>(a.T));
    // the last block goes on past T, for the table entries of tokens that the step leaves out
    const bool closes = blockIdx.x == gridDim.x - 1;
    const long long tiles = (a.R + kPlanTile - 1) / kPlanTile;
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.q_lens) | reinterpret_cast<uintptr_t>(a.ctx_lens)) & 15) == 0;
    long long cu = 0, pages = 0;             // tokens and new pages before this tile
    int bits = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.cu_q[0] = 0;
        if (a.free_used && *a.free_used < 0) bits |= RL_STATUS_LENGTHS;
    }

    // page of the request's table entry `pi`: one of the pages handed out now, or one it has
    auto page_at = [&](long long r, int i, uint32_t pi) -> int {
        const uint32_t had = min(pages_of(static_cast<uint32_t>(s_ctx[i]), p.shift, mask), W);
        int page = -1;
        if (pi >= W) {
            bits |= RL_STATUS_PAGES;
        } else if (pi < had) {
            page = a.block_table[r * a.table_width + pi];
            if (page < 0 || page >= a.n_pages) {
                page = -1;
                bits |= RL_STATUS_PAGE_ID;
            }
        } else {
            const long long k = used + pages + s_n[i] + static_cast<int>(pi - had);
            if (k >= a.n_free) {
                bits |= RL_STATUS_PAGES;
            } else {
                page = a.free_pages[k];
                if (page < 0 || page >= a.n_pages) {
                    page = -1;
                    bits |= RL_STATUS_PAGE_ID;
                }
            }
        }
        return page;
    };

    for (long long tile = 0; tile < tiles; ++tile) {
        const bool mine = tile % gridDim.x == blockIdx.x;
        const long long next_mine = tile + (blockIdx.x + gridDim.x - tile % gridDim.x) % gridDim.x;
        if (!closes && cu >= t1 && next_mine >= tiles) break;        // the block's tokens and tiles are done
        const long long r0 = tile * kPlanTile;
        const int n = static_cast<int>(min(static_cast<long long>(kPlanTile), a.R - r0));
        int q[kPlanItems], ctx[kPlanItems], fresh[kPlanItems];
        long long qs = 0;
        uint32_t ns = 0;                     // at most 8 * 2^28
        const int mine0 = threadIdx.x * kPlanItems;
        if (aligned && mine0 + kPlanItems <= n) {
#pragma unroll
            for (int k = 0; k < kPlanItems; k += 4) {
                const int4 x = *reinterpret_cast<const int4*>(a.q_lens + r0 + mine0 + k), y = *reinterpret_cast<const int4*>(a.ctx_lens + r0 + mine0 + k);
                q[k] = x.x; q[k + 1] = x.y; q[k + 2] = x.z; q[k + 3] = x.w;
                ctx[k] = y.x; ctx[k + 1] = y.y; ctx[k + 2] = y.z; ctx[k + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kPlanItems; ++k) {
                q[k] = mine0 + k < n ? a.q_lens[r0 + mine0 + k] : 0;
                ctx[k] = mine0 + k < n ? a.ctx_lens[r0 + mine0 + k] : 0;
            }
        }
#pragma unroll
        for (int k = 0; k < kPlanItems; ++k) {
            if (q[k] < 0 || ctx[k] < 0) {
                if (mine) bits |= RL_STATUS_LENGTHS;
                q[k] = max(q[k], 0);
                ctx[k] = max(ctx[k], 0);
            }
            const uint32_t had = pages_of(static_cast<uint32_t>(ctx[k]), p.shift, mask);
            const uint32_t need = pages_of(static_cast<uint32_t>(ctx[k]) + static_cast<uint32_t>(q[k]), p.shift, mask);
            fresh[k] = static_cast<int>(min(need, W) - min(had, W));
            if (mine && need > W && q[k] > 0) bits |= RL_STATUS_PAGES;
            qs += q[k];
            ns += static_cast<uint32_t>(fresh[k]);
        }
        long long tq, tn;
        const Scan2 s = block_scan2(qs, static_cast<long long>(ns), warp_a, warp_b, tq, tn);
        const bool tokens = cu < t1 && cu + tq > t0;      // some of the block's tokens are here
        const bool excess = closes && cu + tq > a.T;
        if (mine || tokens || excess) {
            // tile-relative sums past 2^31 are cut there: they lie past T, which is below it
            long long iq = s.a, in = s.b;
            int g = 0;
            if (grouped && tokens) {
                const long long r = r0 + threadIdx.x * kPlanItems;
                int lo = 0, hi = static_cast<int>(a.G);   // first g with group_offsets[g + 1] > r
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (go[mid + 1] > r) hi = mid;
                    else lo = mid + 1;
                }
                g = lo;
            }
#pragma unroll
            for (int k = 0; k < kPlanItems; ++k) {
                const int i = threadIdx.x * kPlanItems + k;
                s_q[i] = static_cast<int>(min(iq, static_cast<long long>(INT_MAX)));
                s_n[i] = static_cast<int>(min(in, static_cast<long long>(INT_MAX)));
                s_ctx[i] = ctx[k];
                int pre = 0;
                if (grouped && tokens && i < n) {
                    while (g < a.G && go[g + 1] <= r0 + i) ++g;
                    if (g < a.G && go[g] <= r0 + i) pre = max(pl[g], 0);
                }
                s_pre[i] = pre;
                iq += q[k];
                in += fresh[k];
                if (mine && i < n) {
                    a.cu_q[r0 + i + 1] = static_cast<int>(min(cu + iq, static_cast<long long>(INT_MAX)));
                    a.kv_lens[r0 + i] = static_cast<int>(
                        min(static_cast<long long>(ctx[k]) + q[k], static_cast<long long>(INT_MAX)));
                }
            }
            if (threadIdx.x == kPlanThreads - 1) {
                s_q[kPlanTile] = static_cast<int>(min(iq, static_cast<long long>(INT_MAX)));
                s_n[kPlanTile] = static_cast<int>(min(in, static_cast<long long>(INT_MAX)));
            }
            __syncthreads();
        }
        if (tokens) {
            const long long b0 = max(t0, cu), b1 = min(t1, cu + tq);
            // four consecutive tokens a thread, aligned to the block's first token (a multiple of 4)
            for (long long t = (b0 & ~3ll) + threadIdx.x * 4; t < b1; t += kPlanThreads * 4) {
                const long long ta = max(t, b0), tb = min(t + 4, b1);
                // tokens of the tile fit 31 bits up to T; those past it are clamped with the sums
                const int x0 = static_cast<int>(min(t - cu, static_cast<long long>(INT_MAX - 4))), xa = static_cast<int>(min(ta - cu, static_cast<long long>(INT_MAX - 4)));
                const int take = static_cast<int>(tb - t), skip = static_cast<int>(ta - t);
                int lo = 0, hi = n;                        // last i with s_q[i] <= xa
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_q[mid] <= xa) lo = mid;
                    else hi = mid;
                }
                long long slot[4];
                int pos[4];
                int page = -1, page_r = -1, from = s_q[lo], to = s_q[lo + 1], ctx0 = s_ctx[lo], pre0 = s_pre[lo];
                uint32_t page_i = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < skip || k >= take) continue;
                    if (x0 + k >= to) {
                        while (lo + 1 < kPlanTile && s_q[lo + 1] <= x0 + k) ++lo;
                        from = s_q[lo];
                        to = s_q[lo + 1];
                        ctx0 = s_ctx[lo];
                        pre0 = s_pre[lo];
                    }
                    const uint32_t at = static_cast<uint32_t>(ctx0) + static_cast<uint32_t>(x0 + k - from);
                    const uint32_t pi = at >> p.shift;
                    if (lo != page_r || pi != page_i) {
                        page = page_at(r0 + lo, lo, pi);
                        page_r = lo;
                        page_i = pi;
                    }
                    // the first token of a new page writes its entry
                    if ((at & mask) == 0 && pi < W) a.block_table[(r0 + lo) * a.table_width + pi] = page;
                    slot[k] = page < 0 ? -1 : (static_cast<long long>(page) << p.shift) + (at & mask);
                    pos[k] = static_cast<int>(min(static_cast<unsigned long long>(at) + pre0, static_cast<unsigned long long>(INT_MAX)));
                }
                const bool whole = ta == t && tb == t + 4;
                if (whole && (reinterpret_cast<uintptr_t>(a.slot_map) & 15) == 0) {
                    longlong2* d = reinterpret_cast<longlong2*>(a.slot_map + t);
                    d[0] = make_longlong2(slot[0], slot[1]);
                    d[1] = make_longlong2(slot[2], slot[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (t + k >= ta && t + k < tb) a.slot_map[t + k] = slot[k];
                }
                if (a.positions) {
                    if (whole && (reinterpret_cast<uintptr_t>(a.positions) & 15) == 0) {
                        *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (t + k >= ta && t + k < tb) a.positions[t + k] = pos[k];
                    }
                }
            }
        }
        if (excess) {
            // the new pages whose first token lies past T, one a thread and step (a row's width bounds them)
            for (long long j = threadIdx.x; j < tn; j += kPlanThreads) {
                int lo = 0, hi = n;                        // last i with s_n[i] <= j
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (s_n[mid] <= j) lo = mid;
                    else hi = mid;
                }
                const uint32_t c = static_cast<uint32_t>(s_ctx[lo]);
                const uint32_t pi = min(pages_of(c, p.shift, mask), W) + static_cast<uint32_t>(j - s_n[lo]);
                const long long first = (static_cast<long long>(pi) << p.shift) - c;      // in the request's step
                if (pi < W && cu + s_q[lo] + first >= a.T) a.block_table[(r0 + lo) * a.table_width + pi] = page_at(r0 + lo, lo, pi);
            }
        }
        cu += tq;
        pages += tn;
        if (tile == tiles - 1) {
            if (mine && threadIdx.x == 0) {
                *a.free_used_out = static_cast<int>(
                    min(min(used + pages, max(used, static_cast<long long>(a.n_free))), static_cast<long long>(INT_MAX)));
                if (cu != a.T) bits |= RL_STATUS_LENGTHS;
            }
            // tokens that no request has
            for (long long t = max(t0, cu) + threadIdx.x; t < t1; t += kPlanThreads) {
                a.slot_map[t] = -1;
                if (a.positions) a.positions[t] = -1;
            }
        }
        if (mine || tokens || excess) __syncthreads();               // the tile's shared arrays have been read
    }
    if (tiles == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        *a.free_used_out = static_cast<int>(used);
        if (a.T != 0) bits |= RL_STATUS_LENGTHS;
    }
    if (tiles == 0)
        for (long long t = t0 + threadIdx.x; t < t1; t += kPlanThreads) {
            a.slot_map[t] = -1;
            if (a.positions) a.positions[t] = -1;
        }
    if (grouped && blockIdx.x == 0 && tiles > 0)                     // (the scan's barriers have been passed)
        for (int g = threadIdx.x; g < a.G; g += kPlanThreads)
            if (go[g] < 0 || go[g + 1] < go[g] || go[g + 1] > a.R) bits |= RL_STATUS_LENGTHS;
    set_status(p.status, bits);
}

int page_plan_impl(const rl_page_plan_args* a, int32_t* status, cudaStream_t stream) {
    PlanArgs p;
    p.a = *a;
    p.status = status;
    p.shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    // up to two blocks a multiprocessor, a whole number of 1024-token steps each (every block scans the
    // lengths up to its tokens, so more of them scan more: four a multiprocessor took 39 us against
    // 26 us for 8192 requests and 2.1M tokens)
    const long long cap = 2ll * num_sms();
    const long long steps = (a->T + 1023) / 1024;
    p.tokens_per_block = ((steps + cap - 1) / cap) * 1024;
    // lengths in place: every block reads them all, so one block does the step (a thread has read the lengths of its
    // requests when it writes them)
    if (a->R > 0 && a->kv_lens == a->ctx_lens) p.tokens_per_block = steps * 1024;
    if (p.tokens_per_block == 0) p.tokens_per_block = 1024;
    long long grid = (a->T + p.tokens_per_block - 1) / p.tokens_per_block;
    if (grid < 1) grid = 1;
    ProfScope prof(RL_PROF_OTHER, stream);
    page_plan_kernel<<<static_cast<unsigned>(grid), kPlanThreads, 0, stream>>>(p);
    count_launch();
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// ---- cache writes --------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

struct AppendArgs {
    rl_kv_append_args a;
    int32_t* status;
    long long units;      // units of one tensor: T * Hkv * (D / elements a unit)
    int per_head;         // units of a head
    int shift;            // log2(page_size)
};

// Unit: 16 bytes where every row is 16-byte aligned, else one element.
template <typename Unit>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs p) {
    const rl_kv_append_args& a = p.a;
    constexpr int E = sizeof(Unit) / 2;
    const long long slots = a.n_pages << p.shift;
    const int per_token = p.per_head * a.Hkv;
    const int mask = a.page_size - 1;
    const bool second = blockIdx.y != 0;
    const uint16_t* src = static_cast<const uint16_t*>(second ? a.v : a.k);
    uint16_t* dst = static_cast<uint16_t*>(second ? a.v_cache : a.k_cache);
    const long long st = second ? a.v_stride_t : a.k_stride_t, sh = second ? a.v_stride_h : a.k_stride_h;
    int bits = 0;
    const long long step = static_cast<long long>(gridDim.x) * kAppendThreads * kAppendUnroll;
    for (long long base = (static_cast<long long>(blockIdx.x) * kAppendUnroll) * kAppendThreads + threadIdx.x;
         base < p.units; base += step) {
        Unit val[kAppendUnroll];
        long long to[kAppendUnroll];
#pragma unroll
        for (int j = 0; j < kAppendUnroll; ++j) {
            const long long x = base + static_cast<long long>(j) * kAppendThreads;
            to[j] = -1;
            if (x >= p.units) continue;
            long long t;
            int rest;
            if (p.units <= UINT_MAX) {                   // 32-bit division where it is enough
                const uint32_t q = static_cast<uint32_t>(x) / static_cast<uint32_t>(per_token);
                t = q;
                rest = static_cast<int>(static_cast<uint32_t>(x) - q * static_cast<uint32_t>(per_token));
            } else {
                t = x / per_token;
                rest = static_cast<int>(x - t * per_token);
            }
            const int h = static_cast<uint32_t>(rest) / static_cast<uint32_t>(p.per_head);
            const int d = (rest - h * p.per_head) * E;
            const long long slot = a.slot_map[t];
            if (slot < 0) continue;
            if (slot >= slots) {
                bits |= RL_STATUS_PAGE_ID;
                continue;
            }
            val[j] = *reinterpret_cast<const Unit*>(src + t * st + h * sh + d);
            to[j] = ((((slot >> p.shift) * a.Hkv + h) << p.shift) + (slot & mask)) * a.D + d;
        }
#pragma unroll
        for (int j = 0; j < kAppendUnroll; ++j)
            if (to[j] >= 0) *reinterpret_cast<Unit*>(dst + to[j]) = val[j];
    }
    set_status(p.status, bits);
}

int kv_append_impl(const rl_kv_append_args* a, int32_t* status, cudaStream_t stream) {
    if (a->T == 0) return RL_OK;
    AppendArgs p;
    p.a = *a;
    p.status = status;
    p.shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    auto wide = [&](const void* base, int64_t st, int64_t sh) {
        return (reinterpret_cast<uintptr_t>(base) & 15) == 0 && st % 8 == 0 && sh % 8 == 0;
    };
    const bool vec = a->D % 8 == 0 && wide(a->k, a->k_stride_t, a->k_stride_h) && wide(a->v, a->v_stride_t, a->v_stride_h);
    p.per_head = vec ? a->D / 8 : a->D;
    p.units = a->T * a->Hkv * p.per_head;
    // one step a thread up to 16 blocks a multiprocessor (8 of each tensor), then more steps
    long long blocks = (p.units + kAppendThreads * kAppendUnroll - 1) / (kAppendThreads * kAppendUnroll);
    const long long cap = 8ll * num_sms();
    if (blocks > cap) blocks = cap;
    const dim3 grid(static_cast<unsigned>(blocks), 2, 1);
    ProfScope prof(RL_PROF_OTHER, stream);
    if (vec)
        kv_append_kernel<uint4><<<grid, kAppendThreads, 0, stream>>>(p);
    else
        kv_append_kernel<uint16_t><<<grid, kAppendThreads, 0, stream>>>(p);
    count_launch();
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // namespace rl
