// Pages of a cache given back, shared, copied and moved together.
//
// Which pages are in use is what the tables say: a call marks the pages that its rows name in a
// bitmap (a bit a page, by atomic OR, whose order does not matter) and reads the answer off the
// bitmap in the order of the ids.  So a page that several rows share needs no count of its
// owners, and the same inputs give the same lists.
//
//  mark_kernel     a warp takes 256 entries of a row
//  sweep_kernel    release: the ids to give back, ascending; every block counts the words before its
//                  own (the bitmaps of 131,072 pages are 32 KB), so that no block waits for another
//  fork_plan_kernel, fork_rows_kernel
//                  fork: one block numbers the new pages, then a warp writes 256 entries of a child's row
//  compact_plan_kernel, compact_rows_kernel
//                  compact: the k-th live page past the number of live pages goes to the k-th hole below
//                  it (the fewest moves), then the tables by a look-up in the bitmap's running counts
//  page_copy_kernel  a warp copies a head's tokens of one page
//
// Lists and tables are latency: launches, and loads that follow on one another (a row's length, its entries, their words; the
// counts before a block's words).  A release of 128 requests 8.3 us, of 8192 13.0 us: by themselves, caches cold, the marks take 7.7 us
// with L2 at 16 % of its rate and the sweep 11 us with L2 at 3 %, most of it each block's count; a compaction's lists and tables
// 12 us (the plan by itself 11).  Copies are HBM:
// 2.35 GB read and written for 512 sequences' moves in 700 us, 6.7 TB/s, as a copy's rate; 0.8 GB of half-filled pages in
// 257 us, 6.3 TB/s.
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace rl {

constexpr int kMoveThreads = 256;
constexpr int kSeg = 256;                 // table entries of one warp step
constexpr int kSweepThreads = 512;

// Entries of a row that its length takes, cut to the row's width.
RL_DEVINL long long entries_of(int len, int shift, long long W, int& bits) {
    if (len < 0) {
        bits |= RL_STATUS_LENGTHS;
        return 0;
    }
    const long long n = (static_cast<long long>(len) + (1ll << shift) - 1) >> shift;
    if (n > W) bits |= RL_STATUS_PAGES;
    return min(n, W);
}

struct MarkRows {
    const int32_t* lens;       // entries below lens are marked
    const int32_t* keep;       // NULL, or: those below keep in `live`, the others in `drop`
    const int32_t* table;
    long long rows, width, segs;
};
struct MarkArgs {
    MarkRows t[2];
    uint32_t *live, *drop;
    long long n_pages;
    int shift;
    int32_t* status;
};

__global__ void __launch_bounds__(kMoveThreads) mark_kernel(const MarkArgs p) {
    let_next_start();
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    const long long first = p.t[0].rows * p.t[0].segs, units = first + p.t[1].rows * p.t[1].segs;
    int bits = 0;
    for (long long id = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); id < units; id += warps) {
        const bool second = id >= first;
        const MarkRows& m = p.t[second ? 1 : 0];
        const long long x = second ? id - first : id, r = x / m.segs, j0 = (x - r * m.segs) * kSeg;
        const int len = m.lens[r];
        int mine = 0;
        const long long n = entries_of(len, p.shift, m.width, mine);
        long long left = n;
        if (m.keep) {
            int keep = m.keep[r];
            if (keep > max(len, 0)) mine |= RL_STATUS_LENGTHS;
            keep = min(keep, max(len, 0));
            left = min(entries_of(keep, p.shift, m.width, mine), n);
        }
        if (j0 == 0) bits |= mine;
        const long long end = min(n, j0 + kSeg);
        for (long long j = j0 + lane; j < end; j += 32) {
            const int page = m.table[r * m.width + j];
            if (page < 0 || page >= p.n_pages) bits |= RL_STATUS_PAGE_ID;
            else atomicOr((j < left ? p.live : p.drop) + (page >> 5), 1u << (page & 31));
        }
    }
    set_status(p.status, bits);
}

// f(words, their number) over a bitmap's words [0, n), 16 bytes a thread and four loads at a time (bitmaps are 16-byte aligned and
// padded to 16 bytes with zeros).
template <typename F>
RL_DEVINL void each_words(const uint32_t* map, long long n, F f) {
    const uint4* m = reinterpret_cast<const uint4*>(map);
    const long long q = (n + 3) / 4;
    for (long long i = threadIdx.x; i < q; i += 4 * blockDim.x) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i + k * blockDim.x < q ? m[i + k * blockDim.x] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) f(v[k], (i + k * blockDim.x) * 4);
    }
}
RL_DEVINL int bits_of(uint4 v) { return __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w); }

// The block's sum of v, in every thread.
RL_DEVINL long long block_total(long long v, long long* red) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    long long s = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) s += red[w];
    return s;
}
// Exclusive block scan of v; the block's total in `total`.
RL_DEVINL int block_prefix(int v, int* red, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int i = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, i, o);
        if (lane >= o) i += x;
    }
    __syncthreads();
    if (lane == 31) red[warp] = i;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
        if (w == warp) before = total;
        total += red[w];
    }
    return before + i - v;
}

// ---- release ---------------------------------------------------------------------------
struct SweepArgs {
    const uint32_t *live, *drop;
    long long words, per_block;          // words of a bitmap, of a block
    int32_t* free_pages;
    long long n_free;
    const int32_t* free_used;
    int32_t* free_used_out;
    int32_t* status;
};

__global__ void __launch_bounds__(kSweepThreads) sweep_kernel(const SweepArgs p) {
    __shared__ long long red[kSweepThreads / 32];
    __shared__ int redi[kSweepThreads / 32];
    const long long w0 = blockIdx.x * p.per_block, w1 = min(w0 + p.per_block, p.words);
    int bits = 0;
    long long before = 0, all = 0;
    wait_for_previous();
    const uint4* live4 = reinterpret_cast<const uint4*>(p.live);
    each_words(p.drop, p.words, [&](uint4 v, long long w) {
        if (w >= p.words) return;
        const uint4 l = live4[w / 4];
        const int n = bits_of(make_uint4(v.x & ~l.x, v.y & ~l.y, v.z & ~l.z, v.w & ~l.w));
        all += n;
        if (w < w0) before += n;
    });
    all = block_total(all, red);
    long long rank = block_total(before, red);
    long long used = *p.free_used;
    if (used < 0) {
        bits |= RL_STATUS_LENGTHS;
        used = 0;
    }
    const long long base = used - all;                 // where the lowest id goes
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (base < 0 || used > p.n_free) bits |= RL_STATUS_PAGES;
        *p.free_used_out = static_cast<int>(max(base, 0ll));
    }
    for (long long w = w0; w < w1; w += kSweepThreads) {
        const long long mine = w + threadIdx.x;
        uint32_t x = mine < w1 ? p.drop[mine] & ~p.live[mine] : 0u;
        int total;
        long long at = base + rank + block_prefix(__popc(x), redi, total);
        while (x) {
            const int b = __ffs(x) - 1;
            x &= x - 1;
            if (at >= 0 && at < p.n_free) p.free_pages[at] = static_cast<int>(mine * 32 + b);
            ++at;
        }
        rank += total;
    }
    set_status(p.status, bits);
}

static long long words_of(int64_t n_pages) { return (n_pages + 127) / 128 * 4; }      // whole 16 bytes
static int mark_blocks(long long units) {
    const long long blocks = (units + kMoveThreads / 32 - 1) / (kMoveThreads / 32), cap = 8ll * num_sms();
    return static_cast<int>(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}
static MarkRows mark_rows(const int32_t* lens, const int32_t* keep, const int32_t* table, int64_t rows, int64_t width) {
    // (a row of no width still has its lengths looked at)
    const long long segs = width > 0 ? (width + kSeg - 1) / kSeg : 1;
    return MarkRows{lens, keep, table, rows, width, segs};
}

size_t page_release_ws_bytes(int64_t n_pages) { return align_up(static_cast<size_t>(words_of(n_pages)) * 8, 256); }

int page_release_impl(const rl_page_release_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    const long long words = words_of(a->n_pages);
    uint32_t* live = static_cast<uint32_t*>(ws);
    ProfScope prof(RL_PROF_OTHER, stream);
    if (words > 0 && cudaMemsetAsync(ws, 0, static_cast<size_t>(words) * 8, stream) != cudaSuccess) return RL_ERR_CUDA;
    MarkArgs m{};
    m.t[0] = mark_rows(a->kv_lens, a->keep_lens, a->block_table, a->R, a->table_width);
    m.t[1] = mark_rows(a->held_lens, nullptr, a->held_table, a->G, a->held_width);
    m.live = live;
    m.drop = live + words;
    m.n_pages = a->n_pages;
    m.shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    m.status = status;
    mark_kernel<<<mark_blocks(m.t[0].rows * m.t[0].segs + m.t[1].rows * m.t[1].segs), kMoveThreads, 0, stream>>>(m);
    SweepArgs s{live, live + words, words, 0, a->free_pages, a->n_free, a->free_used, a->free_used_out, status};
    // a step of the block each, up to a block a multiprocessor: every block counts the words before its own
    long long steps = (words + kSweepThreads - 1) / kSweepThreads;
    if (steps < 1) steps = 1;
    const long long grid = steps < num_sms() ? steps : num_sms();
    s.per_block = (steps + grid - 1) / grid * kSweepThreads;
    const int rc = launch_after(sweep_kernel, dim3(static_cast<unsigned>(grid)), kSweepThreads, 0, true, stream, s);
    if (rc != RL_OK) return rc;
    count_launch(2);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// ---- fork ------------------------------------------------------------------------------
constexpr int kForkThreads = 512;

struct ForkArgs {
    rl_page_fork_args a;
    int32_t* claim;        // [R] the first entry whose child the row is (set for the rows named only)
    int32_t* takes;        // [C] the child's row is written
    int32_t* status;
    int shift;
};

__global__ void __launch_bounds__(kForkThreads) fork_plan_kernel(const ForkArgs p) {
    __shared__ int red[kForkThreads / 32];
    let_next_start();
    const rl_page_fork_args& a = p.a;
    const int mask = a.page_size - 1;
    int bits = 0;
    auto row_ok = [&](int r) { return r >= 0 && r < a.R; };
    for (long long c = threadIdx.x; c < a.C; c += kForkThreads) {
        const int x = a.children[c], y = a.parents[c];
        if (row_ok(x)) p.claim[x] = INT_MAX;
        if (row_ok(y)) p.claim[y] = INT_MAX;
    }
    __syncthreads();
    for (long long c = threadIdx.x; c < a.C; c += kForkThreads)
        if (row_ok(a.children[c])) atomicMin(p.claim + a.children[c], static_cast<int>(c));
    __syncthreads();
    long long used = *a.free_used;
    if (used < 0) {
        bits |= RL_STATUS_LENGTHS;
        used = 0;
    }
    long long fresh = 0;                              // new pages of the tiles before
    for (long long c0 = 0; c0 < a.C; c0 += kForkThreads) {
        const long long c = c0 + threadIdx.x;
        int child = -1, parent = -1, len = 0;
        bool ok = false;
        if (c < a.C) {
            child = a.children[c];
            parent = a.parents[c];
            len = a.lens[c];
            ok = row_ok(child) && row_ok(parent);
            // a row that is twice a child, or a child and a parent, has no order in which it could be written
            if (ok) ok = __ldcg(p.claim + child) == c && __ldcg(p.claim + parent) == INT_MAX;      // (the atomics work in L2)
            if (!ok) bits |= RL_STATUS_ID_RANGE;
            if (ok && (len < 0 || len > a.kv_lens[parent])) {
                bits |= RL_STATUS_LENGTHS;
                ok = false;
            }
            if (ok && ((static_cast<long long>(len) + mask) >> p.shift) > a.table_width) {
                bits |= RL_STATUS_PAGES;
                ok = false;
            }
        }
        const int part = ok ? len & mask : 0;
        int total;
        const long long k = used + fresh + block_prefix(part > 0 ? 1 : 0, red, total);
        fresh += total;
        if (c < a.C) {
            int src = -1, dst = -1;
            if (part > 0) {
                src = a.block_table[parent * a.table_width + (len >> p.shift)];
                if (k < a.n_free) dst = a.free_pages[k];
                else bits |= RL_STATUS_PAGES;
                if (src < 0 || src >= a.n_pages) {
                    bits |= RL_STATUS_PAGE_ID;
                    src = -1;
                }
                if (k < a.n_free && (dst < 0 || dst >= a.n_pages)) {
                    bits |= RL_STATUS_PAGE_ID;
                    dst = -1;
                }
            }
            const bool copies = src >= 0 && dst >= 0;
            p.takes[c] = ok ? (part > 0 ? dst : -1) : INT_MIN;      // the new page, or -1; INT_MIN: left out
            a.src[c] = copies ? src : -1;
            a.dst[c] = copies ? dst : -1;
            a.tokens[c] = copies ? part : 0;
            if (ok) a.kv_lens[child] = len;                // (no parent of the call, so nobody reads it)
        }
    }
    if (threadIdx.x == 0)
        *a.free_used_out = static_cast<int>(min(min(used + fresh, max(used, static_cast<long long>(a.n_free))), static_cast<long long>(INT_MAX)));
    set_status(p.status, bits);
}

__global__ void __launch_bounds__(kMoveThreads) fork_rows_kernel(const ForkArgs p) {
    const rl_page_fork_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const long long segs = (a.table_width + kSeg - 1) / kSeg, units = a.C * segs;
    const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    int bits = 0;
    wait_for_previous();
    for (long long id = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); id < units; id += warps) {
        const long long c = id / segs, j0 = (id - c * segs) * kSeg, end = min(j0 + kSeg, static_cast<long long>(a.table_width));
        const int page = p.takes[c];
        if (page == INT_MIN) continue;
        const int full = a.lens[c] >> p.shift;
        const int32_t* from = a.block_table + a.parents[c] * a.table_width;
        int32_t* to = a.block_table + a.children[c] * a.table_width;
        for (long long j = j0 + lane; j < end; j += 32) {
            int e = -1;
            if (j < full) {
                e = from[j];
                if (e < 0 || e >= a.n_pages) {
                    e = -1;
                    bits |= RL_STATUS_PAGE_ID;
                }
            } else if (j == full) {
                e = page;
            }
            to[j] = e;
        }
    }
    set_status(p.status, bits);
}

size_t page_fork_ws_bytes(int64_t R, int64_t C) { return align_up(static_cast<size_t>(R) * 4, 256) + align_up(static_cast<size_t>(C) * 4, 256); }

int page_fork_impl(const rl_page_fork_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    ForkArgs p;
    p.a = *a;
    Carve cv(ws);
    p.claim = cv.take<int32_t>(static_cast<size_t>(a->R));
    p.takes = cv.take<int32_t>(static_cast<size_t>(a->C));
    p.status = status;
    p.shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    ProfScope prof(RL_PROF_OTHER, stream);
    fork_plan_kernel<<<1, kForkThreads, 0, stream>>>(p);
    int launches = 1;
    const long long units = a->C * ((a->table_width + kSeg - 1) / kSeg);
    if (units > 0) {
        const int rc = launch_after(fork_rows_kernel, dim3(static_cast<unsigned>(mark_blocks(units))), kMoveThreads, 0, true, stream, p);
        if (rc != RL_OK) return rc;
        ++launches;
    }
    count_launch(launches);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// ---- compact -----------------------------------------------------------------------------
struct CompactArgs {
    rl_page_compact_args a;
    const uint32_t* live;
    int32_t* before;         // [words] live pages before a word's
    long long words, per_block;
    int32_t* status;
    int shift;
};

__global__ void __launch_bounds__(kSweepThreads) compact_plan_kernel(const CompactArgs p) {
    __shared__ long long red[kSweepThreads / 32];
    __shared__ int redi[kSweepThreads / 32];
    const rl_page_compact_args& a = p.a;
    const long long w0 = blockIdx.x * p.per_block, w1 = min(w0 + p.per_block, p.words);
    long long before = 0, all = 0;
    wait_for_previous();
    let_next_start();
    each_words(p.live, p.words, [&](uint4 v, long long w) {
        const int n = bits_of(v);
        all += n;
        if (w < w0) before += n;
    });
    const long long n_live = block_total(all, red);
    long long rank = block_total(before, red);
    // live pages below n_live: they stay
    long long stay = 0;
    each_words(p.live, (n_live + 31) / 32, [&](uint4 v, long long w) {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long n = n_live - (w + k) * 32;             // pages of the word below n_live
            if (n > 0) stay += __popc(n < 32 ? x[k] & ((1u << n) - 1u) : x[k]);
        }
    });
    stay = block_total(stay, red);
    const long long moves = n_live - stay;
    for (long long w = w0; w < w1; w += kSweepThreads) {
        const long long mine = w + threadIdx.x;
        const uint32_t x = mine < w1 ? p.live[mine] : 0u;
        int total;
        const long long lives = rank + block_prefix(__popc(x), redi, total);       // live pages before the word
        if (mine < w1) {
            p.before[mine] = static_cast<int>(lives);
            const long long id0 = mine * 32;
            int seen = 0;
            for (int b = 0; b < 32; ++b) {
                const long long id = id0 + b;
                if (id >= a.n_pages) break;
                const bool on = (x >> b) & 1u;
                if (id >= n_live && on) a.src[lives + seen - stay] = static_cast<int>(id);
                if (id < n_live && !on) a.dst[id - lives - seen] = static_cast<int>(id);
                seen += on;
            }
        }
        rank += total;
    }
    const long long tid = static_cast<long long>(blockIdx.x) * kSweepThreads + threadIdx.x, threads = static_cast<long long>(gridDim.x) * kSweepThreads;
    for (long long i = tid; i < a.n_pages; i += threads) a.free_pages[i] = static_cast<int>(i);
    for (long long i = moves + tid; i < a.n_pages / 2; i += threads) {
        a.src[i] = -1;
        a.dst[i] = -1;
    }
    if (tid == 0) *a.free_used_out = static_cast<int>(n_live);
}

__global__ void __launch_bounds__(kMoveThreads) compact_rows_kernel(const CompactArgs p) {
    const rl_page_compact_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const long long segs[2] = {(a.table_width + kSeg - 1) / kSeg, (a.prefix_width + kSeg - 1) / kSeg};
    const long long first = a.R * segs[0], units = first + a.G * segs[1];
    const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    wait_for_previous();
    const int n_live = *a.free_used_out;
    int stay = 0;
    if (n_live > 0) {
        const int w = (n_live - 1) >> 5, k = n_live - w * 32;              // pages of the word below n_live: 1 to 32
        stay = p.before[w] + __popc(k < 32 ? p.live[w] & ((1u << k) - 1u) : p.live[w]);
    }
    int none = 0;
    for (long long id = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); id < units; id += warps) {
        const bool second = id >= first;
        const long long x = second ? id - first : id, sg = segs[second ? 1 : 0], r = x / sg, j0 = (x - r * sg) * kSeg;
        const long long W = second ? a.prefix_width : a.table_width;
        const int32_t* from = (second ? a.prefix_table : a.block_table) + r * W;
        int32_t* to = (second ? a.prefix_table_out : a.block_table_out) + r * W;
        const long long n = entries_of((second ? a.prefix_lens : a.kv_lens)[r], p.shift, W, none), end = min(j0 + kSeg, W);
        for (long long j = j0 + lane; j < end; j += 32) {
            int e = -1;
            if (j < n) {
                const int page = from[j];
                if (page >= 0 && page < a.n_pages) {
                    e = page;
                    if (page >= n_live) e = a.dst[p.before[page >> 5] + __popc(p.live[page >> 5] & ((1u << (page & 31)) - 1u)) - stay];
                }
            }
            to[j] = e;
        }
    }
}

size_t page_compact_ws_bytes(int64_t n_pages) { return 2 * align_up(static_cast<size_t>(words_of(n_pages)) * 4, 256); }

int page_compact_impl(const rl_page_compact_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    const long long words = words_of(a->n_pages);
    Carve cv(ws);
    uint32_t* live = cv.take<uint32_t>(static_cast<size_t>(words));
    CompactArgs p;
    p.a = *a;
    p.live = live;
    p.before = cv.take<int32_t>(static_cast<size_t>(words));
    p.words = words;
    p.status = status;
    p.shift = __builtin_ctz(static_cast<unsigned>(a->page_size));
    ProfScope prof(RL_PROF_OTHER, stream);
    if (words > 0 && cudaMemsetAsync(live, 0, static_cast<size_t>(words) * 4, stream) != cudaSuccess) return RL_ERR_CUDA;
    MarkArgs m{};
    m.t[0] = mark_rows(a->kv_lens, nullptr, a->block_table, a->R, a->table_width);
    m.t[1] = mark_rows(a->prefix_lens, nullptr, a->prefix_table, a->G, a->prefix_width);
    m.live = m.drop = live;
    m.n_pages = a->n_pages;
    m.shift = p.shift;
    m.status = status;
    mark_kernel<<<mark_blocks(m.t[0].rows * m.t[0].segs + m.t[1].rows * m.t[1].segs), kMoveThreads, 0, stream>>>(m);
    long long steps = (words + kSweepThreads - 1) / kSweepThreads;
    if (steps < 1) steps = 1;
    const long long grid = steps < num_sms() ? steps : num_sms();
    p.per_block = (steps + grid - 1) / grid * kSweepThreads;
    int rc = launch_after(compact_plan_kernel, dim3(static_cast<unsigned>(grid)), kSweepThreads, 0, true, stream, p);
    if (rc != RL_OK) return rc;
    int launches = 2;
    const long long units = a->R * ((a->table_width + kSeg - 1) / kSeg) + a->G * ((a->prefix_width + kSeg - 1) / kSeg);
    if (units > 0) {
        rc = launch_after(compact_rows_kernel, dim3(static_cast<unsigned>(mark_blocks(units))), kMoveThreads, 0, true, stream, p);
        if (rc != RL_OK) return rc;
        ++launches;
    }
    count_launch(launches);
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

// ---- copies ------------------------------------------------------------------------------
struct CopyArgs {
    rl_page_copy_args a;
    int32_t* status;
    long long units;         // n * layers * 2 * Hkv
    long long layer_bytes;
    int token_bytes;
};

// Unit: 16 bytes where tokens and layers start on them, else 2 (every type is a multiple).
template <typename Unit>
__global__ void __launch_bounds__(kMoveThreads) page_copy_kernel(const CopyArgs p) {
    const rl_page_copy_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const long long warps = static_cast<long long>(gridDim.x) * (kMoveThreads / 32);
    const uint32_t per_pair = static_cast<uint32_t>(a.layers) * 2u * static_cast<uint32_t>(a.Hkv);
    const long long head_bytes = static_cast<long long>(a.page_size) * p.token_bytes;
    int bits = 0;
    for (long long id = static_cast<long long>(blockIdx.x) * (kMoveThreads / 32) + (threadIdx.x >> 5); id < p.units; id += warps) {
        const long long i = id / per_pair;
        const uint32_t rest = static_cast<uint32_t>(id - i * per_pair);
        const uint32_t h = rest % static_cast<uint32_t>(a.Hkv), lt = rest / static_cast<uint32_t>(a.Hkv);
        const int src = a.src[i], dst = a.dst[i];
        if (src < 0 || dst < 0) continue;
        int n = a.tokens ? a.tokens[i] : a.page_size;
        if (src >= a.n_pages || dst >= a.n_pages) {
            bits |= RL_STATUS_PAGE_ID;
            continue;
        }
        if (n < 0 || n > a.page_size) {
            bits |= RL_STATUS_LENGTHS;
            n = min(max(n, 0), a.page_size);
        }
        char* base = static_cast<char*>(lt & 1u ? a.v_cache : a.k_cache) + (lt >> 1) * p.layer_bytes;
        const Unit* from = reinterpret_cast<const Unit*>(base + (static_cast<long long>(src) * a.Hkv + h) * head_bytes);
        Unit* to = reinterpret_cast<Unit*>(base + (static_cast<long long>(dst) * a.Hkv + h) * head_bytes);
        const long long count = static_cast<long long>(n) * p.token_bytes / static_cast<long long>(sizeof(Unit));
        constexpr int kDeep = 8;
        long long x = lane;
        for (; x + (kDeep - 1) * 32 < count; x += kDeep * 32) {
            Unit v[kDeep];
#pragma unroll
            for (int k = 0; k < kDeep; ++k) v[k] = from[x + k * 32];
#pragma unroll
            for (int k = 0; k < kDeep; ++k) to[x + k * 32] = v[k];
        }
        for (; x < count; x += 32) to[x] = from[x];
    }
    set_status(p.status, bits);
}

int page_copy_impl(const rl_page_copy_args* a, int32_t* status, cudaStream_t stream) {
    CopyArgs p;
    p.a = *a;
    p.status = status;
    const int e = a->dtype == RL_DTYPE_F32 ? 4 : 2;
    p.token_bytes = a->D * e;
    p.layer_bytes = a->layers > 1 ? a->layer_stride * e : 0;
    p.units = a->n * a->layers * 2 * a->Hkv;
    if (p.units == 0) return RL_OK;
    const bool vec = p.token_bytes % 16 == 0 && p.layer_bytes % 16 == 0;
    ProfScope prof(RL_PROF_OTHER, stream);
    if (vec) page_copy_kernel<uint4><<<mark_blocks(p.units), kMoveThreads, 0, stream>>>(p);
    else page_copy_kernel<uint16_t><<<mark_blocks(p.units), kMoveThreads, 0, stream>>>(p);
    count_launch();
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

}  // namespace rl
