// Attention of a decode step over a paged cache: the group's shared prefix, read once for all
// of the group's queries, and each request's own keys.
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j
//
// The keys of a row are cut into parts (stretches of the prefix, stretches of the own keys);
// each part gives (m, l, o) = (max s, sum e^(s - m), sum e^(s - m) v), and the parts of a row are
// joined by their maxima:  o = sum_p e^(m_p - m) o_p / sum_p e^(m_p - m) l_p.
//
//  1. warp_attn_kernel  a part by one block on mma.sync tiles of 16 query rows (the heads that share a
//                       key head, times the step's tokens): four warps, each with 16 of a stage's 64
//                       keys and statistics of its own, joined at the end.  Keys and values come by
//                       TMA, page by page, into a ring of stages; a fifth warp issues the copies.
//                       (Blocks that stay and take part after part, the copies running ahead, were
//                       slower: 113 us against 88 for 64 requests of up to 4096 keys, since the
//                       parts are ragged and the join's memory leaves room for a stage less.)
//  2. tile_attn_kernel  a part with more rows, on the 5th-generation tensor cores
//                       (prefix_attn_tc.cuh).
//  3. join_kernel       one warp a row.
//
// Measured (one GB300, device time): 64 requests of up to 4096 own keys, 32 / 8 heads of 128, bf16
// (0.54 GB of keys and values): 88 us in warp_attn_kernel, 6.1 TB/s, 91 % of a plain copy.  Their
// shared prefix of 32,768 keys: 35 us in tile_attn_kernel, 980 TFLOP/s.  A decode step of 128
// requests in 16 groups (0.1 GB): 32.5 us, where the chain of one part (lengths, page, keys, join: 6 us)
// and the join count as much as the bytes.  Four requests of a 130-key prompt: 7.5 us.
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "gemm_tc.cuh"
#include "internal.h"

namespace rl {

constexpr int kStageKeys = 64;

struct AttnArgs {
    rl_prefix_attn_args a;
    int32_t* status;
    uint64_t wait_ns;
    int gq;               // query heads of a key head
    float c;              // scale * log2(e)
    int sp, so;           // parts of the prefix, of the own keys
    int chunk_p, chunk_o; // keys of a part, multiples of kStageKeys
    int tiles_p, tiles_o; // row tiles: of all groups together, of one request
    int run_p, run_o;     // whether the launch does the prefixes' parts, the own keys' parts
    int both;             // the own keys' blocks do their group's prefix first (sp = 0, so = 1)
    float* ml;            // [sp + so][T * Hq][2]: max (in log2 units), sum
    float* po;            // [sp + so][T * Hq][D] numerators
};

// One part's rows and keys.
struct Item {
    const int32_t* table;  // page ids
    int t0, rows;          // first token, query rows (token-major, then head)
    int m0;                // first row of the tile
    int len;               // keys that the last row sees
    int lim0;              // keys that a row of token t0 sees (each further token one more); prefix: INT_MAX step 0
    int step;
    int k0, k1;            // the part's keys
    int h, part;
    int r;                 // request (parts of own keys)
};

// tokens [first, last) of a request, clamped to the call's
RL_DEVINL int clamp_t(int x, long long T) { return static_cast<int>(min(max(static_cast<long long>(x), 0ll), T)); }

// The keys of group g's prefix from k0 on, at most `chunk` of them.
RL_DEVINL void prefix_keys(const AttnArgs& p, long long g, int k0, int chunk, Item& it, int& bits) {
    const rl_prefix_attn_args& a = p.a;
    int len = a.prefix_lens[g];
    const long long most = min(static_cast<long long>(a.max_prefix), static_cast<long long>(a.prefix_width * a.page_size));
    if (len < 0 || len > most) {
        bits |= RL_STATUS_LENGTHS;
        len = static_cast<int>(min(max(static_cast<long long>(len), 0ll), most));
    }
    it.table = a.prefix_table + g * a.prefix_width;
    it.len = len;
    it.lim0 = len;
    it.step = 0;
    it.k0 = k0;
    it.k1 = static_cast<int>(min(static_cast<long long>(k0) + chunk, static_cast<long long>(len)));
}
// Whether group g's requests are not a stretch of the call's, or not after those of the group before.
RL_DEVINL bool bad_group(const rl_prefix_attn_args& a, long long g) {
    const int ra = a.group_offsets[g], rb = a.group_offsets[g + 1];
    return ra < 0 || rb < ra || rb > a.R;
}
// The whole prefix of the group of `it`'s request (none: no keys).  All lanes of a warp together.
RL_DEVINL void find_prefix(const AttnArgs& p, const Item& it, Item& pre, int& bits) {
    const rl_prefix_attn_args& a = p.a;
    const int lane = threadIdx.x & 31;
    pre.k0 = pre.k1 = 0;
    for (long long g0 = 0; g0 < a.G; g0 += 32) {
        const long long g = g0 + lane;
        if (g < a.G && bad_group(a, g)) bits |= RL_STATUS_LENGTHS;
        const bool mine = g < a.G && a.group_offsets[g] <= it.r && it.r < a.group_offsets[g + 1];
        const unsigned hit = __ballot_sync(0xffffffffu, mine);
        if (hit) {
            prefix_keys(p, g0 + __ffs(hit) - 1, 0, INT_MAX, pre, bits);
            return;
        }
    }
}

// Which part block `id` does; false: none.  All lanes of one warp call it together.
RL_DEVINL bool find_item(const AttnArgs& p, long long id, int tile_rows, Item& it, int& bits) {
    const rl_prefix_attn_args& a = p.a;
    const int lane = threadIdx.x & 31;
    const long long prefix_items = p.run_p ? static_cast<long long>(p.sp) * a.Hkv * p.tiles_p : 0;
    if (id < prefix_items) {
        const int split = static_cast<int>(id % p.sp);
        it.h = static_cast<int>(id / p.sp % a.Hkv);
        long long tile = id / p.sp / a.Hkv;
        it.part = split;
        for (long long g0 = 0; g0 < a.G; g0 += 32) {
            const long long g = g0 + lane;
            int ta = 0, tb = 0;
            if (g < a.G) {
                const int ra = min(max(a.group_offsets[g], 0), static_cast<int>(a.R));
                const int rb = min(max(a.group_offsets[g + 1], ra), static_cast<int>(a.R));
                ta = clamp_t(a.cu_q[ra], a.T);
                tb = max(clamp_t(a.cu_q[rb], a.T), ta);
            }
            const long long rows = static_cast<long long>(tb - ta) * p.gq;
            const int tiles = static_cast<int>((rows + tile_rows - 1) / tile_rows);
            int incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, tile < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                const int mine = static_cast<int>(tile) - (incl - tiles);
                it.t0 = __shfl_sync(0xffffffffu, ta, src);
                it.rows = static_cast<int>(__shfl_sync(0xffffffffu, rows, src));
                it.m0 = __shfl_sync(0xffffffffu, mine, src) * tile_rows;
                prefix_keys(p, g0 + src, split * p.chunk_p, p.chunk_p, it, bits);
                return true;
            }
            tile -= __shfl_sync(0xffffffffu, incl, 31);
        }
        return false;
    }
    id -= prefix_items;
    const int split = static_cast<int>(id % p.so);
    it.h = static_cast<int>(id / p.so % a.Hkv);
    const long long rt = id / p.so / a.Hkv;
    const long long r = rt / p.tiles_o;
    const int tile = static_cast<int>(rt % p.tiles_o);
    it.part = p.sp + split;
    it.r = static_cast<int>(r);
    const int ca = a.cu_q[r], cb = a.cu_q[r + 1];
    const int ta = clamp_t(ca, a.T), tb = max(clamp_t(cb, a.T), ta);
    int n = tb - ta, kv = a.kv_lens[r];
    const long long most = min(static_cast<long long>(a.max_kv), static_cast<long long>(a.table_width * a.page_size));
    if (ca < 0 || cb < ca || cb > a.T || n > a.max_q || kv < n || kv > most || (r == 0 && ca != 0)) bits |= RL_STATUS_LENGTHS;
    n = static_cast<int>(min(static_cast<long long>(n), static_cast<long long>(a.max_q)));
    kv = static_cast<int>(min(max(static_cast<long long>(kv), 0ll), most));
    it.t0 = ta;
    it.rows = n * p.gq;
    it.m0 = tile * tile_rows;
    if (it.m0 >= it.rows) return false;
    it.table = a.block_table + r * a.table_width;
    it.lim0 = kv - n + 1;
    it.step = 1;
    const int last = (min(it.m0 + tile_rows, it.rows) - 1) / p.gq;   // last token of the tile
    it.len = min(kv, it.lim0 + last);
    it.k0 = split * p.chunk_o;
    it.k1 = static_cast<int>(min(static_cast<long long>(it.k0) + p.chunk_o, static_cast<long long>(it.len)));
    return true;
}

// Page of key k, or 0 with a status bit where the table holds none.
RL_DEVINL int page_of(const AttnArgs& p, const int32_t* table, int k, int shift, int& bits) {
    int page = table[k >> shift];
    if (page < 0 || page >= p.a.n_pages) {
        bits |= RL_STATUS_PAGE_ID;
        page = 0;
    }
    return page;
}

// Rows past the last request, where no join follows that writes them.
template <typename T, int D>
RL_DEVINL void clear_padding(const AttnArgs& p, int threads) {
    const rl_prefix_attn_args& a = p.a;
    const int tr = a.R > 0 ? clamp_t(a.cu_q[a.R], a.T) : 0;
    for (long long t = tr + static_cast<long long>(blockIdx.x); t < a.T; t += gridDim.x) {
        for (int x = threadIdx.x; x < a.Hq * D / 8; x += threads)
            reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.Hq * D)[x] = make_uint4(0, 0, 0, 0);
        if (a.lse)
            for (int x = threadIdx.x; x < a.Hq; x += threads) a.lse[t * a.Hq + x] = -INFINITY;
    }
}

template <typename T>
struct Mma;
template <>
struct Mma<__nv_bfloat16> {
    static RL_DEVINL void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static RL_DEVINL uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static RL_DEVINL __nv_bfloat16 one(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Mma<__half> {
    static RL_DEVINL void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static RL_DEVINL uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static RL_DEVINL __half one(float x) { return __float2half_rn(x); }
};
RL_DEVINL void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
RL_DEVINL void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// ---- 1. parts of 16 query rows -----------------------------------------------------------
constexpr int kWarpRows = 16;
constexpr int kWarpThreads = 160;          // four warps that compute, one that copies
constexpr int kWarpStages = 3;

template <int D>
constexpr int warp_stage_bytes() { return 2 * kStageKeys * D * 2; }
template <int D>
constexpr int warp_smem_bytes() { return kWarpStages * warp_stage_bytes<D>() + 1024 + 256; }
// The kernels of a call are programmatic launches.  The next one is let in when a block has its sums:
// let in at the start, its waiting blocks held registers that this one's blocks needed (139 us instead of
// 133 for 64 requests of up to 4096 keys).

template <typename T, int D>
__global__ void __launch_bounds__(kWarpThreads)
    warp_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int kStage = warp_stage_bytes<D>();
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kWarpStages * kStage);
    uint64_t* empty = full + kWarpStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kWarpStages);
    const rl_prefix_attn_args& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kWarpStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    Item it;
    int bits = 0;
    if (p.sp + p.so == 1) clear_padding<T, D>(p, kWarpThreads);
    const bool any = find_item(p, blockIdx.x, kWarpRows, it, bits);   // every warp for itself
    __syncthreads();
    if (!any) {
        if (threadIdx.x == 0) set_status(p.status, bits);
        wait_for_previous();
        return;
    }
    const int nst = it.k1 > it.k0 ? (it.k1 - it.k0 + kStageKeys - 1) / kStageKeys : 0;
    const int shift = 31 - __clz(a.page_size);
    const int g = lane >> 2, tq = lane & 3;

    if (warp == 4) {
        // ---------------- copies ----------------
        const int box = min(a.page_size, kStageKeys);               // keys of one copy
        const int per = kStageKeys / box;                           // copies of a stage and half-row
        bool ok = true;
        int issued = 0;
        for (int s = 0; s < nst; ++s) {
            const int st = s % kWarpStages;
            const uint32_t phase = (s / kWarpStages) & 1;
            // lanes below `per` look their page up; only pages with keys of the part are read
            const int key = it.k0 + s * kStageKeys + lane * box;
            const bool has = lane < per && key < it.k1;
            int row = 0;
            if (has) row = (page_of(p, it.table, key, shift, bits) * a.Hkv + it.h) * a.page_size + (key & (a.page_size - 1));
            const int n = __popc(__ballot_sync(0xffffffffu, has));
            ok = mbar_wait(empty + st, phase ^ 1u, p.status, p.wait_ns) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *abort_flag = 1;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(full + st, static_cast<uint32_t>(n) * box * D * 4);
            __syncwarp();
            if (has) {
                uint8_t* k = smem + st * kStage + lane * box * 128;
                uint8_t* v = k + kStageKeys * D * 2;
#pragma unroll
                for (int x = 0; x < D / 64; ++x) {
                    tma_load_2d(&tmK, full + st, k + x * kStageKeys * 128, x * 64, row);
                    tma_load_2d(&tmV, full + st, v + x * kStageKeys * 128, x * 64, row);
                }
            }
            issued = s + 1;
        }
        set_status(p.status, bits);
        __syncthreads();
        if (*abort_flag && lane == 0) {
            // every copy issued lands before the block can end
            for (int s = max(0, issued - kWarpStages); s < issued; ++s)
                mbar_wait(full + s % kWarpStages, (s / kWarpStages) & 1, p.status);
        }
        __syncthreads();
        wait_for_previous();
        return;
    }

    // ---------------- four warps of 16 keys each ----------------
    uint32_t q[D / 16][4];
    {
        const T* base = static_cast<const T*>(a.q);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int m = it.m0 + g + 8 * half;
            const bool in = m < it.rows;
            const int mm = in ? m : it.m0;
            const T* row = base + (it.t0 + mm / p.gq) * a.q_stride_t + static_cast<int64_t>(it.h * p.gq + mm % p.gq) * a.q_stride_h;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[k][half] = *reinterpret_cast<const uint32_t*>(row + k * 16 + tq * 2);
                q[k][half + 2] = *reinterpret_cast<const uint32_t*>(row + k * 16 + tq * 2 + 8);
            }
        }
    }
    // keys that this lane's two rows see
    const int lim[2] = {min(it.len, it.lim0 + it.step * ((it.m0 + g) / p.gq)), min(it.len, it.lim0 + it.step * ((it.m0 + g + 8) / p.gq))};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

    bool ok = true;
    for (int s = 0; s < nst; ++s) {
        const int st = s % kWarpStages;
        ok = mbar_wait(full + st, (s / kWarpStages) & 1, p.status, p.wait_ns) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
            *abort_flag = 1;
            break;
        }
        uint8_t* kt = smem + st * kStage;
        uint8_t* vt = kt + kStageKeys * D * 2;
        const int w0 = warp * 16;                                    // this warp's keys of the stage
        const int key0 = it.k0 + s * kStageKeys + w0;
        const int left = it.k1 - key0;                               // of which so many are the part's
        if (left < 16) {
            // values past the last key: whatever the page holds must not reach the sum
            for (int r = max(left, 0) + (lane >> 3); r < 16; r += 4)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    *reinterpret_cast<uint4*>(vt + x * kStageKeys * 128 + (w0 + r) * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        if (left > 0) {
            float sc[2][4] = {};
            const int kr = w0 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
            const uint32_t kbase = smem_addr(kt) + kr * 128;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                const int chunk = (k & 3) * 2 + kc;
                ldsm4(kbase + (k >> 2) * kStageKeys * 128 + ((chunk ^ (kr & 7)) << 4), b);
                Mma<T>::run(sc[0], q[k], b[0], b[1]);
                Mma<T>::run(sc[1], q[k], b[2], b[3]);
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = key0 + n * 8 + tq * 2 + (j & 1);
                    const bool seen = key < lim[j >> 1] && key < it.k1;
                    sc[n][j] = seen ? sc[n][j] * p.c : -INFINITY;
                    mx[j >> 1] = fmaxf(mx[j >> 1], sc[n][j]);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mn = fmaxf(m[h], mx[h]);
                    f[h] = m[h] == -INFINITY ? 0.f : exp2_approx(m[h] - mn);
                    m[h] = mn;
                    l[h] *= f[h];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= f[0];
                    o[i][1] *= f[0];
                    o[i][2] *= f[1];
                    o[i][3] *= f[1];
                }
            }
            const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sc[n][j] = exp2_approx(sc[n][j] - mu[j >> 1]);
                    l[j >> 1] += sc[n][j];
                }
            const uint32_t pa[4] = {Mma<T>::pack(sc[0][0], sc[0][1]), Mma<T>::pack(sc[0][2], sc[0][3]),
                                    Mma<T>::pack(sc[1][0], sc[1][1]), Mma<T>::pack(sc[1][2], sc[1][3])};
            const int vr = w0 + (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
            const uint32_t vbase = smem_addr(vt) + vr * 128;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t b[4];
                const int chunk = (i & 3) * 2 + vc;
                ldsm4_t(vbase + (i >> 2) * kStageKeys * 128 + ((chunk ^ (vr & 7)) << 4), b);
                Mma<T>::run(o[2 * i], pa, b[0], b[1]);
                Mma<T>::run(o[2 * i + 1], pa, b[2], b[3]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + st);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();                       // every stage has been read: its memory is free
    let_next_start();
    const bool dead = *abort_flag != 0;
    // join the four warps: (m, l) of all, then the numerators on one scale
    float* sm = reinterpret_cast<float*>(smem);                  // [4][16][2]
    float* so = sm + 4 * kWarpRows * 2;                          // [4][16][D + 4]
    constexpr int kPad = D + 4;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (tq == 0 && !dead) {
            sm[(warp * kWarpRows + g + 8 * h) * 2] = m[h];
            sm[(warp * kWarpRows + g + 8 * h) * 2 + 1] = l[h];
        }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (!dead) *reinterpret_cast<float2*>(so + (warp * kWarpRows + g + 8 * h) * kPad + i * 8 + tq * 2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    __syncthreads();
    if (dead) {
        wait_for_previous();
        return;
    }
    const long long rows_all = a.T * a.Hq;
    const bool whole = p.sp + p.so == 1;
    constexpr int kLanes = D / 4;                                // lanes of a row
    for (int x = threadIdx.x; x < kWarpRows * kLanes; x += 128) {
        const int r = x / kLanes, d = (x % kLanes) * 4;
        const int mr = it.m0 + r;
        if (mr >= it.rows) continue;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sm[(w * kWarpRows + r) * 2]);
        float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float mw = sm[(w * kWarpRows + r) * 2], lw = sm[(w * kWarpRows + r) * 2 + 1];
            if (lw == 0.f) continue;                             // no key seen (NaN goes on)
            const float f = exp2_approx(mw - mm);
            ll += f * lw;
            const float4 v = *reinterpret_cast<const float4*>(so + (w * kWarpRows + r) * kPad + d);
            acc[0] += f * v.x;
            acc[1] += f * v.y;
            acc[2] += f * v.z;
            acc[3] += f * v.w;
        }
        const long long row = static_cast<long long>(it.t0 + mr / p.gq) * a.Hq + it.h * p.gq + mr % p.gq;
        if (whole) {
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + row * D + d) =
                make_uint2(Mma<T>::pack(acc[0] * inv, acc[1] * inv), Mma<T>::pack(acc[2] * inv, acc[3] * inv));
            if (d == 0 && a.lse) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
        } else {
            if (ll != 0.f) *reinterpret_cast<float4*>(p.po + (it.part * rows_all + row) * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (d == 0) *reinterpret_cast<float2*>(p.ml + (it.part * rows_all + row) * 2) = make_float2(mm, ll);
        }
    }
    wait_for_previous();
}

}  // namespace rl

#include "prefix_attn_tc.cuh"

namespace rl {

// ---- 3. the parts of a row joined -----------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnArgs p) {
    const rl_prefix_attn_args& a = p.a;
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && p.sp > 0)
        for (long long g = threadIdx.x; g < a.G; g += kJoinThreads)
            if (bad_group(a, g)) set_status(p.status, RL_STATUS_LENGTHS);
    wait_for_previous();
    const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const long long rows = a.T * a.Hq;
    if (row >= rows) return;
    const int t = static_cast<int>(row / a.Hq);
    // the parts that this token's blocks have written
    const bool own = a.R > 0 && t < a.cu_q[a.R];
    bool pre = own && p.sp > 0;
    if (pre) {
        const int ra = min(max(a.group_offsets[0], 0), static_cast<int>(a.R)), rb = min(max(a.group_offsets[a.G], 0), static_cast<int>(a.R));
        pre = t >= a.cu_q[ra] && t < a.cu_q[rb];
    }
    const int first = pre ? 0 : p.sp, last = own ? p.sp + p.so : first;
    // at most 64 parts of the prefix and 64 of the own keys: four a lane
    constexpr int kPer = 4;
    float2 ml[kPer];
    float mm = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int x = first + j * 32 + lane;
        ml[j] = x < last ? *reinterpret_cast<const float2*>(p.ml + (x * rows + row) * 2) : make_float2(-INFINITY, 0.f);
        mm = fmaxf(mm, ml[j].x);
    }
    mm = warp_max(mm);
    float ll = 0.f, f[kPer], acc[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        f[j] = ml[j].y == 0.f ? 0.f : exp2_approx(ml[j].x - mm);      // a sum of NaN makes the row NaN
        ll += f[j] * ml[j].y;
    }
    ll = warp_sum(ll);
    // the numerators, eight parts' loads in flight; a part without keys has written none
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int n = min(32, last - first - j * 32);
#pragma unroll 1
        for (int y0 = 0; y0 < n; y0 += 8) {
            float v[8][D / 32], w[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                w[y] = __shfl_sync(0xffffffffu, f[j], (y0 + y) & 31);
                if (y0 + y >= n) w[y] = 0.f;
                if (w[y] > 0.f) {
                    const float* o = p.po + (static_cast<long long>(first + j * 32 + y0 + y) * rows + row) * D + lane * (D / 32);
                    if constexpr (D == 128) {
                        const float4 q = *reinterpret_cast<const float4*>(o);
                        v[y][0] = q.x; v[y][1] = q.y; v[y][2] = q.z; v[y][3] = q.w;
                    } else {
                        const float2 q = *reinterpret_cast<const float2*>(o);
                        v[y][0] = q.x; v[y][1] = q.y;
                    }
                } else {
#pragma unroll
                    for (int d = 0; d < D / 32; ++d) v[y][d] = 0.f;
                }
            }
#pragma unroll
            for (int y = 0; y < 8; ++y)
#pragma unroll
                for (int d = 0; d < D / 32; ++d) acc[d] = fmaf(w[y], v[y][d], acc[d]);
        }
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    T* out = static_cast<T*>(a.out) + row * D + lane * (D / 32);
#pragma unroll
    for (int j = 0; j < D / 32; j += 2) *reinterpret_cast<uint32_t*>(out + j) = Mma<T>::pack(acc[j] * inv, acc[j + 1] * inv);
    if (lane == 0 && a.lse) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// A bound of 0 on the prefixes' lengths takes their parts out of the call: a length that says otherwise is an
// error.  One block, in such calls alone (the check in the other kernels cost 1 % of a ragged extension).
__global__ void __launch_bounds__(kJoinThreads) no_prefix_kernel(const AttnArgs p) {
    for (long long g = threadIdx.x; g < p.a.G; g += kJoinThreads)
        if (p.a.prefix_lens[g] != 0) set_status(p.status, RL_STATUS_LENGTHS);
}

// ---- host ------------------------------------------------------------------------------
// Which kernel does the parts with so many query rows: mma.sync tiles of 16 (kWarp), one tensor-core
// tile of 128 rows that takes two key tiles at a time (kKeys: bound by reading the keys), or two
// tiles of rows (kRows: bound by the products and exponentials).
enum AttnKind { kWarp = 0, kKeys = 1, kRows = 2 };
// Up to two tiles of 16 rows read the keys twice, the second time from L2.
static AttnKind kind_of(int64_t rows) { return rows <= 2 * kWarpRows ? kWarp : rows <= kTileRows ? kKeys : kRows; }
static int rows_of(AttnKind k) { return k == kWarp ? kWarpRows : k == kKeys ? kTileRows : 2 * kTileRows; }

// How the keys are cut into parts: as many as let the blocks of all row tiles fill the device (kWarp
// and kKeys twice over; kRows once, since each part of its rows costs a numerator to write and read
// again), none shorter than 256 keys; kWarp's none longer than 1024, so that ragged requests
// even out.
static int parts_of(AttnKind kind, int64_t keys, int64_t items, int* chunk) {
    const int64_t target = (kind == kRows ? 1ll : 2ll) * num_sms();
    const int64_t unit = kind == kWarp ? kStageKeys : kTileKeys;
    int64_t n = items > 0 ? (kind == kWarp ? (target + items - 1) / items : target / items) : 1;
    if (kind == kWarp && n < (keys + 1023) / 1024) n = (keys + 1023) / 1024;
    const int64_t most = (keys + 255) / 256;
    if (n > most) n = most;
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    int64_t c = (keys + n - 1) / n;
    c = (c + unit - 1) / unit * unit;
    if (c < unit) c = unit;
    *chunk = static_cast<int>(c);
    return static_cast<int>(keys > 0 ? (keys + c - 1) / c : 1);
}

static AttnArgs attn_view(const rl_prefix_attn_args* a, void* ws, size_t* bytes, AttnKind* kp, AttnKind* ko) {
    AttnArgs p{};
    p.a = *a;
    p.gq = a->Hq / a->Hkv;
    // A scale of 0 makes all weights alike.  Unseen keys are scores of -inf, and the tensor-core kernel scales
    // after it masks: the least normal number in place of 0 keeps them out (-inf * 0 is NaN), and times
    // any score below 2^100 it is less than half a step of a weight.
    p.c = fmaxf(a->scale * kLog2e, FLT_MIN);
    const bool prefix = a->G > 0 && a->max_prefix > 0;
    *kp = kind_of(prefix ? (a->T * p.gq + a->G - 1) / a->G : 0);
    *ko = kind_of(a->max_q * p.gq);
    const int rp = rows_of(*kp), ro = rows_of(*ko);
    p.tiles_p = prefix ? static_cast<int>(a->T * p.gq / rp + a->G) : 0;      // a bound: each group rounds up once
    p.tiles_o = static_cast<int>((a->max_q * p.gq + ro - 1) / ro);
    const int64_t about = a->T * p.gq / rp > a->G ? a->T * p.gq / rp : a->G; // row tiles to expect
    // Requests that bring a tile of rows or more each, and enough of them to fill the device: one block
    // takes a tile of a request over the prefix and the own keys, and nothing is left to join.
    // (32 requests of 0 to 256 tokens, 8 heads a key head, on up to 4096 shared keys: 96 us so,
    // 123 us in two parts and a join.)
    p.both = prefix && *ko == kRows && a->R > 0 && a->T * p.gq / a->R >= 2 * kTileRows && a->T * p.gq / ro * a->Hkv >= num_sms() / 2;
    p.sp = prefix && !p.both ? parts_of(*kp, a->max_prefix, about * a->Hkv, &p.chunk_p) : 0;
    p.so = p.both ? 1 : parts_of(*ko, a->max_kv, a->R * p.tiles_o * a->Hkv, &p.chunk_o);
    if (p.both) p.chunk_o = INT_MAX;
    Carve cv(ws);
    const size_t rows = static_cast<size_t>(a->T) * a->Hq;
    const int parts = p.sp + p.so;
    if (parts > 1) {
        p.ml = cv.take<float>(rows * parts * 2);
        p.po = cv.take<float>(rows * parts * a->D);
    }
    if (bytes) *bytes = align_up(cv.off, 256);
    return p;
}

size_t prefix_attn_ws_bytes(const rl_prefix_attn_args* a) {
    size_t b = 0;
    AttnKind kp, ko;
    attn_view(a, nullptr, &b, &kp, &ko);
    return b;
}

template <typename T, int D>
static int launch_parts(AttnArgs p, AttnKind kind, bool prefix, bool own, bool follows, cudaStream_t stream, int* launches) {
    const rl_prefix_attn_args& a = p.a;
    p.run_p = prefix;
    p.run_o = own;
    const int64_t items = (prefix ? static_cast<int64_t>(p.sp) * a.Hkv * p.tiles_p : 0) +
                          (own ? static_cast<int64_t>(p.so) * a.Hkv * a.R * p.tiles_o : 0);
    if (items == 0) return RL_OK;
    if (items >= INT_MAX) {
        set_last_error("too many parts for one launch");
        return RL_ERR_UNSUPPORTED;
    }
    CUtensorMap tmK, tmV;
    const int64_t rows = a.n_pages * a.Hkv * a.page_size;
    const int most = kind == kWarp ? kStageKeys : kTileKeys;
    const int box = a.page_size < most ? a.page_size : most;
    const CUtensorMapDataType dt = a.dtype == RL_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    int rc = make_tmap_2d(&tmK, a.k_cache, dt, 2, rows, D, D, 64, box, 128);
    if (rc == RL_OK) rc = make_tmap_2d(&tmV, a.v_cache, dt, 2, rows, D, D, 64, box, 128);
    if (rc != RL_OK) return rc;
    const bool poll = kind != kWarp && p.wait_ns <= kPollBelowNs;
    const auto kernel = kind == kWarp   ? warp_attn_kernel<T, D>
                        : kind == kKeys ? (poll ? tile_attn_kernel<T, D, true, true> : tile_attn_kernel<T, D, true, false>)
                                        : (poll ? tile_attn_kernel<T, D, false, true> : tile_attn_kernel<T, D, false, false>);
    const int smem = kind == kWarp   ? warp_smem_bytes<D>()
                     : kind == kKeys ? TileShape<D, true>::kSmemBytes
                                     : TileShape<D, false>::kSmemBytes;
    static std::atomic<uint64_t> done[5];
    if (!allow_smem(kernel, smem, done[poll ? kind + 2 : kind])) return RL_ERR_CUDA;
    ++*launches;
    return launch_after(kernel, dim3(static_cast<unsigned>(items)), kind == kWarp ? kWarpThreads : kTileThreads, smem, follows, stream, tmK, tmV, p);
}

template <typename T, int D>
static int attn_run(const AttnArgs& p, AttnKind kp, AttnKind ko, cudaStream_t stream) {
    const rl_prefix_attn_args& a = p.a;
    ProfScope prof(RL_PROF_OTHER, stream);
    int launches = 0, rc;
    const bool no_prefix = a.G > 0 && a.max_prefix == 0;
    if (no_prefix) no_prefix_kernel<<<1, kJoinThreads, 0, stream>>>(p);
    if (p.sp > 0 && kp == ko) {
        rc = launch_parts<T, D>(p, kp, true, true, false, stream, &launches);
    } else {
        rc = p.sp > 0 ? launch_parts<T, D>(p, kp, true, false, false, stream, &launches) : RL_OK;
        if (rc == RL_OK) rc = launch_parts<T, D>(p, ko, false, true, launches > 0, stream, &launches);
    }
    if (rc != RL_OK) return rc;
    const int64_t rows_q = a.T * a.Hq;
    if (p.sp + p.so > 1 || launches == 0) {
        rc = launch_after(join_kernel<T, D>, dim3(static_cast<unsigned>((rows_q + kJoinThreads / 32 - 1) / (kJoinThreads / 32))), kJoinThreads, 0, launches > 0, stream, p);
        if (rc != RL_OK) return rc;
        ++launches;
    }
    count_launch(launches + (no_prefix ? 1 : 0));
    return cudaPeekAtLastError() == cudaSuccess ? RL_OK : RL_ERR_CUDA;
}

int prefix_attn_impl(const rl_prefix_attn_args* a, void* ws, int32_t* status, cudaStream_t stream) {
    if (a->T == 0) return RL_OK;
    AttnKind kp, ko;
    AttnArgs p = attn_view(a, ws, nullptr, &kp, &ko);
    p.status = status;
    p.wait_ns = wait_limit_ns();
    if (a->dtype == RL_DTYPE_BF16)
        return a->D == 128 ? attn_run<__nv_bfloat16, 128>(p, kp, ko, stream) : attn_run<__nv_bfloat16, 64>(p, kp, ko, stream);
    return a->D == 128 ? attn_run<__half, 128>(p, kp, ko, stream) : attn_run<__half, 64>(p, kp, ko, stream);
}

}  // namespace rl
