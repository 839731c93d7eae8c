// Attention parts on the 5th-generation tensor cores, for parts with more than 16 query rows.
//
// One block, 384 threads, 128 keys a step:
//   warp 0       copies K and V tiles, page by page, into a ring of shared-memory units (TMA);
//                pages past the last key are filled with zeros by a copy that starts past the cache
//   warp 1       issues the products:  S = Q K^T (both in shared memory), O += P V (P in TMEM, V in
//                shared memory, key-major).  The whole warp runs the loop and an elected lane issues, with
//                operands the compiler can see to be alike in all lanes: from one lane's branch
//                each instruction took about 100 cycles to issue, longer than it runs.
//   warps 4-7    softmax of accumulator 0, a thread a row: its 128 scores come from TMEM at once,
//   warps 8-11   of accumulator 1;  P goes back to TMEM over the scores
// TMEM: S0, S1 (128 columns each), O0, O1 (D columns each).  While one accumulator's scores are
// exponentiated the tensor core works on the other's products, and the values of
// a tile's first 64 keys are taken while the weights of the others are still being made.  The two
// accumulators are
//   kKeys2 = false   two tiles of 128 rows over the same keys (256 rows a block)
//   kKeys2 = true    the even and the odd key tiles of one tile of up to 128 rows, joined at the
//                    end through shared memory: for parts that are bound by reading the keys
// The running maximum is only followed when it grows by more than 2^8: until then the weights
// stay below 2^8 of it and O is left alone.  That O may be rescaled is known from the scores'
// barrier: the scores' product was issued after the last product into O.
//
// The keys of a block are a stretch of a prefix (all rows see all of it), a stretch of a request's own
// keys (causal), or one after the other: where every request of a step brings at least a tile of
// rows, its blocks run over the prefix and its own keys and write the result at once.
//
// Measured: 2850 to 3000 cycles for 256 rows by 128 keys, D = 128, where the products alone need 2048
// (a row's chain - scores 1100, maximum 290, exponentials 950, hand-over - does not quite hide behind
// the other accumulator's products); some 7000 cycles before a block's
// first scores and 4600 after its last.
// 32 requests of 0 to 256 tokens, 16 / 2 heads, up to 4096 shared and 1024 own keys: 95.5 us, 877 TFLOP/s
// of the visible keys' products.  One prompt, 32 / 8 heads of 128, bf16: 157 us for 4096 tokens (877 TFLOP/s of the
// causal products), 1520 for 16,384 (1447), 5665 for 32,768 (1553).
//
// Every wait is bounded; a wait that runs out raises the block's abort flag, all roles leave
// their loops, and copies and products in flight are waited for before TMEM is released.
#pragma once

#include "gemm_tc.cuh"
#include "internal.h"

namespace rl {

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kTileThreads = 384;

template <int D, bool kKeys2>
struct TileShape {
    static constexpr int kUnitBytes = kTileKeys * D * 2;
    static constexpr int kQTiles = kKeys2 ? 1 : 2;
    static constexpr int kQBytes = kQTiles * kTileRows * D * 2;
    static constexpr int kUnits = D == 128 ? (kKeys2 ? 5 : 4) : 8;
    // results pass through the memory of the ring and the queries: rows of two accumulators, (m, l)
    static constexpr int kRowBytes = (D + 4) * 4;         // padded: 16-byte steps of 32 rows on all banks
    static constexpr int kSmemBytes = kUnits * kUnitBytes + kQBytes + 1024 + 256;
    static_assert(kUnits * kUnitBytes + kQBytes >= 2 * kTileRows * kRowBytes + kTileRows * 8, "the results fit");
};

template <typename T>
constexpr uint32_t tile_idesc(uint32_t n, bool b_mn) {
    return (std::is_same<T, __nv_bfloat16>::value ? idesc_bf16_f32(kTileRows, n)
                                                  : ((1u << 4) | ((n >> 3) << 17) | ((kTileRows >> 4) << 24))) |
           (b_mn ? 1u << 16 : 0u);
}
// D[tmem] (+)= A[tmem] * B[smem]^T
RL_DEVINL void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
RL_DEVINL void tmem_st_32x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// One bulk copy shared -> global (16-byte aligned, size a multiple of 16), in the thread's bulk group.
RL_DEVINL void bulk_store(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes) : "memory");
}
RL_DEVINL bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
RL_DEVINL uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
RL_DEVINL void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bounded wait.  A sleeping try of the hardware outlasts a limit of some microseconds: such limits are kept by
// polling, in kernels of their own, since the polls beside the tries cost the others 2.5 to 5 % (94 us and 98.5 for
// the ragged extension below).
constexpr uint64_t kPollBelowNs = 10000;
template <bool kPoll>
RL_DEVINL bool wait_within(uint64_t* bar, uint32_t parity, const AttnArgs& p) {
    if constexpr (kPoll) {
        const long long t0 = clock64(), cycles = static_cast<long long>(2 * p.wait_ns);     // at 2.07 GHz at most
        while (true) {
            uint32_t ok;
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                "selp.u32 %0, 1, 0, p;\n\t}"
                : "=r"(ok)
                : "r"(smem_addr(bar)), "r"(parity)
                : "memory");
            if (ok) return true;
            if (clock64() - t0 > cycles) {
                set_status(p.status, RL_STATUS_TIMEOUT);
                return false;
            }
        }
    }
    return mbar_wait(bar, parity, p.status, p.wait_ns);
}

template <typename T, int D, bool kKeys2, bool kPoll>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_attn_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const AttnArgs p) {
    using Shape = TileShape<D, kKeys2>;
    constexpr int kUnits = Shape::kUnits, kUnit = Shape::kUnitBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* sq = smem + kUnits * kUnit;
    uint64_t* full = reinterpret_cast<uint64_t*>(sq + Shape::kQBytes);
    uint64_t* empty = full + kUnits;
    uint64_t* s_full = empty + kUnits;      // [2] scores of an accumulator are in TMEM
    uint64_t* p_half = s_full + 2;          // [2] its weights of the first 64 keys are
    uint64_t* p_ready = p_half + 2;         // [2] all of them are
    uint64_t* o_full = p_ready + 2;         // [2] its last product is done
    uint64_t* q_full = o_full + 2;          // the queries are in shared memory
    uint64_t* done_bar = q_full + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const rl_prefix_attn_args& a = p.a;
    const int warp = static_cast<int>(uniform(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    if (p.sp + p.so == 1) clear_padding<T, D>(p, kTileThreads);
    Item it;
    int bits = 0;
    constexpr int kItemRows = kKeys2 ? kTileRows : 2 * kTileRows;
    if (!find_item(p, blockIdx.x, kItemRows, it, bits)) {             // every warp for itself, all alike
        if (threadIdx.x == 0) set_status(p.status, bits);
        wait_for_previous();
        return;
    }
    const int rows = min(it.rows - it.m0, kItemRows);                 // of this block, at least 1
    // key tiles: `na` of the prefix stretch (it2 of a block that does both), then those of the own keys
    Item pre = it;
    if (p.both) find_prefix(p, it, pre, bits);
    else if (it.step) pre.k1 = pre.k0 = 0;
    if (!p.both && !it.step) it.k1 = it.k0 = 0;
    const int na = static_cast<int>(uniform(pre.k1 > pre.k0 ? (pre.k1 - pre.k0 + kTileKeys - 1) / kTileKeys : 0));
    const int nb = static_cast<int>(uniform(it.k1 > it.k0 ? (it.k1 - it.k0 + kTileKeys - 1) / kTileKeys : 0));
    const int n = na + nb;
    const bool two = kKeys2 ? n > 1 : rows > kTileRows;               // the second accumulator is in use

    if (threadIdx.x == 0) {
        for (int s = 0; s < kUnits; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full + t, 1);
            mbar_init(p_half + t, 4);
            mbar_init(p_ready + t, 4);
            mbar_init(o_full + t, 1);
        }
        mbar_init(q_full, 8);
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // queries: rows of 128 bytes with the 128-byte swizzle, 64 columns a sub-tile; zeros past the rows
    if (warp >= 4 && n > 0) {
        const int ch = (threadIdx.x - 128) % (D / 8), first = it.m0 / p.gq, rem = it.m0 % p.gq;
        const float inv = 1.f / static_cast<float>(p.gq);
        const T* base = static_cast<const T*>(a.q) + (it.t0 + first) * a.q_stride_t + static_cast<int64_t>(it.h * p.gq) * a.q_stride_h + ch * 8;
        for (int r = (threadIdx.x - 128) / (D / 8); r < Shape::kQTiles * kTileRows; r += 256 / (D / 8)) {
            const int x = rem + (r < rows ? r : 0);
            const int dt = static_cast<int>((static_cast<float>(x) + 0.5f) * inv);        // x / gq: x is small
            const T* src = base + dt * a.q_stride_t + (x - dt * p.gq) * a.q_stride_h;
            const int tile = r / kTileRows, rr = r % kTileRows;
            const uint32_t dst = smem_addr(sq) + tile * kTileRows * D * 2 + (ch >> 3) * kTileRows * 128 + rr * 128 +
                                 (((ch & 7) ^ (rr & 7)) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(r < rows ? 16 : 0) : "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    int issued_units = 0;                                             // warp 0: units of the ring filled so far

    if (warp == 0) {
        // ---------------- copies ----------------
        const int box = min(a.page_size, kTileKeys);
        const int per = kTileKeys / box;
        const int shift = 31 - __clz(a.page_size);
        const int past = static_cast<int>(a.n_pages * a.Hkv * a.page_size);     // a row past the cache: zeros
        int unit = 0;
        uint32_t phase = 0;
        bool ok = true;
        auto load = [&](const CUtensorMap* map, int tile) {
            const bool in_a = tile < na;
            const int key = (in_a ? pre.k0 + tile * kTileKeys : it.k0 + (tile - na) * kTileKeys) + lane * box;
            int row = past;
            if (lane < per && key < (in_a ? pre.k1 : it.k1))
                row = (page_of(p, in_a ? pre.table : it.table, key, shift, bits) * a.Hkv + it.h) * a.page_size + (key & (a.page_size - 1));
            ok = wait_within<kPoll>(empty + unit, phase ^ 1u, p) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *abort_flag = 1;
                return;
            }
            if (lane == 0) mbar_arrive_expect_tx(full + unit, kUnit);
            __syncwarp();
            if (lane < per)
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_2d(map, full + unit, smem + unit * kUnit + x * kTileKeys * 128 + lane * box * 128, x * 64, row);
            ++issued_units;
            if (++unit == kUnits) {
                unit = 0;
                phase ^= 1u;
            }
        };
        if (kKeys2) {
            for (int i = 0; i < 2 && i < n && ok; ++i) load(&tmK, i);
            for (int i = 0; i < n && ok; ++i) {
                load(&tmV, i);
                if (i + 2 < n && ok) load(&tmK, i + 2);
            }
        } else {
            for (int i = 0; i < n && ok; ++i) {
                load(&tmK, i);
                if (ok) load(&tmV, i);
            }
        }
        set_status(p.status, bits);
    } else if (warp == 1) {
        if (n > 0) {
            // ---------------- products ----------------
            constexpr uint32_t kIdescS = tile_idesc<T>(kTileKeys, false), kIdescO = tile_idesc<T>(D, true);
            int unit = 0;
            uint32_t phase = 0;
            bool issued = false;
            bool ok = wait_within<kPoll>(q_full, 0, p) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            auto wait_unit = [&]() {
                ok = ok && wait_within<kPoll>(full + unit, phase, p) && !*abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) umma_commit(bar);
                __syncwarp();
            };
            auto next_unit = [&]() {
                commit(empty + unit);
                if (++unit == kUnits) {
                    unit = 0;
                    phase ^= 1u;
                }
            };
            // descriptors of the ring's first unit and of the queries; a step within them adds its
            // distance in 16-byte steps (addresses stay below 2^18, so nothing carries out)
            const uint64_t dk = sdesc_kmajor_sw128(smem_addr(smem)), dq = sdesc_kmajor_sw128(smem_addr(sq));
            const uint64_t dv = sdesc_mnmajor_sw128(smem_addr(smem), kTileKeys * 128);
            auto scores = [&](int t) {
                const uint64_t k = dk + uniform(unit * (kUnit >> 4));
                const uint64_t q = dq + (kKeys2 ? 0u : uniform(t * ((kTileRows * D * 2) >> 4)));
                const uint32_t d = uniform(tmem + t * kTileKeys);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t off = ((x >> 2) * 128 * 128 + (x & 3) * 32) >> 4;
                        umma_bf16(d, q + off, k + off, kIdescS, x != 0);
                    }
                    umma_commit(s_full + t);
                }
                __syncwarp();
                issued = true;
            };
            // O += P V of step i of accumulator t, in two halves of the keys
            auto values = [&](int t, int i) {
                const uint64_t v = dv + uniform(unit * (kUnit >> 4));
                const uint32_t o = uniform(tmem + 2 * kTileKeys + t * D), w = uniform(tmem + t * kTileKeys);
                const uint32_t more = uniform(i != 0);
                if (elect_one()) {
#pragma unroll
                    for (int x = 0; x < kTileKeys / 32; ++x) umma_ts(o, w + x * 8, v + x * (2048 >> 4), kIdescO, x != 0 ? 1u : more);
                }
                __syncwarp();
                ok = ok && wait_within<kPoll>(p_ready + t, i & 1, p) && !*abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                if (ok && elect_one()) {
#pragma unroll
                    for (int x = kTileKeys / 32; x < kTileKeys / 16; ++x) umma_ts(o, w + x * 8, v + x * (2048 >> 4), kIdescO, 1u);
                }
                __syncwarp();
            };
            auto wait_p = [&](int t, int i) {
                ok = ok && wait_within<kPoll>(p_half + t, i & 1, p) && !*abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
            };
            if (kKeys2) {
                for (int i = 0; i < 2 && i < n; ++i) {
                    wait_unit();
                    if (!ok) break;
                    scores(i);
                    next_unit();
                }
                for (int i = 0; i < n && ok; ++i) {
                    const int t = i & 1;
                    wait_p(t, i >> 1);
                    wait_unit();
                    if (!ok) break;
                    values(t, i >> 1);
                    if (!ok) break;
                    next_unit();
                    if (i + 2 >= n) commit(o_full + t);
                    if (i + 2 < n) {
                        wait_unit();
                        if (!ok) break;
                        scores(t);
                        next_unit();
                    }
                }
            } else {
                wait_unit();
                if (ok) {
                    scores(0);
                    if (two) scores(1);
                    next_unit();
                }
                for (int i = 0; i < n && ok; ++i) {
                    // V of this step is the current unit, K of the next step the one after it
                    const int vu = unit;
                    const uint32_t vp = phase;
                    for (int t = 0; t < (two ? 2 : 1); ++t) {
                        wait_p(t, i);
                        unit = vu;
                        phase = vp;
                        if (t == 0) wait_unit();
                        if (!ok) break;
                        values(t, i);
                        if (!ok) break;
                        if (i + 1 == n) commit(o_full + t);
                        const bool last_t = t == 1 || !two;
                        if (last_t) commit(empty + unit);
                        if (++unit == kUnits) {
                            unit = 0;
                            phase ^= 1u;
                        }
                        if (i + 1 < n) {
                            if (t == 0) wait_unit();
                            if (!ok) break;
                            scores(t);
                            if (last_t) next_unit();
                        }
                    }
                }
            }
            if (!ok) *abort_flag = 1;
            if (issued) {           // every product is done before TMEM is released
                commit(done_bar);
                mbar_wait(done_bar, 0, p.status);
            }
        }
    } else if (warp >= 4) {
        if (n > 0) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        // ---------------- softmax ----------------
        const int t = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;                         // row of the tile
        const bool active = n > 0 && (t == 0 || two);
        const int m_row = it.m0 + (kKeys2 ? 0 : t * kTileRows) + r;
        const bool valid = m_row < it.rows && (kKeys2 || m_row - it.m0 < rows);
        const int lim_own = min(it.k1, it.lim0 + it.step * (m_row / p.gq));          // own keys below this are seen
        const uint32_t ts = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * kTileKeys;
        const uint32_t to = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 2 * kTileKeys + t * D;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        int steps = 0;
        if (active)
            for (int i = kKeys2 ? t : 0; i < n; i += kKeys2 ? 2 : 1, ++steps) {
                ok = wait_within<kPoll>(s_full + t, steps & 1, p) && !*abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int x = 0; x < 4; ++x) tmem_ld_32x32(ts + x * 32, s[x]);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    asm volatile("tcgen05.wait::ld.sync.aligned;"
                                 : "+r"(s[x][0]), "+r"(s[x][1]), "+r"(s[x][2]), "+r"(s[x][3]), "+r"(s[x][4]), "+r"(s[x][5]),
                                   "+r"(s[x][6]), "+r"(s[x][7]), "+r"(s[x][8]), "+r"(s[x][9]), "+r"(s[x][10]), "+r"(s[x][11]),
                                   "+r"(s[x][12]), "+r"(s[x][13]), "+r"(s[x][14]), "+r"(s[x][15]), "+r"(s[x][16]),
                                   "+r"(s[x][17]), "+r"(s[x][18]), "+r"(s[x][19]), "+r"(s[x][20]), "+r"(s[x][21]),
                                   "+r"(s[x][22]), "+r"(s[x][23]), "+r"(s[x][24]), "+r"(s[x][25]), "+r"(s[x][26]),
                                   "+r"(s[x][27]), "+r"(s[x][28]), "+r"(s[x][29]), "+r"(s[x][30]), "+r"(s[x][31])
                                 :
                                 : "memory");
                const bool in_a = i < na;
                const int key0 = in_a ? pre.k0 + i * kTileKeys : it.k0 + (i - na) * kTileKeys;
                const int last = in_a ? pre.k1 : it.k1, lim = in_a ? pre.k1 : lim_own;
                if (__any_sync(0xffffffffu, key0 + kTileKeys > lim)) {
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (key0 + x * 32 + j >= lim) s[x][j] = 0xff800000u;
                }
                float mx4[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) mx4[x] = __uint_as_float(s[x][0]);
#pragma unroll
                for (int j = 1; j < 32; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) mx4[x] = fmaxf(mx4[x], __uint_as_float(s[x][j]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                if ((kKeys2 || t == 0) && last < key0 + kTileKeys) {
                    // the last values' page may hold anything past the last key
                    const int u = !kKeys2 || i == n - 1 ? (n == 1 ? 1 : kKeys2 ? 2 * n - 1 : 2 * i + 1) : 2 * i + 2;  // place in the ring's order
                    ok = wait_within<kPoll>(full + u % kUnits, (u / kUnits) & 1, p) && !*abort_flag;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    uint8_t* v = smem + (u % kUnits) * kUnit;
                    const int first = last - key0;
                    for (int y = (warp & 3) * 32 + lane; y < (kTileKeys - first) * (D / 8); y += 128) {
                        const int key = first + y / (D / 8), ch = y % (D / 8);
                        *reinterpret_cast<uint4*>(v + (ch >> 3) * kTileKeys * 128 + key * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                // follow the maximum when it has grown past what the weights' type bears easily
                const float grown = (mx - m) * p.c;
                if (__any_sync(0xffffffffu, grown > 8.f || (m == -INFINITY && mx > -INFINITY))) {
                    const float mn = fmaxf(m, mx);
                    const float f = m == -INFINITY ? 0.f : exp2_approx((m - mn) * p.c);
                    m = mn;
                    l *= f;
                    if (steps > 0) {
#pragma unroll 1
                        for (int x = 0; x < D / 32; ++x) {
                            uint32_t o[32];
                            tmem_load_row32(to + x * 32, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_st_32x32(to + x * 32, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * p.c;
                float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t w[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float e0 = exp2_approx(fmaf(__uint_as_float(s[2 * x + (j >> 4)][(2 * j) & 31]), p.c, -mc));
                        const float e1 = exp2_approx(fmaf(__uint_as_float(s[2 * x + (j >> 4)][(2 * j + 1) & 31]), p.c, -mc));
                        l4[(j & 1) * 2] += e0;
                        l4[(j & 1) * 2 + 1] += e1;
                        w[j] = Mma<T>::pack(e0, e1);
                    }
                    tmem_st_32x32(ts + x * 32, w);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive((x == 0 ? p_half : p_ready) + t);
                }
                l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
            }
        if (n > 0 && ok) {                  // with all products done the ring and the queries are free
            ok = wait_within<kPoll>(o_full, 0, p) && (!two || wait_within<kPoll>(o_full + 1, 0, p)) && !*abort_flag;
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
        }
        if (!ok) *abort_flag = 1;
        let_next_start();
        // ---------------- results ----------------
        float* stage = reinterpret_cast<float*>(smem + t * kTileRows * Shape::kRowBytes + r * Shape::kRowBytes);   // this row's
        float2* jm = reinterpret_cast<float2*>(smem + 2 * kTileRows * Shape::kRowBytes);       // (m, l) of accumulator 1
        float f0 = 1.f, f1 = 0.f;
        if (kKeys2 && two) {
            if (t == 1) {
                jm[r] = make_float2(m, l);
                if (ok)
#pragma unroll 1
                    for (int x = 0; x < D / 32; ++x) {
                        uint32_t o[32];
                        tmem_load_row32(to + x * 32, o);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) *reinterpret_cast<uint4*>(stage + x * 32 + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (t == 0) {
                const float2 q = jm[r];
                const float mn = fmaxf(m, q.x);
                f0 = m == -INFINITY ? 0.f : exp2_approx((m - mn) * p.c);
                f1 = q.x == -INFINITY ? 0.f : exp2_approx((q.x - mn) * p.c);
                l = l * f0 + q.y * f1;
                m = mn;
            }
        }
        const bool writes = kKeys2 ? t == 0 : (t == 0 || rows > kTileRows);
        if (writes && !__any_sync(0xffffffffu, !ok || *abort_flag != 0)) {
            const long long rows_all = a.T * a.Hq;
            const long long row = static_cast<long long>(it.t0 + m_row / p.gq) * a.Hq + it.h * p.gq + m_row % p.gq;
            const bool whole = p.sp + p.so == 1;
            // a sum of 0 is a row that sees nothing; one of NaN stays NaN, in the result as in lse
            const float inv = l == 0.f ? 0.f : whole || l != l ? 1.f / l : 1.f;
            f0 *= inv;
            f1 *= inv;
            // a row through shared memory, so that it leaves in one piece
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
                float v[32];
                if (n > 0) {
                    uint32_t o[32];
                    tmem_load_row32(to + x * 32, o);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = f0 != 0.f ? __uint_as_float(o[j]) * f0 : 0.f;
                    if (kKeys2 && two && f1 != 0.f)
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 q = *reinterpret_cast<const float4*>(stage + kTileRows * (D + 4) + x * 32 + j);
                            v[j] = fmaf(q.x, f1, v[j]);
                            v[j + 1] = fmaf(q.y, f1, v[j + 1]);
                            v[j + 2] = fmaf(q.z, f1, v[j + 2]);
                            v[j + 3] = fmaf(q.w, f1, v[j + 3]);
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.f;
                }
                if (whole) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8)
                        *reinterpret_cast<uint4*>(reinterpret_cast<T*>(stage) + x * 32 + j) =
                            make_uint4(Mma<T>::pack(v[j], v[j + 1]), Mma<T>::pack(v[j + 2], v[j + 3]), Mma<T>::pack(v[j + 4], v[j + 5]),
                                       Mma<T>::pack(v[j + 6], v[j + 7]));
                } else {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) *reinterpret_cast<float4*>(stage + x * 32 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            }
            fence_proxy_async_smem();
            if (valid) {
                void* dst = whole ? static_cast<void*>(static_cast<T*>(a.out) + row * D) : static_cast<void*>(p.po + (it.part * rows_all + row) * D);
                if (whole || l != 0.f) bulk_store(dst, stage, whole ? D * 2 : D * 4);
                const float ml = m == -INFINITY ? m : m * p.c;        // in log2 units
                if (whole) {
                    if (a.lse) a.lse[row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * kLn2;
                } else {
                    *reinterpret_cast<float2*>(p.ml + (it.part * rows_all + row) * 2) = make_float2(ml, l);
                }
            }
            bulk_commit();
            bulk_wait_all();
        }
    }
    tc_fence_before();
    __syncthreads();
    // Whichever role gave up, copies may be under way still (the first kUnits wait for nothing): they land
    // before the block ends and its memory is another's.
    if (warp == 0 && lane == 0 && *abort_flag)
        for (int s = max(0, issued_units - kUnits); s < issued_units; ++s) mbar_wait(full + s % kUnits, (s / kUnits) & 1, p.status);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    wait_for_previous();
}

}  // namespace rl
