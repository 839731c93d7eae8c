// Weights e^x as unevaluated pairs of floats and their sums, for decisions that follow exact
// arithmetic to about 2^-36 of a row's total (sampling, verification):
//   w = 2^p, p = z log2(e) / T - ref with the factor as two floats;  p = n + j/2048 + r;
//   2^(j/2048) = hi (1 + rho) from a table, 2^r - 1 = r ln2 + (r ln2)^2 / 2 (the next term is
//   below 2^-40), so w = 2^n hi (1 + rho + ...) is the unevaluated pair (2^n hi, v).
#pragma once

#include <cfloat>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ff.cuh"

namespace rl {

constexpr float kLog2eHi = 1.44269502162933349609f, kLog2eLo = 1.92596299112661746887e-8f;
// |m c| up to which a sum of 2^(z c - fl(m c)) can be put right by 2^(fl(m c) - m c): half a last place is at most 1/2 there
// (past 2^31 both factors leave the range of floats, the one upwards and the other down).
constexpr float kFusedRef = 0x1p24f;

// Entry j: bits of the float nearest 2^(j/2048) less j << 12 (so that adding the phase's bits
// gives the scaled value), and the relative error of that float.  Made by the compiler, by the
// exponential series in double.
struct ExpTable {
    uint32_t bits[2048];
    float rho[2048];
};
constexpr double exp2_series(double x) {              // 0 <= x < 1
    const double y = x * 0.693147180559945309417;
    double t = 1.0, s = 1.0;
    for (int i = 1; i < 26; ++i) {
        t *= y / i;
        s += t;
    }
    return s;
}
constexpr ExpTable make_exp_table() {
    ExpTable t{};
    for (int j = 0; j < 2048; ++j) {
        const double v = exp2_series(j / 2048.0);
        const float h = static_cast<float>(v);        // in [1, 2): 1 + mantissa / 2^23
        const uint32_t mant = static_cast<uint32_t>((static_cast<double>(h) - 1.0) * 8388608.0);
        t.bits[j] = (0x3f800000u | mant) - (static_cast<uint32_t>(j) << 12);
        t.rho[j] = static_cast<float>((v - static_cast<double>(h)) / static_cast<double>(h));
    }
    return t;
}
static __device__ const ExpTable kExpTable = make_exp_table();

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

RL_DEVINL float max_nan(float a, float b) {           // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

RL_DEVINL void fill_table(float2* tab, int tid, int threads) {
    for (int j = tid; j < 2048; j += threads) tab[j] = make_float2(__uint_as_float(kExpTable.bits[j]), kExpTable.rho[j]);
}
// Weights of lower exponents count as 0.  As a bound of logits, M + kLeastExp / c, it is rounded to a float: where the logits' spacing is as
// large as the bound's distance, the last of them that passes has an exponent of -(62 + spacing c / 2), and no spacing c
// above 124 lets any pass.  So weights' exponents stay above -126, where the addition to a float's exponent is sound.
constexpr float kLeastExp = -62.f;
// 2^(x c - ref) as hi + v, for x c - ref in [-126, 1] and magic = 6144 - ref: the last place of
// 6144 + y is 2^-11, so the bits of t are 0x45C00000 + 2048 n + j for the nearest n + j/2048, and
// what is left of x c, r, comes from one more product.  (x + x_lo for an argument of two floats.)
RL_DEVINL void weight_pair(float x, float x_lo, FF c, float magic, const float2* tab, float& hi, float& v) {
    const float t = fmaf(x, c.hi, magic);
    float r = fmaf(x, c.hi, -__fsub_rn(t, magic));
    r = fmaf(x, c.lo, r);
    r = fmaf(x_lo, c.hi, r);
    const uint32_t tb = __float_as_uint(t);
    const float2 q = tab[tb & 2047u];
    hi = __uint_as_float(__float_as_uint(q.x) + (tb << 12));
    v = hi * fmaf(r, fmaf(r, 0.24022650695910072f, 0.69314718055994531f), q.y);
}
RL_DEVINL float power_of_2(int k) { return __int_as_float((127 + k) << 23); }
// Sum of up to four weights of at most 1 in a lane, hi + v each: in a float that starts at 24, so
// that it only takes whole steps of 2^-19, and the rest apart (below 2^-17).  Both become integers;
// a warp's total is (top << 31) + (low << 7) in units of 2^-50, a lane's part rounded to 2^-43.  The
// weights are relative to the largest of their chunk or part, so that the roundings of a long flat tail, which
// all go one way, are small beside the tail and not beside the row's largest weight alone.
struct LaneSum {
    float top = 24.f, low = 0.f;
    RL_DEVINL void add(float hi, float v) {
        const float n = __fadd_rn(top, __fadd_rn(hi, v));
        low += __fadd_rn(__fsub_rn(hi, __fsub_rn(n, top)), v);
        top = n;
    }
    RL_DEVINL uint32_t warp_top() const { return __reduce_add_sync(0xffffffffu, __float_as_uint(top) - 0x41c00000u); }
    RL_DEVINL int warp_low() const { return __reduce_add_sync(0xffffffffu, __float2int_rn(low * 0x1p43f)); }
    static RL_DEVINL unsigned long long total(uint32_t a, int b) {
        const long long w = (static_cast<long long>(a) << 31) + (static_cast<long long>(b) << 7);
        return w > 0 ? static_cast<unsigned long long>(w) : 0ull;
    }
};
// The weight of z relative to M in units of 2^-k; `zlow` = M + kLeastExp / c, at least
// -FLT_MAX: below it the weight is 0 (M itself where the difference is lost).
RL_DEVINL unsigned long long weight_fixed(float z, float M, FF c, float zlow, int k, const float2* tab) {
    if (!(z >= zlow)) return 0ull;
    float hi, v;
    const FF d = two_sum(z, -M);
    weight_pair(d.hi, d.lo, c, 6144.f, tab, hi, v);
    const float wh = __fadd_rn(hi, v), wl = __fsub_rn(v, __fsub_rn(wh, hi));
    if (!(wh < 2.f)) return 0ull;             // differences past the range of floats
    const uint32_t b = __float_as_uint(wh);
    const int sh = static_cast<int>(b >> 23) - 127 - 23 + k;           // the 24-bit significand times 2^sh
    const unsigned long long m = (b & 0x7fffffu) | 0x800000u;
    const unsigned long long w = sh >= 0 ? m << sh : (sh > -25 ? (m + (1ull << (-sh - 1))) >> -sh : 0ull);
    return w + static_cast<long long>(__float2int_rn(wl * power_of_2(k)));       // below 2^(k - 24)
}
// floor(f x) for 0 <= f < 1
RL_DEVINL unsigned long long fraction_of(float f, unsigned long long x) {
    const uint32_t b = __float_as_uint(f);
    const int e = static_cast<int>(b >> 23);             // f = m 2^(e - 150)
    const unsigned long long m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int sh = e - 150 + 64;                         // m 2^sh = f 2^64 (below 2^-64 it hardly matters)
    const unsigned long long q = sh >= 0 ? m << sh : sh > -64 ? m >> -sh : 0ull;
    return __umul64hi(q, x);
}

// e^x of a pair to about 2^-38, by the table in memory (constant memory serves a warp's different places one
// after another): a tenth of exp_ff's time where every lane has its own x.  Below -87 it is 0.
RL_DEVINL FF exp_table(FF x) {
    if (!(x.hi >= -87.f)) return {x.hi < -87.f ? 0.f : x.hi, 0.f};      // (NaN goes on)
    if (x.hi > 88.f) return {INFINITY, 0.f};
    const float ref = ceilf(x.hi * kLog2eHi), magic = 6144.f - ref;
    const float t = fmaf(x.hi, kLog2eHi, magic);
    float r = fmaf(x.hi, kLog2eHi, -__fsub_rn(t, magic));
    r = fmaf(x.hi, kLog2eLo, r);
    r = fmaf(x.lo, kLog2eHi, r);
    const uint32_t tb = __float_as_uint(t), j = tb & 2047u;
    const float hi = __uint_as_float(__ldg(&kExpTable.bits[j]) + (tb << 12));
    const FF e = fast_two_sum(hi, hi * fmaf(r, fmaf(r, 0.24022650695910072f, 0.69314718055994531f), __ldg(&kExpTable.rho[j])));
    const float k = power_of_2(static_cast<int>(ref));
    return {e.hi * k, e.lo * k};
}
// ln x of a positive pair, likewise: one Newton step from the float's.
RL_DEVINL FF ln_table(FF x) {
    const bool small = x.hi < 0x1p-64f;                  // (1 / x is to be a float, and subnormal ones hold fewer bits)
    if (small) x = {x.hi * 0x1p100f, x.lo * 0x1p100f};
    const float y = logf(x.hi);
    const FF r = ff_mul(x, exp_table({-y, 0.f}));        // 1 + d
    const float d = __fadd_rn(__fsub_rn(r.hi, 1.f), r.lo);
    FF l = fast_two_sum(y, fmaf(-0.5f * d, d, d));
    if (small) l = ff_add(l, {-69.31472015380859375f, 2.0978141e-06f});      // - 100 ln 2
    return l;
}

}  // namespace rl
