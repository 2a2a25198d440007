// Weights of a row's logits, w = exp((z - max) / T): one by one in whole units
// (weight), and added up in packed floats (WeightSum). Only roundings, products,
// sums and shifts, whose results are the same on the host: the tests compile this
// file there, with these few functions of the device beside it (f32x2 and ff of
// sv_device.cuh among them), and compare it with 64-bit and longer arithmetic.
#pragma once

namespace sv {

typedef unsigned long long u64;

constexpr int CL_EXP_BITS = 8;
constexpr int CL_EXP = 1 << CL_EXP_BITS;  // entries of the table of 2^(i / 256)
constexpr int CL_FRACTION = 44;           // bits behind the point of a weight's mantissa in [1, 2)
constexpr float CL_MAGIC = 12582912.0f;   // 1.5 * 2^23: adding it rounds to whole numbers

// 2^(i / 256) as the sum of two floats.
struct alignas(8) ExpEntry {
    float hi, lo;
};
constexpr int CL_COPIES = 4;  // of the table, side by side, for whole rows: lane l reads copy l % 4
struct ExpTable {
    ExpEntry e[CL_EXP];
};
constexpr double exp_series(double x) {
    double sum = 1.0, term = 1.0;
    for (int i = 1; i < 30; ++i) {
        term *= x / i;
        sum += term;
    }
    return sum;
}
constexpr ExpTable make_exp_table() {
    ExpTable t = {};
    for (int i = 0; i < CL_EXP; ++i) {
        const double v = exp_series(0.69314718055994530942 * i / CL_EXP);
        t.e[i].hi = (float)v;
        t.e[i].lo = (float)(v - (double)(float)v);
    }
    return t;
}
constexpr float CL_L1 = 2.7076061740622863e-3f;  // ln 2 / 256
constexpr float CL_L1_LOW = (float)(0.69314718055994530942 / 256.0 - (double)2.7076061740622863e-3f);  // what that drops
constexpr float CL_L2 = 3.6655655969053526e-6f;  // its square / 2
constexpr float CL_L3 = 3.3083027270131e-9f;     // its cube / 6

struct RowScale {
    float top;       // the row's maximum
    float ch, cl;    // 256 log2(e) / T in two floats
    float low;       // a logit of weight 2^-100; NaN where the row's maximum has no room for one
    float shift, frac, rest;  // for WeightSum, where there is room
    int unit;        // weights are whole numbers in units of 2^-unit
    float none;      // what an exponent has to lie above, 2 more than the unit's
};

// The finest unit in which weights of this sum (at least 1/2) stay below 2^63. Equal
// weights are all rounded the same way, so that the unit's half counts as often as
// there are tokens: V 2^-62 of the sum or less. (In units of 2^-44 throughout, as many
// as 262144 largest weights leave room for, 262143 logits 28 below the largest were
// off by 1.3 %, their sum by 2e-9 of the row's.)
__device__ __forceinline__ int unit_of(float sum) {
    const int e = (int)(__float_as_uint(sum) >> 23) - 127;
    return e < 0 ? 62 : 62 - e;
}
__device__ __forceinline__ float none_of(int unit) { return CL_MAGIC - (float)((unit + 2) * CL_EXP); }
__device__ __forceinline__ void set_unit(RowScale& s, int unit) {
    s.unit = unit;
    s.none = none_of(unit);
}

// What a row's maximum decides; low_by: how far below it a weight is 2^-100.
__device__ __forceinline__ void set_scale(RowScale& s, float top, float ch, float cl, float low_by) {
    // (rounded as WeightSum rounds it: from y, next to a half, the maximum's own
    // exponent came out as 1 / 256)
    const float y = __fmul_rn(top, ch), whole = __fsub_rn(__fmaf_rn(top, ch, CL_MAGIC), CL_MAGIC);
    s.top = top;
    s.ch = ch;
    s.cl = cl;
    s.low = fabsf(y) < 0x1p21f ? top - low_by : __uint_as_float(0x7fc00000u);
    s.shift = CL_MAGIC - whole;
    const float a = __fsub_rn(y, whole), low = __fmaf_rn(top, cl, __fmaf_rn(top, ch, -y)), frac = __fadd_rn(a, low);
    s.frac = frac;
    s.rest = -__fadd_rn(__fsub_rn(a, frac), low) * CL_L1;
}

// exp((z - top) / T) in units of 2^-unit, for the few elements that decide: those of a
// list, of a draw's last part, of a pass that is made again. With d = z - top in two
// floats, exactly, y = 256 d log2(e) / T = n + r + x, n whole, |r| <= 1/2 and x its
// rounding errors: 2^(n / 256) = hi + lo comes from the table and a shift, and with u
// = (r + x) ln 2 / 256 = uh + ul in two floats e^u - 1 = uh + el from its series, el
// with every term that uh and ul have in common. Right to 2^-40 of itself and half a
// unit; the maximum's is 2^unit exactly.
__device__ __forceinline__ u64 weight(float z, const RowScale& s, const ExpEntry* table, int unit, float none) {
    const float dh = __fsub_rn(z, s.top);
    const float bb = __fsub_rn(dh, z);
    const float dl = __fsub_rn(__fsub_rn(z, __fsub_rn(dh, bb)), __fadd_rn(s.top, bb));
    const float t = __fmaf_rn(dh, s.ch, CL_MAGIC);
    const float p = __fmul_rn(dh, s.ch), r = __fsub_rn(p, __fsub_rn(t, CL_MAGIC));
    const float x = __fmaf_rn(dl, s.ch, __fmaf_rn(dh, s.cl, __fmaf_rn(dh, s.ch, -p)));
    const float uh = __fmul_rn(r, CL_L1), ul = __fmaf_rn(x, CL_L1, __fmaf_rn(r, CL_L1_LOW, __fmaf_rn(r, CL_L1, -uh)));
    const float el = __fmaf_rn(__fmul_rn(uh, uh), __fmaf_rn(uh, __fmaf_rn(uh, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f),
                               __fmaf_rn(__fmaf_rn(ul, 0.5f, uh), ul, ul));
    const uint32_t tb = __float_as_uint(t);
    const ExpEntry en = table[tb & (CL_EXP - 1)];  // (the magic number's low bits are 0)
    const float second = __fmul_rn(en.hi, uh);
    const float third = __fadd_rn(__fmaf_rn(en.hi, el, __fmaf_rn(en.lo, uh, en.lo)), __fmaf_rn(en.hi, uh, -second));
    const u64 q = ((u64)((__float_as_uint(en.hi) & 0x7FFFFFu) | 0x800000u) << (CL_FRACTION - 23)) +
                  (u64)(__float2ll_rn(__fmul_rn(second, 0x1p44f)) + __float2int_rn(__fmul_rn(third, 0x1p44f)));
    const int k = (int)((0x4B400000u + CL_EXP - 1 - tb) >> CL_EXP_BITS);  // ceil(-n / 256)
    const int sh = k + CL_FRACTION - unit;                               // at most 46
    const u64 w = sh >= 0 ? (q + ((1ull << (sh & 63)) >> 1)) >> (sh & 63) : q << (-sh & 63);
    return t > none ? w : 0ull;  // (and where d is -inf)
}
__device__ __forceinline__ u64 weight(float z, const RowScale& s, const ExpEntry* table) { return weight(z, s, table, s.unit, s.none); }

// Adds up weights in floats, two elements at a time in packed instructions, for
// the passes over whole rows (shifting integers took twice as long). Here y = z c -
// top c, formed at once: r.shift is the magic number less the whole part of top c
// and r.frac the rest, so that t's low bits are n again. What r.frac's rounding
// dropped would move all weights alike, by 2^-34 of themselves; it is added to e,
// whose own rounding takes it up on average. The maximum's own weight is made 1
// exactly, which keeps ties exact. w = (hi + (lo + hi e)) 2^-k; the sum s of the first
// parts begins at 1, so that s >= any of them and a - (s' - s) is the rounding error of
// s' = s + a exactly. A piece's errors and second parts are added up and go to c,
// whose own errors go to d.
//
// What that leaves. A weight: |x| <= 1.2 is rounded three times (2^-26, 2^-25, 2^-24,
// times ln 2 / 256), its polynomial twice (2^-33 each), ln 2 / 256 once (2^-33.3),
// hi e + lo once (2^-32.3 of hi): CL_PAIR_ERROR of itself. A piece's sum: 4 additions
// at most that a second part (2^-8.2 of its weight) meets, 2^-24 each: CL_ADD_ERROR.
// First parts too small for s go to c whole, rounded like the others: 4 2^-24 of V
// weights of at most 2^-24 of what s is, 1 and the thread's own (sum_error). Over the
// thousands of weights of a usual row these cancel, to about 2^-37 of the sum; where a
// decision comes nearer than the bound it is made with weight() (cut_by_mass).
constexpr float CL_PAIR_ERROR = 0x1p-30f, CL_ADD_ERROR = 0x1.8p-31f;
struct WeightSum {
    f32x2 s, c, d, part;
    __device__ __forceinline__ WeightSum() : s(pack2(1.0f, 1.0f)), c(pack2(0.0f, 0.0f)), d(c), part(c) {}
    // The two parts of a pair's weights; z0, z1 >= r.low.
    static __device__ __forceinline__ void pair(float z0, float z1, const RowScale& r, const ExpEntry* table, f32x2& a, f32x2& rest) {
        const f32x2 z = pack2(z0, z1), minus = pack2(-1.0f, -1.0f), ch = pack2(r.ch, r.ch), shift = pack2(r.shift, r.shift);
        const f32x2 t = fma2(z, ch, shift);
        const f32x2 x = add2(fma2(z, ch, fma2(t, minus, shift)), fma2(z, pack2(r.cl, r.cl), pack2(-r.frac, -r.frac)));
        float t0, t1, e0, e1;
        unpack2(fma2(x, fma2(x, fma2(x, pack2(CL_L3, CL_L3), pack2(CL_L2, CL_L2)), pack2(CL_L1, CL_L1)), pack2(r.rest, r.rest)), e0, e1);
        unpack2(t, t0, t1);
        e0 = z0 == r.top ? 0.0f : e0;
        e1 = z1 == r.top ? 0.0f : e1;
        const uint32_t b0 = __float_as_uint(t0), b1 = __float_as_uint(t1);
        const ExpEntry p = table[(b0 & (CL_EXP - 1)) * CL_COPIES], q = table[(b1 & (CL_EXP - 1)) * CL_COPIES];
        // 2^floor(n / 256): the magic number's upper bits leave the word
        const auto scale = [](uint32_t b) { return __uint_as_float((b & ~(uint32_t)(CL_EXP - 1)) * (1u << (23 - CL_EXP_BITS)) + 0x3F800000u); };
        const float pow0 = scale(b0), pow1 = scale(b1);
        a = pack2(__fmul_rn(p.hi, pow0), __fmul_rn(q.hi, pow1));
        rest = pack2(__fmul_rn(__fmaf_rn(p.hi, e0, p.lo), pow0), __fmul_rn(__fmaf_rn(q.hi, e1, q.lo), pow1));
    }
    // One pair of a piece, whose last one is followed by end_piece().
    __device__ __forceinline__ void add(f32x2 a, f32x2 rest, bool first) {
        const f32x2 minus = pack2(-1.0f, -1.0f), sum = add2(s, a), q = add2(fma2(fma2(s, minus, sum), minus, a), rest);
        part = first ? q : add2(part, q);
        s = sum;
    }
    __device__ __forceinline__ void end_piece() {
        // (Knuth's two-sum: either may be the larger one)
        const f32x2 minus = pack2(-1.0f, -1.0f), sum = add2(c, part), of_part = fma2(c, minus, sum), of_c = fma2(of_part, minus, sum);
        d = add2(d, add2(fma2(of_c, minus, c), fma2(of_part, minus, part)));
        c = sum;
    }
    __device__ __forceinline__ void add(float z0, float z1, const RowScale& r, const ExpEntry* table, bool first) {
        f32x2 a, rest;
        pair(z0, z1, r, table, a, rest);
        add(a, rest, first);
    }
    __device__ __forceinline__ u64 total(int unit) const {
        float s0, s1, c0, c1, d0, d1;
        unpack2(s, s0, s1);
        unpack2(c, c0, c1);
        unpack2(d, d0, d1);
        // (differences from 1 are exact, and a double's units are few)
        const ff sum = two_sum(__fsub_rn(s0, 1.0f), __fsub_rn(s1, 1.0f)), more = two_sum(c0, c1);
        const float units = __uint_as_float((uint32_t)(127 + unit) << 23);
        const long long v = __float2ll_rn(sum.hi * units) + __float2ll_rn(more.hi * units) +
                            __float2ll_rn(__fadd_rn(__fadd_rn(sum.lo, more.lo), __fadd_rn(d0, d1)) * units);
        return v > 0 ? (u64)v : 0ull;
    }
};

// What a sum of sums in units of 2^-unit may be off by, beside CL_PAIR_ERROR of each
// weight: `sum` is them added up, each times what it counts. (Behind it: a unit and a
// half for each of 8 CTAs' threads and two sums, half a one for each of a list's
// entries or a part's elements.)
__device__ __forceinline__ float sum_error(float sum, int V, int unit) {
    const float one = __uint_as_float((uint32_t)(127 + unit) << 23);
    return sum * CL_ADD_ERROR + (float)V * 0x1p-45f * (one + sum * (1.0f / 512.0f)) + 32768.0f;
}

}  // namespace sv
