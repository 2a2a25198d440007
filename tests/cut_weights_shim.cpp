// Test-only shim: compiles the kernels' weights (csrc/cut_weights.cuh) for the
// host, where the few functions of the device that they use are written out, so
// that the tests can compare single weights and sums with longer arithmetic.
#include <cmath>
#include <cstdint>
#include <cstring>

#define __device__
#define __forceinline__ inline

static float __fadd_rn(float a, float b) { return a + b; }
static float __fsub_rn(float a, float b) { return a - b; }
static float __fmul_rn(float a, float b) { return a * b; }
static float __fmaf_rn(float a, float b, float c) { return std::fmaf(a, b, c); }
// (nearest, ties to even: the mode that a process starts with; out of range or NaN, as
// where a weight is not used, gives some number)
static long long __float2ll_rn(float x) { return std::fabs(x) < 0x1p63f ? std::llrintf(x) : 0; }
static int __float2int_rn(float x) { return std::fabs(x) < 0x1p31f ? (int)std::llrintf(x) : 0; }
static uint32_t __float_as_uint(float x) {
    uint32_t u;
    std::memcpy(&u, &x, 4);
    return u;
}
static float __uint_as_float(uint32_t u) {
    float x;
    std::memcpy(&x, &u, 4);
    return x;
}
using std::fabs;

namespace sv {
struct f32x2 {
    float a, b;
};
static f32x2 pack2(float a, float b) { return {a, b}; }
static void unpack2(f32x2 r, float& a, float& b) { a = r.a, b = r.b; }
static f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) { return {std::fmaf(x.a, y.a, z.a), std::fmaf(x.b, y.b, z.b)}; }
static f32x2 add2(f32x2 x, f32x2 y) { return {x.a + y.a, x.b + y.b}; }
struct ff {
    float hi, lo;
};
static ff two_sum(float a, float b) {
    const float s = a + b, bb = s - a;
    return {s, (a - (s - bb)) + (b - bb)};
}
}  // namespace sv

#include "cut_weights.cuh"

static const sv::ExpTable table = sv::make_exp_table();

static sv::RowScale scale(float top, float T) {
    const double c = 1.4426950408889634 * sv::CL_EXP * (1.0 / (double)T);
    sv::RowScale s;
    sv::set_scale(s, top, (float)c, (float)(c - (double)(float)c), (float)(100.0 / 1.4426950408889634) * T);
    sv::set_unit(s, 44);
    return s;
}

extern "C" int cut_unit() { return 44; }
extern "C" int cut_unit_of(float sum) { return sv::unit_of(sum); }

// Each logit's weight in units.
extern "C" void cut_weights(const float* z, int n, float top, float T, unsigned long long* out) {
    const sv::RowScale s = scale(top, T);
    for (int i = 0; i < n; ++i) out[i] = sv::weight(z[i], s, table.e);
}
extern "C" void cut_weights_in(const float* z, int n, float top, float T, int unit, unsigned long long* out) {
    const sv::RowScale s = scale(top, T);
    for (int i = 0; i < n; ++i) out[i] = sv::weight(z[i], s, table.e, unit, sv::none_of(unit));
}

// The sum of one thread's logits in floats, in units of 2^-unit: pieces of `per`
// elements, an even number of them; below `low` a logit counts as that.
extern "C" unsigned long long cut_sum(const float* z, int n, float top, float T, int per, int unit) {
    static sv::ExpEntry copies[sv::CL_EXP * sv::CL_COPIES];
    for (int i = 0; i < sv::CL_EXP * sv::CL_COPIES; ++i) copies[i] = table.e[i / sv::CL_COPIES];
    const sv::RowScale s = scale(top, T);
    sv::WeightSum sum;
    for (int i = 0; i + per <= n; i += per) {
        for (int e = 0; e < per; e += 2) {
            const float a = z[i + e], b = z[i + e + 1];
            sum.add(a >= s.low ? a : s.low, b >= s.low ? b : s.low, s, copies, e == 0);
        }
        sum.end_piece();
    }
    return sum.total(unit);
}

extern "C" float cut_pair_error() { return sv::CL_PAIR_ERROR; }
extern "C" float cut_sum_error(float sum, int V, int unit) { return sv::sum_error(sum, V, unit); }
