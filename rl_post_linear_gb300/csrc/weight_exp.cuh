// weight_exp.cuh -- softmax weights as fixed-point integers.
//
// The sampler compares running sums of exp((x_v - max)/T) with u times their total.  Near
// a border that needs sums good to about 1e-12 of the total (152k borders a row), which
// fp32 does not give, and fp64 arithmetic runs at 1/64 of the fp32 rate.  So a weight is
//
//   w = round( 2^bits 2^(-t) ),   t = (max - x) log2(e) / T
//
// as a 64-bit integer: sums are exact, associative (any split of the row gives the same
// sum) and compared as integers.  What is lost is each weight's rounding, half a unit: V 2^-47 of
// the maximum's weight in all at most with 46 bits, 1e-9 for 152k weights that are rounded the same
// way (a long tail of equal, light tokens), and far less where they are not.
//
// 2^(-t) is formed by the table method of P. T. P. Tang ("Table-driven implementation of
// the exponential function in IEEE floating-point arithmetic", ACM TOMS 15(2), 1989) in
// integer arithmetic: t is carried as an unevaluated sum of two floats, split into
// n + j/1024 + y with |y| <= 2^-11, and 2^(-t) = 2^-n T[j] (1 - q), T[j] = 2^(-j/1024) from
// a table and q = 1 - e^(-a), a = y ln 2, from three terms of its series (the fourth is
// below 2^-50).  Each step keeps 41 or more fractional bits of a value near 1: w is off by
// at most 3 units of 2^-41 of itself, plus half a unit of its own (against 80-bit host
// arithmetic over 8 M arguments: at most 2^-39.9, 2^-41.8 in the root mean square).  A weight below
// half a unit is 0.
#ifndef RLK_WEIGHT_EXP_CUH_
#define RLK_WEIGHT_EXP_CUH_

#include <cstdint>

namespace rlk {

constexpr int kExpEntries = 1024;

struct ExpTable {
    unsigned long long v[kExpEntries];   // 2^(-j/1024) * 2^62
};

constexpr ExpTable make_exp_table() {
    ExpTable t{};
    for (int j = 0; j < kExpEntries; ++j) {
        const double a = -double(j) / kExpEntries * 0.69314718055994530942;
        double sum = 1.0, term = 1.0;
        for (int i = 1; i < 24; ++i) {
            term *= a / i;
            sum += term;
        }
        // 2^62 sum, from a double: exact scaling
        t.v[j] = static_cast<unsigned long long>(sum * 4611686018427387904.0);
    }
    return t;
}

__device__ const __align__(16) ExpTable kExpTable = make_exp_table();

// t = d (ch + cl), d = m - x
struct WeightScale {
    float m;        // row maximum
    float ch, cl;   // log2(e)/T in two floats
    int shift;      // 62 - bits
};

// t = th + tl of an x <= m; x = -inf gives th = inf (and no meaning to tl)
__device__ __forceinline__ void scaled_distance(float x, const WeightScale& s, float& th,
                                                float& tl) {
    // d = dh + dl exactly (two-sum)
    const float dh = s.m - x;
    const float bb = dh - s.m;
    const float dl = (s.m - (dh - bb)) + (-x - bb);
    th = __fmul_rn(dh, s.ch);
    tl = fmaf(dh, s.cl, fmaf(dl, s.ch, fmaf(dh, s.ch, -th)));
}

// 2^bits 2^(-t) from t = th + tl split as th = k / 1024 + r (k = idx), |r| <= 2^-11
__device__ __forceinline__ unsigned long long fixed_power(int idx, float r_scaled, float tl_scaled,
                                                          const WeightScale& s,
                                                          const unsigned long long* table) {
    // y = t - k / 1024 and a = y ln 2 by 2^41, |a| < 2^30 (a tl without meaning ends at w = 0)
    const int y = __float2int_rn(r_scaled) + __float2int_rn(tl_scaled);
    const int a = static_cast<int>((static_cast<long long>(y) * 1488522236 + (1LL << 30)) >> 31);
    const int a2 = __mulhi(a, a);                      // a^2 by 2^50
    const int a3 = __mulhi(a2, a);                     // a^3 by 2^59
    const int q = a - (a2 >> 10) + (__mulhi(a3, 715827883) >> 18);
    const unsigned long long t62 = table[idx & (kExpEntries - 1)];
    const unsigned long long w =
        t62 - ((static_cast<long long>(q) * static_cast<int>(t62 >> 32)) >> 9);
    const int sh = min((idx >> 10) + s.shift - 1, 63);     // 15 <= sh; w < 2^62 + 2^51
    return ((w >> sh) + 1) >> 1;
}

constexpr float kTwo41 = 2199023255552.f;

// table: the 1024 entries (shared memory).  x <= m, both finite or x = -inf.
__device__ __forceinline__ unsigned long long fixed_weight(float x, const WeightScale& s,
                                                           const unsigned long long* table) {
    float th, tl;
    scaled_distance(x, s, th, tl);
    th = fminf(th, 63.f);                              // below half a unit from 62 on
    const float big = th + 12288.f;                    // ulp 2^-10: rounds t to k / 1024
    const float r = th - (big - 12288.f);              // exact
    return fixed_power(__float_as_int(big) - __float_as_int(12288.f), r * kTwo41, tl * kTwo41, s,
                       table);
}

#ifdef __CUDACC__
// Two weights, the same values, with paired fp32 instructions.
__device__ __forceinline__ void fixed_weights(float2 x, const WeightScale& s,
                                              const unsigned long long* table,
                                              unsigned long long& w0, unsigned long long& w1) {
    const float2 m = make_float2(s.m, s.m), minus = make_float2(-1.f, -1.f);
    const float2 dh = __ffma2_rn(x, minus, m);         // m - x, as rounded once
    const float2 bb = __fadd2_rn(dh, make_float2(-s.m, -s.m));
    const float2 dl = __fadd2_rn(__ffma2_rn(__ffma2_rn(bb, minus, dh), minus, m),
                                 __ffma2_rn(x, minus, make_float2(-bb.x, -bb.y)));
    const float2 ch = make_float2(s.ch, s.ch), cl = make_float2(s.cl, s.cl);
    float2 th = __fmul2_rn(dh, ch);
    const float2 tl = __ffma2_rn(
        dh, cl, __ffma2_rn(dl, ch, __ffma2_rn(dh, ch, make_float2(-th.x, -th.y))));
    th = make_float2(fminf(th.x, 63.f), fminf(th.y, 63.f));
    const float2 big = __fadd2_rn(th, make_float2(12288.f, 12288.f));
    const float2 r = __ffma2_rn(__fadd2_rn(big, make_float2(-12288.f, -12288.f)), minus, th);
    const float2 up = make_float2(kTwo41, kTwo41);
    const float2 rs = __fmul2_rn(r, up), ts = __fmul2_rn(tl, up);
    constexpr int kZero = 0x46400000;                  // bits of 12288.f
    w0 = fixed_power(__float_as_int(big.x) - kZero, rs.x, ts.x, s, table);
    w1 = fixed_power(__float_as_int(big.y) - kZero, rs.y, ts.y, s, table);
}
#endif

}  // namespace rlk

#endif  // RLK_WEIGHT_EXP_CUH_
