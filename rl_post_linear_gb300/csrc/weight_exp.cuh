// weight_exp.cuh -- softmax weights as fixed-point integers.
//
// The sampler compares running sums of exp((x_v - max)/T) with u times their total.  Near
// a border that needs sums good to about 1e-12 of the total (152k borders a row), which
// fp32 does not give, and fp64 arithmetic runs at 1/64 of the fp32 rate.  So a weight is
//
//   w = round( 2^bits 2^(-t) ),   t = (max - x) log2(e) / T
//
// as a 64-bit integer: sums are exact, associative (any split of the row gives the same
// sum) and compared as integers.
//
// 2^(-t) is formed by the table method of P. T. P. Tang ("Table-driven implementation of
// the exponential function in IEEE floating-point arithmetic", ACM TOMS 15(2), 1989) in
// integer arithmetic: t is carried as an unevaluated sum of two floats, split into
// n + j/1024 + y with |y| <= 2^-11, and 2^(-t) = 2^-n T[j] (1 - q), T[j] = 2^(-j/1024) from
// a table and q = 1 - e^(-a), a = y ln 2, from three terms of its series (the fourth is
// below 2^-50).  Each step keeps 41 or more fractional bits of a value near 1: w is off by
// at most 3 units of 2^-41 of itself, plus half a unit of its own (against 80-bit host
// arithmetic over 8 M arguments: at most 2^-39.9, 2^-41.8 in the root mean square).
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

// table: the 1024 entries (shared memory).  x <= m, both finite or x = -inf.
__device__ __forceinline__ unsigned long long fixed_weight(float x, const WeightScale& s,
                                                           const unsigned long long* table) {
    float th, tl;
    scaled_distance(x, s, th, tl);
    th = fminf(th, 63.f);                              // below half a unit from 62 on
    const float big = th + 12288.f;                    // ulp 2^-10: rounds t to j / 1024
    const int idx = __float_as_int(big) - __float_as_int(12288.f);
    const float r = th - (big - 12288.f);              // exact, |r| <= 2^-11
    // y = t - j / 1024 and a = y ln 2 by 2^41, |a| < 2^30 (a tl without meaning ends at w = 0)
    const int y = __float2int_rn(r * 2199023255552.f) + __float2int_rn(tl * 2199023255552.f);
    const int a = static_cast<int>((static_cast<long long>(y) * 1488522236 + (1LL << 30)) >> 31);
    const int a2 = __mulhi(a, a);                      // a^2 by 2^50
    const int a3 = __mulhi(a2, a);                     // a^3 by 2^59
    const int q = a - (a2 >> 10) + (__mulhi(a3, 715827883) >> 18);
    const unsigned long long t62 = table[idx & (kExpEntries - 1)];
    const unsigned long long w =
        t62 - ((static_cast<long long>(q) * static_cast<int>(t62 >> 32)) >> 9);
    const int sh = min((idx >> 10) + s.shift, 64);     // 16 <= sh; w < 2^62 + 2^51
    return ((w >> (sh - 1)) + 1) >> 1;
}

}  // namespace rlk

#endif  // RLK_WEIGHT_EXP_CUH_
