// sample.cu -- sampling with temperature, top-k, top-p and min-p from given uniforms.
//
// The rollout side of the consistency contract ("RL-Kernel integration roadmap for
// vime", Consistency Contract: logp_old is what the rollout assigned to the token it
// drew, at its temperature): row t of the logits, x_v, with uniform u in [0, 1) gives
//
//   w_v   = exp((x_v - max x) / T)
//   order : x descending, lowest index first among equals
//   n_k   = top_k (all V when 0 or >= V);   S_n = sum of the first n weights of the order
//   n_p   = min{ n : S_n >= top_p S_{n_k} } (n_k when top_p >= 1)
//   n_m   = #{ v : w_v >= min_p }
//   kept  = the first min(n_k, n_p, n_m) of the order
//   token = the first kept v in index order whose running sum of kept weights
//           exceeds u times their total
//
// Every set above is a prefix of the order, so it is described by a pair (key, ties): all
// elements above a key, and the first `ties` in index order of those equal to it.  Sums
// are integers (weight_exp.cuh), so the token depends on the row alone: not on the batch,
// on how the row is split among threads, or on the alignment.
//
// One block scores one row.  Boundaries are found by radix selection, 8 bits of the
// key at a time, on histograms of counts (top-k) or of counts and weights (top-p).
#include <cuda_bf16.h>

#include <cmath>

#include "rlk_internal.h"
#include "weight_exp.cuh"

namespace rlk {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf)
constexpr uint32_t kKeyPosInf = 0xff800000u;   // order_key(+inf)

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Unsigned integers in the order of the floats; -0 and +0 get the same one.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// floor(f * s) for 0 <= f < 1, f = mant 2^-shift; `rest` tells whether the product had a
// fraction.
__device__ __forceinline__ u64 mul_floor(u64 mant, int shift, u64 s, bool& rest) {
    const u64 lo = mant * s, hi = __umul64hi(mant, s);
    rest = false;
    if (shift == 0) return lo;                 // only mant = 0 comes here
    if (shift < 64) {
        rest = (lo << (64 - shift)) != 0;
        return (hi << (64 - shift)) | (lo >> shift);
    }
    if (shift >= 128) {
        rest = (hi | lo) != 0;
        return 0;
    }
    const int t = shift - 64;
    rest = lo != 0 || (t > 0 && (hi << (64 - t)) != 0);
    return hi >> t;
}
// f = mant 2^-shift exactly, for 0 <= f < 1
__device__ __forceinline__ void split_unit(double f, u64& mant, int& shift) {
    const u64 b = __double_as_longlong(f);
    const int e = int(b >> 52);
    mant = e == 0 ? 0 : ((b & 0xfffffffffffffULL) | 0x10000000000000ULL);
    shift = mant == 0 ? 0 : 1075 - e;
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

struct Shared {
    u64 table[kExpEntries];
    unsigned cnt[256], lo[256], hi[256];
    u64 part[kWarps];
    unsigned part_n[kWarps];
    float part_m[kWarps];
    unsigned bad;
    uint32_t key;
    unsigned above_n;
    u64 above_w;
    u64 total;
};

// block-wide sum, in every thread
__device__ __forceinline__ u64 block_sum(u64 v, Shared& sh) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kWarps; ++i) t += sh.part[i];
    return t;
}

// The boundary of a prefix of the order: elements with a key above `key`, and the first
// `ties` of those equal to it.  `above_n` / `above_w`: count and weight above the key.
struct Bound {
    uint32_t key;
    unsigned ties;
    u64 above_w;
};

// Radix selection among the elements of key >= floor_key: the key at which the running
// count (BY_WEIGHT false) or weight of the order reaches `need` >= 1.
template <typename T, bool BY_WEIGHT>
__device__ Bound select(const T* row, int V, const WeightScale& ws, uint32_t floor_key, u64 need,
                        Shared& sh) {
    uint32_t prefix = 0;
    u64 above = 0, above_w = 0;
    for (int level = 3; level >= 0; --level) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += kThreads) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
        const uint32_t mask = level == 3 ? 0u : 0xffffffffu << (8 * (level + 1));
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const float x = to_f32(row[v]);
            const uint32_t k = order_key(x);
            if ((k & mask) != prefix || k < floor_key) continue;
            const uint32_t b = (k >> (8 * level)) & 255u;
            atomicAdd(&sh.cnt[b], 1u);
            const u64 w = fixed_weight(x, ws, sh.table);
            if (w != 0) {
                const unsigned wl = static_cast<unsigned>(w);
                const unsigned old = atomicAdd(&sh.lo[b], wl);
                atomicAdd(&sh.hi[b], static_cast<unsigned>(w >> 32) + (old + wl < old ? 1u : 0u));
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 n = above, w = above_w;
            int b = 255;
            for (; b > 0; --b) {
                const u64 bw = (u64(sh.hi[b]) << 32) | sh.lo[b];
                if ((BY_WEIGHT ? w + bw : n + sh.cnt[b]) >= need) break;
                n += sh.cnt[b];
                w += bw;
            }
            sh.key = prefix | (uint32_t(b) << (8 * level));
            sh.above_n = static_cast<unsigned>(n);
            sh.above_w = w;
        }
        __syncthreads();
        prefix = sh.key;
        above = sh.above_n;
        above_w = sh.above_w;
    }
    Bound r;
    r.key = prefix;
    r.above_w = above_w;
    if (BY_WEIGHT) {
        const u64 w = fixed_weight(key_value(prefix), ws, sh.table);
        r.ties = w == 0 ? 0u : static_cast<unsigned>((need - above_w + w - 1) / w);
    } else {
        r.ties = static_cast<unsigned>(need - above);
    }
    return r;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const T* __restrict__ logits,
                                                          const SampleArgs a) {
    __shared__ Shared sh;
    const int64_t row_i = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.mask != nullptr && a.mask[row_i] == 0) {
        if (tid == 0) {
            a.tokens[row_i] = -1;
            if (a.logp != nullptr) a.logp[row_i] = 0.f;
            if (a.kept_logp != nullptr) a.kept_logp[row_i] = 0.f;
        }
        return;
    }
    const T* row = logits + row_i * a.stride;
    const int V = a.V;
    const double temp = a.temperature_rows != nullptr ? a.temperature_rows[row_i] : a.temperature;
    const int64_t top_k = a.top_k_rows != nullptr ? a.top_k_rows[row_i] : a.top_k;
    const double top_p = a.top_p_rows != nullptr ? a.top_p_rows[row_i] : a.top_p;
    const double min_p = a.min_p_rows != nullptr ? a.min_p_rows[row_i] : a.min_p;
    const float u = a.uniforms[row_i];
    const bool params_ok = temp >= kSampleMinT && temp <= kSampleMaxT && top_k >= 0 &&
                           top_p > 0.0 && min_p >= 0.0 && min_p <= 1.0 && u >= 0.f && u < 1.f;

    if (tid == 0) sh.bad = 0;
    for (int i = tid; i < kExpEntries; i += kThreads) sh.table[i] = kExpTable.v[i];
    __syncthreads();
    // the maximum; NaN and +inf have no softmax
    float m = -INFINITY;
    bool bad = false;
    for (int v = tid; v < V; v += kThreads) {
        const float x = to_f32(row[v]);
        bad |= !(x < INFINITY);
        m = fmaxf(m, x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh.part_m[warp] = m;
    if (bad) atomicOr(&sh.bad, 1u);
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, sh.part_m[i]);
    bad = sh.bad != 0 || m == -INFINITY;
    if (!params_ok || bad) {
        if (tid == 0) {
            a.tokens[row_i] = -1;
            if (a.logp != nullptr) a.logp[row_i] = quiet_nan();
            if (a.kept_logp != nullptr) a.kept_logp[row_i] = quiet_nan();
            if (a.err != nullptr)
                atomicOr(a.err, (bad ? RLK_DEVERR_LOGITS : 0u) |
                                    (params_ok ? 0u : RLK_DEVERR_SAMPLE_PARAM));
        }
        return;
    }
    const double c = 1.4426950408889634074 / temp;
    WeightScale ws;
    ws.m = m;
    ws.ch = static_cast<float>(c);
    ws.cl = static_cast<float>(c - static_cast<double>(ws.ch));
    ws.shift = 62 - a.bits;

    u64 part = 0;
    for (int v = tid; v < V; v += kThreads) part += fixed_weight(to_f32(row[v]), ws, sh.table);
    const u64 all = block_sum(part, sh);

    Bound keep{kKeyNegInf, 0u, all};       // nothing cut: the -inf entries weigh nothing
    u64 kept_k = all;                      // weight of the first n_k
    if (top_k > 0 && top_k < V) {
        keep = select<T, false>(row, V, ws, 0u, static_cast<u64>(top_k), sh);
        kept_k = keep.above_w + keep.ties * fixed_weight(key_value(keep.key), ws, sh.table);
    }
    if (top_p < 1.0) {
        u64 mant;
        int shift;
        bool rest;
        split_unit(top_p, mant, shift);
        u64 need = mul_floor(mant, shift, kept_k, rest);
        need += rest ? 1 : 0;
        if (need == 0) need = 1;
        keep = select<T, true>(row, V, ws, keep.key, need, sh);
    }
    if (min_p > 0.0) {
        // the smallest float with x >= max + T log(min_p): every element from it on is kept
        const double at = static_cast<double>(m) + temp * log(min_p);
        float f = static_cast<float>(at);
        uint32_t k = order_key(f);
        if (static_cast<double>(f) < at) k += 1;
        if (k > keep.key) keep = Bound{k - 1, 0u, 0};
    }

    // the kept set in index order: thread j owns a contiguous stretch of the row
    const int each = (V + kThreads - 1) / kThreads;
    const int v0 = min(V, tid * each), v1 = min(V, v0 + each);
    const u64 wt = fixed_weight(key_value(keep.key), ws, sh.table);
    u64 w_mine = 0;
    unsigned n_mine = 0;
    for (int v = v0; v < v1; ++v) {
        const float x = to_f32(row[v]);
        const uint32_t k = order_key(x);
        if (k > keep.key) w_mine += fixed_weight(x, ws, sh.table);
        n_mine += k == keep.key ? 1u : 0u;
    }
    u64 w_before = w_mine;
    unsigned n_before = n_mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const u64 ow = __shfl_up_sync(0xffffffffu, w_before, off);
        const unsigned on = __shfl_up_sync(0xffffffffu, n_before, off);
        if (lane >= off) w_before += ow, n_before += on;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = w_before, sh.part_n[warp] = n_before;
    __syncthreads();
    w_before -= w_mine;
    n_before -= n_mine;
    u64 w_all = 0;
    unsigned n_all = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) w_before += sh.part[i], n_before += sh.part_n[i];
        w_all += sh.part[i], n_all += sh.part_n[i];
    }
    const u64 kept = w_all + min(n_all, keep.ties) * wt;
    u64 mant;
    int shift;
    bool rest;
    split_unit(static_cast<double>(u), mant, shift);
    const u64 target = mul_floor(mant, shift, kept, rest);     // token: running sum > target
    u64 run = w_before + min(n_before, keep.ties) * wt;
    const u64 end = run + w_mine + (min(n_before + n_mine, keep.ties) - min(n_before, keep.ties)) * wt;
    if (!(run <= target && target < end)) return;
    unsigned seen = n_before;
    for (int v = v0; v < v1; ++v) {
        const float x = to_f32(row[v]);
        const uint32_t k = order_key(x);
        if (k > keep.key)
            run += fixed_weight(x, ws, sh.table);
        else if (k == keep.key && seen++ < keep.ties)
            run += wt;
        if (run > target) {
            a.tokens[row_i] = v;
            const double z = (static_cast<double>(x) - static_cast<double>(m)) / temp;
            const u64 one = u64(1) << a.bits;
            const float unit = exp2f(static_cast<float>(-a.bits));
            // the largest weight is `one`, so sums minus it are never negative
            if (a.logp != nullptr)
                a.logp[row_i] = static_cast<float>(
                    z - log1pf(static_cast<float>(all - one) * unit));
            if (a.kept_logp != nullptr)
                a.kept_logp[row_i] = static_cast<float>(
                    z - log1pf(static_cast<float>(kept - one) * unit));
            return;
        }
    }
}

}  // namespace

size_t sample_workspace(int64_t N, int64_t V) {
    (void)N;
    (void)V;
    return 0;
}

cudaError_t launch_sample(const void* logits, bool bf16, const SampleArgs& args,
                          cudaStream_t stream) {
    if (bf16)
        sample_kernel<__nv_bfloat16><<<args.N, kThreads, 0, stream>>>(
            static_cast<const __nv_bfloat16*>(logits), args);
    else
        sample_kernel<float><<<args.N, kThreads, 0, stream>>>(static_cast<const float*>(logits),
                                                             args);
    return cudaGetLastError();
}

}  // namespace rlk
