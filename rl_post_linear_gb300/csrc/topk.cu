// topk.cu -- the largest K log-probs of each row of logits, with their tokens.
//
// What a teacher keeps of its logits for a student (rlk_linear_topk_kl_fwd takes it), and what
// a server returns with a token.  Per row x_v at temperature T:
//
//   lse = log sum_v exp(x_v / T);  order: x descending, lowest index first among equals
//   ids, logp = the order's first K v, x_v / T - lse
//
// One pass over the row: a warp takes units of 1024 columns, of which each lane holds 32 (its
// segment).  A unit leaves its maximum and an fp32 sum of 2^((x - max) k), k = log2(e)/T; each
// segment leaves its maximum.  K segments reach the K-th largest of the segments' maxima, so
// every element of the answer reaches it too, and lies in a segment that does.  One block of the
// row's cluster takes such a bound from a histogram of the maxima, reads the few segments that
// reach it again, and sorts what it finds there.  A row where more is found than the list holds
// (ties in great number, a row sorted by token) is searched by its keys' digits instead.
//
// Order and ties go by whole numbers: keys in the order of the floats, over the column.  Sums
// run in an order that depends on V alone, so a row's results do not depend on the batch.
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnit = 1024;              // columns of a unit
constexpr int kBins = 2048;
constexpr int kList = 2048;              // elements of the list, a power of two
constexpr int kMaxSegments = 8192;
constexpr uint32_t kKeyNegInf = 0x007fffffu;
constexpr float kLn2 = 0.693147180559945309f;

// Unsigned integers in the order of the floats; -0 and +0 get the same one.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <typename P>
__device__ __forceinline__ P* peer(P* p, uint32_t rank) {
    u64 a;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
    return reinterpret_cast<P*>(a);
}

// How a row's units are divided into segments: `halves` of a lane's columns, or `lanes` of them
// together.
struct Segments {
    int halves, lanes;
    __host__ __device__ int per_unit() const { return 32 * halves / lanes; }
};

// VEC consecutive columns from c on, as floats; -inf past the row's end.
template <typename T>
__device__ __forceinline__ void load_piece(const T* row, int V, int c, bool vec,
                                           float (&x)[16 / sizeof(T)]) {
    constexpr int VEC = 16 / sizeof(T);
    alignas(16) T v[VEC];
    if (vec && c + VEC <= V) {
        *reinterpret_cast<uint4*>(v) = __ldg(reinterpret_cast<const uint4*>(row + c));
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = to_f32(v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = c + e < V ? to_f32(row[c + e]) : -INFINITY;
    }
}

struct Shared {
    uint32_t hist[kBins];
    u64 list[kList];
    float warp_f[kWarps];
    uint32_t warp_n[kWarps];
    uint32_t n, queued;
    uint32_t bin, below, through;        // of the histogram: the bin K falls on, counts to it
};

// Exclusive prefix of n over the block, and the total.
__device__ __forceinline__ uint32_t block_prefix(uint32_t n, Shared& sh, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    __syncthreads();
    if (lane == 31) sh.warp_n[warp] = inc;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh.warp_n[w];
        total += sh.warp_n[w];
    }
    return before + inc - n;
}

// The first bin at which the running count, `base` before the first, reaches `want`.
__device__ __forceinline__ void find_bin(Shared& sh, int bins, uint32_t base, uint32_t want) {
    const int each = bins / kThreads;
    uint32_t own = 0;
    for (int b = 0; b < each; ++b) own += sh.hist[threadIdx.x * each + b];
    uint32_t total;
    uint32_t run = base + block_prefix(own, sh, total);
    if (run < want && run + own >= want) {
        for (int b = 0; b < each; ++b) {
            const uint32_t n = sh.hist[threadIdx.x * each + b];
            if (run + n >= want) {
                sh.bin = threadIdx.x * each + b;
                sh.below = run;
                sh.through = run + n;
                break;
            }
            run += n;
        }
    }
    __syncthreads();
}

// A key that at least `want` segments reach, and not many more: the histogram's window closes
// in on it.  All segments above -inf have one; `want` of them at least.
__device__ __noinline__ uint32_t segment_bound(const float* segmax, int nseg, uint32_t lo,
                                               uint32_t hi, uint32_t want, Shared& sh) {
    const uint32_t slack = max(32u, want / 4);
    uint32_t base = 0;
    while (true) {
        const int shift = max(0, 21 - __clz((hi - lo) | 1u));      // (hi - lo) >> shift < 2048
        for (int b = threadIdx.x; b < kBins; b += kThreads) sh.hist[b] = 0;
        __syncthreads();
        for (int s = threadIdx.x; s < nseg; s += kThreads) {
            const uint32_t key = order_key(segmax[s]);
            if (key >= lo && key <= hi) atomicAdd(&sh.hist[(hi - key) >> shift], 1u);
        }
        __syncthreads();
        find_bin(sh, kBins, base, want);
        const uint32_t bin = sh.bin, through = sh.through;
        base = sh.below;
        const u64 edge = (u64(bin) + 1) << shift;                  // keys of bins 0 .. bin
        const uint32_t bound = edge > u64(hi - lo) ? lo : hi - static_cast<uint32_t>(edge) + 1;
        if (through <= want + slack || shift == 0) return bound;
        hi -= bin << shift;
        lo = bound;
        __syncthreads();
    }
}

// Sorts sh.list[0, n) descending; n <= kList.
__device__ __noinline__ void sort_list(Shared& sh, int n) {
    int size = 2;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) sh.list[i] = 0;
    __syncthreads();
    for (int run = 2; run <= size; run <<= 1) {
        for (int d = run >> 1; d > 0; d >>= 1) {
            for (int i = threadIdx.x; i < size; i += kThreads) {
                const int j = i ^ d;
                if (j > i) {
                    const u64 p = sh.list[i], q = sh.list[j];
                    if ((p < q) == ((i & run) == 0)) {
                        sh.list[i] = q;
                        sh.list[j] = p;
                    }
                }
            }
            __syncthreads();
        }
    }
}

__device__ __forceinline__ u64 element(uint32_t key, int col) {
    return (u64(key) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}

// The K largest of the row into the list, by the digits of their keys: for rows whose segments
// say too little.  Leaves sh.n.
template <typename T>
__device__ __noinline__ void select_digits(const T* row, int V, uint32_t K, Shared& sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t prefix = 0, above = 0;          // above: keys larger than the prefix's
    for (int shift = 24; shift >= 0; shift -= 8) {
        sh.hist[tid] = 0;
        __syncthreads();
        for (int c0 = 0; c0 < V; c0 += kThreads) {
            const int c = c0 + tid;
            const uint32_t key = c < V ? order_key(to_f32(row[c])) : 0;
            // bins in descending order of the digit; -inf is never counted
            const bool in = key > kKeyNegInf && (shift == 24 || (key >> (shift + 8)) == prefix);
            const uint32_t bin = in ? 255 - ((key >> shift) & 255) : 256;
            const uint32_t same = __match_any_sync(0xffffffffu, bin);
            if (in && lane == __ffs(same) - 1) atomicAdd(&sh.hist[bin], __popc(same));
        }
        if (tid == 0) sh.through = 0;
        __syncthreads();
        find_bin(sh, 256, above, K);
        if (sh.through == 0) break;          // fewer than K above -inf (in the first step only)
        prefix = (prefix << 8) | (255 - sh.bin);
        above = sh.below;
        __syncthreads();
    }
    // everything above the K-th key, and of its equals the lowest columns
    const bool all = sh.through == 0;
    const uint32_t kth = all ? kKeyNegInf : prefix;
    uint32_t n = 0, ties = all ? 0 : K - above;
    for (int c0 = 0; c0 < V && n < K; c0 += kThreads) {
        const int c = c0 + tid;
        const uint32_t key = c < V ? order_key(to_f32(row[c])) : 0;
        uint32_t total_tie = 0, total;
        const uint32_t before = block_prefix(key == kth && !all ? 1 : 0, sh, total_tie);
        const bool take = key > kth || (!all && key == kth && before < ties);
        const uint32_t at = block_prefix(take ? 1 : 0, sh, total);
        if (take) sh.list[n + at] = element(key, c);
        n += total;
        ties -= min(ties, total_tie);
    }
    __syncthreads();
    if (tid == 0) sh.n = n;
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    topk_kernel(const T* logits, const TopkArgs a, const Segments seg, int units, int ranks) {
    constexpr int VEC = 16 / sizeof(T), LOADS = kUnit / 32 / VEC;
    extern __shared__ uint4 smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    float2* unit_ms = reinterpret_cast<float2*>(&sh + 1);
    float* segmax = reinterpret_cast<float*>(unit_ms + units);
    const int nseg = units * seg.per_unit();
    const int row = blockIdx.x / ranks;
    const uint32_t rank = ranks > 1 ? cluster_ctarank() : 0u;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.mask != nullptr && a.mask[row] == 0) {
        if (rank == 0) {
            for (int j = tid; j < a.K; j += kThreads) {
                a.ids[static_cast<int64_t>(row) * a.K + j] = -1;
                a.logp[static_cast<int64_t>(row) * a.K + j] = 0.f;
            }
            if (tid == 0 && a.lse != nullptr) a.lse[row] = 0.f;
        }
        return;
    }
    const T* x_row = logits + row * a.stride;
    float2* to_ms = unit_ms;
    float* to_seg = segmax;
    if (ranks > 1) {
        cluster_sync();                          // the first block is there
        to_ms = peer(unit_ms, 0);
        to_seg = peer(segmax, 0);
    }
    for (int u = static_cast<int>(rank) * kWarps + warp; u < units; u += ranks * kWarps) {
        float x[LOADS][VEC];
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
            load_piece(x_row, a.V, u * kUnit + (j * 32 + lane) * VEC, a.vec_ok, x[j]);
        float half[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                half[2 * j / LOADS] = fmaxf(half[2 * j / LOADS], x[j][e]);
        float m = fmaxf(half[0], half[1]);
        if (seg.halves == 2) {
            to_seg[u * 64 + lane * 2] = half[0];
            to_seg[u * 64 + lane * 2 + 1] = half[1];
            m = warp_max(m);
        } else {
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                if (off == seg.lanes && lane % off == 0) to_seg[(u * 32 + lane) / off] = m;
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            }
            if (seg.lanes == 32 && lane == 0) to_seg[u] = m;
        }
        const float mm = m == -INFINITY ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += ex2_approx((x[j][e] - mm) * a.k);
        s = warp_sum(s);
        if (lane == 0) to_ms[u] = make_float2(m, s);
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // the row's maximum and sum; the range of the segments' maxima
    float m = -INFINITY, low = INFINITY;
    for (int u = tid; u < units; u += kThreads) m = fmaxf(m, unit_ms[u].x);
    uint32_t finite = 0;
    for (int s = tid; s < nseg; s += kThreads) {
        const float v = segmax[s];
        if (v > -INFINITY) ++finite, low = fminf(low, v);
    }
    m = warp_max(m);
    if (lane == 0) sh.warp_f[warp] = m;
    uint32_t total;
    block_prefix(finite, sh, total);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh.warp_f[w]);
    __syncthreads();
    low = -warp_max(-low);
    if (lane == 0) sh.warp_f[warp] = low;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) low = fminf(low, sh.warp_f[w]);
    const float mm = m == -INFINITY ? 0.f : m;
    float s = 0.f;
    for (int u = tid; u < units; u += kThreads) {
        const float2 p = unit_ms[u];
        if (!(p.x == -INFINITY && p.y == 0.f))   // nothing in it (but not NaN)
            s = fmaf(p.y, ex2_approx((p.x - mm) * a.k), s);
    }
    s = warp_sum(s);
    __syncthreads();
    if (lane == 0) sh.warp_f[warp] = s;
    if (tid == 0) sh.n = sh.queued = 0;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sh.warp_f[w];
    int64_t* ids = a.ids + static_cast<int64_t>(row) * a.K;
    float* logp = a.logp + static_cast<int64_t>(row) * a.K;
    if (!(s > 0.f && s < INFINITY && fabsf(m) < INFINITY)) {
        for (int j = tid; j < a.K; j += kThreads) {
            ids[j] = -1;
            logp[j] = __int_as_float(0x7fc00000);
        }
        if (tid == 0) {
            if (a.lse != nullptr) a.lse[row] = __int_as_float(0x7fc00000);
            if (a.err != nullptr) atomicOr(a.err, RLK_DEVERR_LOGITS);
        }
        return;
    }
    const float ln_s = lg2_approx(s) * kLn2;
    if (tid == 0 && a.lse != nullptr) a.lse[row] = fmaf(m, a.inv_t, ln_s);

    const uint32_t K = static_cast<uint32_t>(a.K);
    const uint32_t bound =
        total < K ? kKeyNegInf + 1
                  : segment_bound(segmax, nseg, order_key(low), order_key(m), K, sh);
    __syncthreads();
    // the segments that reach it (their numbers take the histogram's place), then their elements
    for (int g = tid; g < nseg; g += kThreads)
        if (order_key(segmax[g]) >= bound) {
            const uint32_t at = atomicAdd(&sh.queued, 1u);
            if (at < kBins) sh.hist[at] = g;
        }
    __syncthreads();
    const uint32_t queued = sh.queued;
    if (queued <= kBins) {
        const int loads = LOADS / seg.halves, pieces = loads * seg.lanes;
        const int per_unit = seg.per_unit();
        for (int i = tid; i < static_cast<int>(queued) * pieces; i += kThreads) {
            const int g = sh.hist[i / pieces], p = i % pieces;
            const int u = g / per_unit, in = g % per_unit;
            const int j = p / seg.lanes + (seg.halves == 2 ? (in & 1) * loads : 0);
            const int l = seg.halves == 2 ? in / 2 : in * seg.lanes + p % seg.lanes;
            const int c = u * kUnit + (j * 32 + l) * VEC;
            float x[VEC];
            load_piece(x_row, a.V, c, a.vec_ok, x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const uint32_t key = order_key(x[e]);
                if (key < bound) continue;
                const uint32_t at = atomicAdd(&sh.n, 1u);
                if (at < kList) sh.list[at] = element(key, c + e);
            }
        }
    }
    __syncthreads();
    if (queued > kBins || sh.n > kList) select_digits(x_row, a.V, K, sh);
    const int n = static_cast<int>(sh.n);
    sort_list(sh, n);
    for (int j = tid; j < a.K; j += kThreads) {
        if (j < n) {
            const u64 el = sh.list[j];
            ids[j] = static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(el));
            logp[j] = fmaf(key_value(static_cast<uint32_t>(el >> 32)) - m, a.inv_t, -ln_s);
        } else {
            ids[j] = -1;
            logp[j] = -INFINITY;
        }
    }
}

template <typename T>
cudaError_t launch_typed(const T* logits, const TopkArgs& a, cudaStream_t stream) {
    const int units = (a.V + kUnit - 1) / kUnit;
    Segments seg{1, 1};
    if (units * 32 < 4 * a.K) seg.halves = 2;
    while (units * seg.per_unit() > kMaxSegments) seg.lanes *= 2;
    int ranks = units >= 64 ? 8 : units >= 32 ? 4 : units >= 16 ? 2 : 1;
    while (ranks > 1 && static_cast<int64_t>(a.N) * ranks > 608) ranks /= 2;
    const size_t smem = sizeof(Shared) + units * sizeof(float2) +
                        static_cast<size_t>(units) * seg.per_unit() * sizeof(float);
    constexpr int kMost = 100 * 1024;        // of any vocabulary
    static_assert(sizeof(Shared) + kMaxTopkColumns / kUnit * 8 + kMaxSegments * 4 <= kMost,
                  "a block's shared memory");
    void (*kernel)(const T*, const TopkArgs, const Segments, int, int) = topk_kernel<T>;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, logits, a, seg, units, ranks);
}

}  // namespace

cudaError_t launch_topk(const void* logits, bool bf16, const TopkArgs& args, cudaStream_t stream) {
    if (bf16) return launch_typed(static_cast<const __nv_bfloat16*>(logits), args, stream);
    return launch_typed(static_cast<const float*>(logits), args, stream);
}

}  // namespace rlk
