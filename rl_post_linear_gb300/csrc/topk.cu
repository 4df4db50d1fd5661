// topk.cu -- the largest K log-probs of each row of logits, with their tokens.
//
// What a teacher keeps of its logits for a student (rlk_linear_topk_kl_fwd takes it), and what
// a server returns with a token.  Per row x_v at temperature T:
//
//   lse = log sum_v exp(x_v / T);  order: x descending, lowest index first among equals
//   ids, logp = the order's first K v, x_v / T - lse
//
// One pass over the row, in units of four 16-byte loads a lane of a warp.  Units are dealt to a
// number of streams that depends on V alone; of a stream each lane carries its maximum and an fp32
// sum of 2^((x - max) k), k = log2(e)/T.  Each segment of a unit (a lane's columns, or those of a
// few lanes) leaves the key of its maximum.  K segments reach the K-th largest of the segments'
// maxima, so every element of the answer reaches it too, and lies in a segment that does.  One
// block of the row's cluster takes such a bound from a histogram of the maxima, reads the few
// segments that reach it again, and puts what it finds there in order by a second histogram.  A
// row where more is found than the list holds (ties in great number, a row sorted by token) is
// searched by its keys' digits instead.
//
// Order and ties go by whole numbers: keys in the order of the floats, over the column.  Sums
// run in an order that depends on V alone, so a row's results do not depend on the batch.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

typedef unsigned long long u64;

constexpr int kLoads = 4;                // 16-byte loads a lane of a unit
constexpr int kBins = 2048;
constexpr int kQueue = 2048;             // segments that are read again
constexpr int kPieces = 8192;            // and 16-byte pieces of them
constexpr int kList = 2048;              // elements of the longest list
constexpr int kMaxSegments = 10240;
constexpr int kMaxStreams = 128;
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

// maximum over the warp, by an integer reduction of order-preserving bits
__device__ __forceinline__ float warp_max(float v) {
    const int b = __float_as_int(v);
    const int k = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
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

template <typename T>
struct Unit {
    static constexpr int VEC = 16 / sizeof(T), WORDS = 4 * kLoads;
    static constexpr int kColumns = 32 * kLoads * VEC;
    uint32_t w[WORDS];                   // as they lie in memory

    __device__ __forceinline__ static int column(int unit, int load, int lane) {
        return unit * kColumns + (load * 32 + lane) * VEC;
    }
    // A unit into a slot of a warp's ring in shared memory, on its way while others are worked
    // on; -inf past the row's end.  `off` is how many bytes behind a 16-byte border the row
    // starts: the copies start on the border, so a slot holds one piece more than a unit.  At 0
    // each lane copies just what it reads itself and no barrier is needed.  A unit whose last
    // piece reaches past the row is read by its elements.
    __device__ __forceinline__ static bool whole(int V, int unit, int off) {
        return (unit + 1) * kColumns + (off != 0 ? VEC : 0) <= V;
    }
    __device__ __forceinline__ static void fetch(uint4* slot, const T* row, int V, int unit,
                                                 int lane, int off) {
        if (whole(V, unit, off)) {
            const uint8_t* from = reinterpret_cast<const uint8_t*>(row + column(unit, 0, 0)) - off;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) copy16(slot + j * 32 + lane, from + (j * 32 + lane) * 16);
            if (off != 0 && lane == 0) copy16(slot + kLoads * 32, from + kLoads * 512);
        } else {
            fetch_edge(slot + lane, row, V, unit, lane);
        }
    }
    // all loads on their way at once
    __device__ __noinline__ static void fetch_edge(uint4* slot, const T* row, int V, int unit,
                                                   int lane) {
        alignas(16) T v[kLoads][VEC];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int c = column(unit, j, lane) + e;
                v[j][e] = c < V ? row[c] : T(-INFINITY);
            }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) slot[j * 32] = *reinterpret_cast<const uint4*>(v[j]);
    }
    __device__ __forceinline__ static void copy16(uint4* to, const uint8_t* from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
                     : "memory");
    }
    __device__ __forceinline__ void read(const uint4* slot, int lane, int off) {
        if (off == 0) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint4 v = slot[j * 32 + lane];
                w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(slot + j * 32 + lane) + off / 4;
                if constexpr (sizeof(T) == 2) {
                    const uint32_t v[5] = {p[0], p[1], p[2], p[3], p[4]};
                    const int half = (off & 2) * 8;              // 0 or 16
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[4 * j + i] = __funnelshift_r(v[i], v[i + 1], half);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[4 * j + i] = p[i];
                }
            }
        }
    }
    __device__ __noinline__ static void load_edge(const T* row, int V, int c, uint32_t* to) {
        alignas(16) T v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = c + e < V ? row[c + e] : T(-INFINITY);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = p[i];
    }
    // the largest of 4 * loads words
    __device__ __forceinline__ static float largest(const uint32_t* w, int loads) {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(w);
            __nv_bfloat162 m = p[0];
#pragma unroll
            for (int i = 1; i < 4 * loads; ++i) m = __hmax2(m, p[i]);
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            float m = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < 4 * loads; ++i) m = fmaxf(m, __uint_as_float(w[i]));
            return m;
        }
    }
    // sum of 2^((x - m) k), pairs of columns at a time
    __device__ __forceinline__ float weight(float m, float k) const {
        const float mk = m * k;
        float2 sum = make_float2(0.f, 0.f);
        const float2 kk = make_float2(k, k);
        if (fabsf(mk) < 65536.f) {
            // one fma a column; what the product m k was rounded by (at most 2^-9) comes off the sum
            const float2 by = make_float2(-mk, -mk);
#pragma unroll
            for (int i = 0; i < WORDS / kWordsPair; ++i) {
                const float2 t = __ffma2_rn(pair(i), kk, by);
                sum = __fadd2_rn(sum, make_float2(ex2_approx(t.x), ex2_approx(t.y)));
            }
            return (sum.x + sum.y) * ex2_approx(-fmaf(m, k, -mk));
        }
        const float2 by = make_float2(-m, -m);
#pragma unroll 1
        for (int i = 0; i < WORDS; ++i) {
            float2 t = make_float2(0.f, -INFINITY);
            uint32_t word = w[0];
#pragma unroll
            for (int j = 1; j < WORDS; ++j) word = i == j ? w[j] : word;
            if constexpr (sizeof(T) == 2)
                t = make_float2(__uint_as_float(word << 16), __uint_as_float(word & 0xffff0000u));
            else
                t.x = __uint_as_float(word);
            t = __fmul2_rn(__fadd2_rn(t, by), kk);
            sum = __fadd2_rn(sum, make_float2(ex2_approx(t.x), ex2_approx(t.y)));
        }
        return sum.x + sum.y;
    }
    static constexpr int kWordsPair = sizeof(T) == 2 ? 1 : 2;
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 2)
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

// VEC consecutive columns from c < V on; -inf past the row's end.  A row that does not start on 16
// bytes is read by words: each holds an element of the row.
template <typename T, bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const T* row, int V, int c) {
    uint32_t w[5];
    if (c + Unit<T>::VEC > V) {
        Unit<T>::load_edge(row, V, c, w);
    } else if (ALIGNED) {
        return __ldg(reinterpret_cast<const uint4*>(row + c));
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
        const uint32_t* p = reinterpret_cast<const uint32_t*>(at & ~uintptr_t(3));
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __ldg(p + i);
        if (sizeof(T) == 2 && (at & 2) != 0) {
            w[4] = __ldg(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ float piece_value(const uint4& v, int e) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&v);
    if (sizeof(T) == 4) return __uint_as_float(p[e]);
    return __uint_as_float((e & 1) ? (p[e / 2] & 0xffff0000u) : (p[e / 2] << 16));
}

// What a stream leaves: its maximum and the sum of its weights.
struct Stream {
    float m, s;
};

// Behind it the list.  While the row is read the warps' rings take the place of both.
struct Shared {
    alignas(16) uint32_t hist[kBins];
    uint16_t queue[kQueue];
    alignas(4) uint8_t bits[kPieces + 4];
    uint32_t warp_n[32], warp_low[32];
    uint32_t n, queued;
    uint32_t bin, below, through;        // of the histogram: the bin K falls on, counts to it
};

// Elements the list holds: about K are found where segments are many, and never more than
// twice as many that a histogram would let through.
__host__ __device__ constexpr int list_size(int K) { return K <= 256 ? 1024 : kList; }

template <int THREADS>
__device__ __forceinline__ void clear_hist(Shared& sh) {
    uint4* h = reinterpret_cast<uint4*>(sh.hist);
    for (int b = threadIdx.x; b < kBins / 4; b += THREADS) h[b] = make_uint4(0, 0, 0, 0);
}

// Exclusive prefix of n over the block, and the total.
template <int THREADS>
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
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sh.warp_n[w];
        total += sh.warp_n[w];
    }
    return before + inc - n;
}

// The first bin at which the running count, `base` before the first, reaches `want`.
template <int THREADS>
__device__ __forceinline__ void find_bin(Shared& sh, int bins, uint32_t base, uint32_t want) {
    const int each = max(1, bins / THREADS);
    uint32_t own = 0;
    if (threadIdx.x * each < bins)
        for (int b = 0; b < each; ++b) own += sh.hist[threadIdx.x * each + b];
    uint32_t total;
    uint32_t run = base + block_prefix<THREADS>(own, sh, total);
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
// in on it.  `want` segments at least are above -inf; the histogram is 0 on entry.
template <int THREADS>
__device__ __noinline__ uint32_t segment_bound(const uint32_t* segkey, int nseg, uint32_t lo,
                                               uint32_t hi, uint32_t want, Shared& sh) {
    const uint32_t slack = max(32u, want / 4);
    uint32_t base = 0;
    while (true) {
        const int shift = max(0, 21 - __clz((hi - lo) | 1u));      // (hi - lo) >> shift < 2048
        for (int i = threadIdx.x * 4; i < nseg; i += THREADS * 4) {   // keys of 0 behind the last
            const uint4 v = *reinterpret_cast<const uint4*>(segkey + i);
            const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (key[e] >= lo && key[e] <= hi) atomicAdd(&sh.hist[(hi - key[e]) >> shift], 1u);
        }
        __syncthreads();
        find_bin<THREADS>(sh, kBins, base, want);
        const uint32_t bin = sh.bin, through = sh.through;
        base = sh.below;
        const u64 edge = (u64(bin) + 1) << shift;                  // keys of bins 0 .. bin
        const uint32_t bound = edge > u64(hi - lo) ? lo : hi - static_cast<uint32_t>(edge) + 1;
        if (through <= want + slack || shift == 0) return bound;
        hi -= bin << shift;
        lo = bound;
        clear_hist<THREADS>(sh);
        __syncthreads();
    }
}

__device__ __forceinline__ u64 element(uint32_t key, int col) {
    return (u64(key) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}

// The K largest of the row into the list, by the digits of their keys: for rows whose segments
// say too little.  Leaves sh.n; returns a key that all of them reach.
template <typename T, int THREADS>
__device__ __noinline__ uint32_t select_digits(const T* row, int V, uint32_t K, Shared& sh,
                                            u64* list) {
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t prefix = 0, above = 0;          // above: keys larger than the prefix's
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) sh.hist[tid] = 0;
        __syncthreads();
        for (int c0 = 0; c0 < V; c0 += THREADS) {
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
        find_bin<THREADS>(sh, 256, above, K);
        if (sh.through == 0) break;          // fewer than K above -inf (in the first step only)
        prefix = (prefix << 8) | (255 - sh.bin);
        above = sh.below;
        __syncthreads();
    }
    // everything above the K-th key, and of its equals the lowest columns
    const bool all = sh.through == 0;
    const uint32_t kth = all ? kKeyNegInf : prefix;
    uint32_t n = 0, ties = all ? 0 : K - above;
    for (int c0 = 0; c0 < V && n < K; c0 += THREADS) {
        const int c = c0 + tid;
        const uint32_t key = c < V ? order_key(to_f32(row[c])) : 0;
        uint32_t total_tie = 0, total;
        const uint32_t before = block_prefix<THREADS>(key == kth && !all ? 1 : 0, sh, total_tie);
        const bool take = key > kth || (!all && key == kth && before < ties);
        const uint32_t at = block_prefix<THREADS>(take ? 1 : 0, sh, total);
        if (take) list[n + at] = element(key, c);
        n += total;
        ties -= min(ties, total_tie);
    }
    __syncthreads();
    if (tid == 0) sh.n = n;
    __syncthreads();
    return all ? kKeyNegInf + 1 : kth;
}

// How the row is divided, and the shares of shared memory: where the segments' keys were, the
// list is put in order.
constexpr int kSlots = 2, kSlot = kLoads * 32 + 1;         // of a ring, and 16-byte pieces of one
constexpr size_t kListOff = (sizeof(Shared) + 15) / 16 * 16;
struct Plan {
    int units, streams, ranks, lanes, log_lanes, halves, nseg, list;
    size_t stream_off, seg_off, bytes;
};

// ALIGNED: all rows start on 16 bytes.
template <typename T, int THREADS, bool ALIGNED>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
    topk_kernel(const T* logits, const TopkArgs args, const Plan plan) {
    typedef Unit<T> U;
    constexpr int VEC = U::VEC;
    extern __shared__ uint4 smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    uint8_t* base = reinterpret_cast<uint8_t*>(smem);
    u64* list = reinterpret_cast<u64*>(base + kListOff);
    Stream* of_stream = reinterpret_cast<Stream*>(base + plan.stream_off);
    uint32_t* segkey = reinterpret_cast<uint32_t*>(base + plan.seg_off);
    TopkArgs a = args;
    const int units = plan.units, ranks = plan.ranks, nseg = plan.nseg, streams = plan.streams;
    const int row = blockIdx.x / ranks;
    const uint32_t rank = ranks > 1 ? cluster_ctarank() : 0u;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_previous(logits, a.mask);
    if (a.mask != nullptr && a.mask[row] == 0) {
        if (rank == 0) {
            for (int j = tid; j < a.K; j += THREADS) {
                a.ids[static_cast<int64_t>(row) * a.K + j] = -1;
                a.logp[static_cast<int64_t>(row) * a.K + j] = 0.f;
            }
            if (tid == 0 && a.lse != nullptr) a.lse[row] = 0.f;
        }
        return;
    }
    const T* x_row = logits + row * a.stride;
    // this warp's streams, one after the other, and its ring: units i, i + 1 on their way
    const int step = ranks * (THREADS / 32), last = min(streams, units);
    int stream = static_cast<int>(rank) * (THREADS / 32) + warp;
    int u = stream, ahead = stream, ahead_stream = stream;
    uint4* ring = smem + warp * kSlots * kSlot;
    const int off = ALIGNED ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(x_row) & 15);
    const auto fetch_next = [&](uint4* slot) {
        if (ahead_stream < last) {
            U::fetch(slot, x_row, a.V, ahead, lane, off);
            ahead += streams;
            if (ahead >= units) ahead = ahead_stream += step;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int q = 0; q < kSlots; ++q) fetch_next(ring + q * kSlot);
    Stream* to_stream = of_stream;
    uint32_t* to_seg = segkey;
    if (ranks > 1) {
        __syncwarp();
        cluster_sync();                          // the first block is there
        to_stream = peer(to_stream, 0);
        to_seg = peer(to_seg, 0);
    }
    int slot = 0;
    float m = -INFINITY, s = 0.f;
    while (stream < last) {
        U now;
        asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 1) : "memory");
        if (!ALIGNED) __syncwarp();              // the other lanes' copies too
        now.read(ring + slot * kSlot, lane, U::whole(a.V, u, off) ? off : 0);
        if (!ALIGNED) __syncwarp();              // read before it is written again
        fetch_next(ring + slot * kSlot);
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        const int at = u;
        const bool ends = u + streams >= units;
        const int to = ends ? stream + step : stream;
        u = ends ? to : u + streams;
        float mu;
        if (plan.halves == 2) {
            const float m0 = U::largest(now.w, kLoads / 2),
                        m1 = U::largest(now.w + 2 * kLoads, kLoads / 2);
            *reinterpret_cast<uint2*>(to_seg + (at * 32 + lane) * 2) =
                make_uint2(order_key(m0), order_key(m1));
            mu = fmaxf(m0, m1);
        } else {
            mu = U::largest(now.w, kLoads);
            float g = mu;
            for (int off = 1; off < plan.lanes; off <<= 1)
                g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, off));
            if (lane % plan.lanes == 0) to_seg[(at * 32 + lane) >> plan.log_lanes] = order_key(g);
        }
        // the lane's running maximum and sum; 0 stands in for a maximum of -inf
        const float nm = fmaxf(m, mu), ref = nm == -INFINITY ? 0.f : nm;
        s = fmaf(s, ex2_approx((m - ref) * a.k), now.weight(ref, a.k));
        m = nm;
        if (ends) {
            const float top = warp_max(m), at_top = top == -INFINITY ? 0.f : top;
            s = warp_sum(s * (m == -INFINITY ? 1.f : ex2_approx((m - at_top) * a.k)));
            if (lane == 0) to_stream[stream] = Stream{top, s};
            m = -INFINITY, s = 0.f;
            stream = to;
        }
    }
    if (rank == 0) {
        if (tid < 4 && (nseg & ~3) + tid >= nseg && nseg % 4 != 0) segkey[(nseg & ~3) + tid] = 0;
    }
    if (ranks > 1) {
        __syncwarp();
        cluster_sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    clear_hist<THREADS>(sh);
    if (tid == 0) sh.n = sh.queued = 0;

    // the row's maximum and sum, each warp for itself, in one order; the least of the segments' keys
    // above -inf, and how many there are
    for (int i = lane; i < last; i += 32) m = fmaxf(m, of_stream[i].m);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    for (int i = lane; i < last; i += 32) {
        const Stream p = of_stream[i];
        s = fmaf(p.s, p.m == -INFINITY ? 1.f : ex2_approx((p.m - ref) * a.k), s);
    }
    s = warp_sum(s);
    uint32_t low = ~0u, count = 0;
    for (int i = tid * 4; i < nseg; i += THREADS * 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(segkey + i);
        const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (key[e] > kKeyNegInf) low = min(low, key[e]), ++count;
    }
    low = __reduce_min_sync(0xffffffffu, low);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) sh.warp_n[warp] = count, sh.warp_low[warp] = low;
    const uint32_t K = static_cast<uint32_t>(a.K);
    int64_t* ids = a.ids + static_cast<int64_t>(row) * a.K;
    float* logp = a.logp + static_cast<int64_t>(row) * a.K;
    if (!(s > 0.f && s < INFINITY && fabsf(m) < INFINITY)) {
        for (int j = tid; j < a.K; j += THREADS) {
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

    // the segments that reach the bound, then their elements
    __syncthreads();
    count = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) count += sh.warp_n[w], low = min(low, sh.warp_low[w]);
    uint32_t bound = kKeyNegInf + 1;
    if (count >= K) bound = segment_bound<THREADS>(segkey, nseg, low, order_key(m), K, sh);
    for (int i = tid * 4; i < nseg; i += THREADS * 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(segkey + i);
        const uint32_t key[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (key[e] >= bound) {
                const uint32_t at = atomicAdd(&sh.queued, 1u);
                if (at < kQueue) sh.queue[at] = static_cast<uint16_t>(i + e);
            }
    }
    __syncthreads();
    const uint32_t queued = sh.queued;
    // pieces of 16 bytes of a segment: 2, 4, 8 .. 128
    const int log_pieces = (plan.halves == 2 ? 1 : 2) + plan.log_lanes;
    const auto piece_column = [&](int i) {
        const int g = sh.queue[i >> log_pieces], p = i & ((1 << log_pieces) - 1);
        if (plan.halves == 2)
            return U::column(g >> 6, (g & 1) * (kLoads / 2) + p, (g & 63) >> 1);
        const int first = g << plan.log_lanes;   // unit * 32 + its first lane
        return U::column(first >> 5, p >> plan.log_lanes, (first & 31) + (p & (plan.lanes - 1)));
    };
    uint32_t* columns = segkey;                  // read until here
    uint32_t n = kList + 1;
    if (queued <= kQueue) {
        // as many segments at a time as there is room for their pieces: all of them up to V = 163840
        // fp32 and 327680 bf16, 64 at V = 2^22 (a search by digits instead, K = 1024 of [16, 262144]
        // fp32: 1307 us)
        const uint32_t room = kPieces >> log_pieces;
        const float least = key_value(bound);    // x >= least where its key reaches the bound
        n = 0;
        for (uint32_t q0 = 0; q0 < queued && n <= static_cast<uint32_t>(plan.list); q0 += room) {
            if (q0 > 0) __syncthreads();         // the bits are read until here
            // which columns of each piece reach the bound, a bit each
            const int first = static_cast<int>(q0) << log_pieces;
            const int pieces = static_cast<int>(min(room, queued - q0)) << log_pieces;
            constexpr int kAhead = 4;
            for (int i0 = tid; i0 < pieces; i0 += kAhead * THREADS) {
                uint4 v[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const int i = i0 + q * THREADS, c = i < pieces ? piece_column(first + i) : a.V;
                    // past the row: NaN, which reaches nothing
                    v[q] = make_uint4(~0u, ~0u, ~0u, ~0u);
                    if (c < a.V) v[q] = load_piece<T, ALIGNED>(x_row, a.V, c);
                }
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    uint32_t bits = 0;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        bits |= piece_value<T>(v[q], e) >= least ? 1u << e : 0u;
                    if (i0 + q * THREADS < pieces)
                        sh.bits[i0 + q * THREADS] = static_cast<uint8_t>(bits);
                }
            }
            if (tid < 3) sh.bits[pieces + tid] = 0;
            __syncthreads();
            // the columns, in the pieces' order: four pieces at a time
            const uint32_t* bits4 = reinterpret_cast<const uint32_t*>(sh.bits);
            const int words = (pieces + 3) / 4, each = (words + THREADS - 1) / THREADS;
            const int w0 = min(words, tid * each), w1 = min(words, w0 + each);
            uint32_t own = 0, found;
            for (int w = w0; w < w1; ++w) own += __popc(bits4[w]);
            uint32_t at = n + block_prefix<THREADS>(own, sh, found);
            n += found;
            if (n <= static_cast<uint32_t>(plan.list))
                for (int w = w0; w < w1; ++w)
                    for (uint32_t b = bits4[w]; b != 0; b &= b - 1) {
                        const int bit = __ffs(b) - 1;
                        columns[at++] = piece_column(first + 4 * w + bit / 8) + bit % 8;
                    }
        }
    }
    clear_hist<THREADS>(sh);
    __syncthreads();
    const bool searched = n > static_cast<uint32_t>(plan.list);
    if (searched) {
        bound = select_digits<T, THREADS>(x_row, a.V, K, sh, list);
        n = sh.n;
        clear_hist<THREADS>(sh);
        __syncthreads();
    }

    // in order: bins of the key from the largest on, then among the few of a bin
    const uint32_t top = order_key(m);
    const int shift = max(0, 21 - __clz((top - bound) | 1u));
    constexpr int kEach = 2048 / THREADS;
    uint32_t arrived[kEach];
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        if (q * THREADS >= n) break;
        const uint32_t i = tid + q * THREADS;
        if (i < n) {
            if (!searched) {
                const int c = static_cast<int>(columns[i]);
                list[i] = element(order_key(to_f32(x_row[c])), c);
            }
            arrived[q] = atomicAdd(&sh.hist[(top - static_cast<uint32_t>(list[i] >> 32)) >> shift], 1u);
        }
    }
    __syncthreads();
    {
        uint32_t own[kBins / THREADS], sum = 0, all;
#pragma unroll
        for (int b = 0; b < kBins / THREADS; ++b) {
            own[b] = sh.hist[tid * (kBins / THREADS) + b];
            sum += own[b];
        }
        uint32_t run = block_prefix<THREADS>(sum, sh, all);
#pragma unroll
        for (int b = 0; b < kBins / THREADS; ++b) {
            sh.hist[tid * (kBins / THREADS) + b] = run;
            run += own[b];
        }
    }
    __syncthreads();
    u64* ordered = reinterpret_cast<u64*>(segkey);
#pragma unroll
    for (int q = 0; q < kEach; ++q) {
        if (q * THREADS >= n) break;
        const uint32_t i = tid + q * THREADS;
        if (i < n) {
            const u64 el = list[i];
            ordered[sh.hist[(top - static_cast<uint32_t>(el >> 32)) >> shift] + arrived[q]] = el;
        }
    }
    __syncthreads();
    for (uint32_t i = tid; i < n; i += THREADS) {
        const u64 el = ordered[i];
        const uint32_t key = static_cast<uint32_t>(el >> 32), bin = (top - key) >> shift;
        const int from = static_cast<int>(sh.hist[bin]);
        const int end = bin + 1 < kBins ? static_cast<int>(sh.hist[bin + 1]) : static_cast<int>(n);
        if (from >= a.K) continue;
        int place = from;
        for (int j = from; j < end; ++j) place += ordered[j] > el;
        if (place >= a.K) continue;
        ids[place] = static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(el));
        logp[place] = fmaf(key_value(key) - m, a.inv_t, -ln_s);
    }
    for (int j = static_cast<int>(n) + tid; j < a.K; j += THREADS) {
        ids[j] = -1;
        logp[j] = -INFINITY;
    }
}

template <typename T, int THREADS, bool ALIGNED>
cudaError_t launch_threads(const T* logits, const TopkArgs& a, const Plan& p,
                           cudaStream_t stream) {
    constexpr size_t kMost = 112 * 1024;     // of any vocabulary
    static_assert(std::max(kListOff + 2048 * 8, size_t(THREADS / 32) * kSlots * kSlot * 16) +
                          kMaxStreams * sizeof(Stream) + kMaxSegments * 4 <= kMost,
                  "a block's shared memory");
    if (p.bytes > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(reinterpret_cast<const void*>(topk_kernel<T, THREADS, ALIGNED>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMost));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = p.ranks;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    return launch_early(topk_kernel<T, THREADS, ALIGNED>, dim3(static_cast<unsigned>(a.N) * p.ranks),
                        THREADS, p.bytes, stream, &cluster, logits, a, p);
}

template <typename T>
cudaError_t launch_typed(const T* logits, const TopkArgs& a, cudaStream_t stream) {
    Plan p{};
    p.units = (a.V + Unit<T>::kColumns - 1) / Unit<T>::kColumns;
    p.streams = p.units >= 256 ? 128 : 64;
    p.lanes = p.halves = 1;
    if (p.units * 32 < 4 * a.K) p.halves = 2;
    // 32 segments and more for each element that is looked for leave few others among the K
    // largest of their maxima; more of them cost more than they save (K = 64 of [2048, 151936] bf16:
    // 4768 segments 131 us, 2384 of them 125, 1192 126).
    while (p.units * 32 * p.halves / p.lanes > kMaxSegments ||
           (p.halves == 1 && p.lanes < 32 &&
            p.units * 32 / (2 * p.lanes) >= std::max(1024, 32 * a.K)))
        p.lanes *= 2, ++p.log_lanes;
    p.nseg = p.units * 32 * p.halves / p.lanes;
    p.list = list_size(a.K);
    // 512 threads a block while two of them on each of 152 SMs hold all rows, with as many blocks
    // a row as that leaves; else four of 256 on an SM, a row each
    const int threads = a.N <= 304 ? 512 : 256;
    p.ranks = p.units >= 64 ? 8 : p.units >= 32 ? 4 : p.units >= 16 ? 2 : 1;
    while (p.ranks > 1 && static_cast<int64_t>(a.N) * p.ranks > (threads == 512 ? 304 : 608))
        p.ranks /= 2;
    p.stream_off = std::max(kListOff + p.list * sizeof(u64), size_t(threads / 32) * kSlots * kSlot * 16);
    p.seg_off = p.stream_off + p.streams * sizeof(Stream);
    p.bytes = p.seg_off + std::max((p.nseg + 3) / 4 * 4 * sizeof(uint32_t), p.list * sizeof(u64));
    if (threads == 512)
        return a.vec_ok ? launch_threads<T, 512, true>(logits, a, p, stream)
                        : launch_threads<T, 512, false>(logits, a, p, stream);
    return a.vec_ok ? launch_threads<T, 256, true>(logits, a, p, stream)
                    : launch_threads<T, 256, false>(logits, a, p, stream);
}

}  // namespace

cudaError_t launch_topk(const void* logits, bool bf16, const TopkArgs& args, cudaStream_t stream) {
    if (bf16) return launch_typed(static_cast<const __nv_bfloat16*>(logits), args, stream);
    return launch_typed(static_cast<const float*>(logits), args, stream);
}

}  // namespace rlk
