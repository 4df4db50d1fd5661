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
// elements above a key, and the first `ties` in index order of those equal to it.  Nothing
// is sorted.  Sums that decide are integers (weight_exp.cuh), so the token depends on the
// row alone: not on the batch, on how the row is split, or on the alignment.
//
// Two launches.  The scan: up to 8 blocks a row (a cluster), a warp a chunk of 512 columns;
// per chunk its maximum and an fp32 sum of 2^((x - chunk max) c), c = log2(e)/T, and with
// truncation the maxima of its segments of 128 or 256 columns, go to the workspace.  This is
// the only pass over HBM.  One block of the cluster then forms the chunks' weights as
// integers, in the same order whatever the split, and finishes the rows that need no further
// pass over all columns:
//
//   no truncation: the chunk and the element that u times the total falls on come from the
//   fast weights, together with a bound on their error (kFastErr); only when the target lies
//   within it of a border of the running sums -- one row in twenty at V ~ 150k -- is the row
//   left open.
//
//   truncation: elements from some value on are gathered from the segments whose maximum
//   reaches it, and their order is counted out.  The value is one that top_k segment maxima
//   reach, that segment maxima of top_p of the total reach, or min_p's own; in rows in no
//   particular order few other elements reach it.
//
// The second launch takes the rows that are left.  Without truncation they are weighed
// exactly.  With it (a wide nucleus, a large top_k, a row sorted by token) they are searched:
// histograms of 2048 bins of the scaled distance from the maximum, then of the keys inside
// the remaining window (with the weights as integers, so each leaves one bin of it), close in on
// the boundary until its window fits a list or is a single value.  One block of the cluster decides each step; the blocks work on their own chunks in
// between.
//
// Measured at V = 151936, fp32 (HBM's floor in brackets): one row 10.7 us; [256] 54 us (23),
// of which the scan takes 33 and the rows weighed exactly 17; [64] with top_k = 50 and top_p
// 24 us (5.7); [1024] 141 us (92).  A row with a wide nucleus takes 56 us by itself, 256 of
// them 420 us: 168 instructions an element in all, and block 0's decisions, for which the
// other blocks wait, bind the search, not memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstddef>

#include "ptx.cuh"
#include "rlk_internal.h"
#include "weight_exp.cuh"

namespace rlk {

namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;            // of a scan block
constexpr int kWarps = kThreads / 32;
constexpr int kSearch = 512;             // of a search block
constexpr int kExact = 1024;             // of a block that weighs rows exactly
constexpr int kChunk = 512;              // columns of a chunk
constexpr int kLane = kChunk / 32;       // of a lane
constexpr int kBins = 2048;
constexpr int kList = 1920;              // elements of the search's list
constexpr int kSelect = 1024;            // bins of the selection in it
constexpr int kShort = 1024;             // of the scan's list
constexpr int kMaxSegments = 8192;       // of a row whose truncation the scan tries itself
constexpr int kMaxShortK = 700;          // and its top_k, with finer segments
constexpr float kRange = 48.f;           // weights below 2^-47 round to 0 (bits <= 46)
constexpr int kMaxSteps = 32;            // far more than any row takes
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf)

// The fast weights' relative error, in units of 2^-24: 4 for ex2.approx, 9 roundings of a
// chunk's sum, and log(2) t_i (1 for x - max, 1 for its product with c) for each element: the
// weighted mean of t over 512 elements with sum s >= 1 is at most log2(512 / s) <= 9, so 12.5.
// A relative error e of all weights leaves 2 u (1 - u) e of sum(prefix) - u sum(all) at its
// zero.  The prefix inside a chunk is summed exactly: there up to kSumErr of the chunk's weight
// comes on top, and whole units: half a unit of a chunk's largest weight, 512 times, and one for
// each product, are below one for each column (kFastUnits for the columns past V).
constexpr float kFastErr = 26.f / 16777216.f;
constexpr float kSumErr = 9.f / 16777216.f;
constexpr u64 kFastUnits = 8192;
// Of the weight of a histogram of the distance: 12-bit codes relative to the weight at the bin's
// start, in bins of 0.023 powers of 2 (half a code of 4030, and 2^-17 for distance and exponential).
constexpr float kBinErr = 1.f / 4096.f;

// Unsigned integers in the order of the floats; -0 and +0 get the same one.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// floor (up = false) or ceiling of f s, 0 <= f < 1, f.shift >= 1
__device__ __noinline__ u64 part_of(SampleFraction f, u64 s, bool up) {
    const u64 lo = f.mant * s, hi = __umul64hi(f.mant, s);
    u64 r = 0;
    bool rest;
    if (f.shift < 64) {
        r = (hi << (64 - f.shift)) | (lo >> f.shift);
        rest = (lo << (64 - f.shift)) != 0;
    } else if (f.shift < 128) {
        const int t = f.shift - 64;
        r = hi >> t;
        rest = lo != 0 || (t > 0 && (hi << (64 - t)) != 0);
    } else {
        rest = (hi | lo) != 0;
    }
    return r + (up && rest ? 1 : 0);
}
// a float in [0, 1), exactly
__device__ __forceinline__ SampleFraction fraction(float f) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    SampleFraction r;
    r.mant = e == 0 ? b : (b & 0x7fffffu) | 0x800000u;
    r.shift = 150 - static_cast<int>(max(e, 1u));
    return r;
}
// floor(w f) of a float 0 <= w <= 512 and an integer f <= 2^46.  The product has up to 70 bits, of
// which the 14 that are always behind the point go first; bits cut off f instead would be much of
// the weight of a light chunk, whose f is small.
__device__ __forceinline__ u64 scale_weight(float w, u64 f) {
    const uint32_t b = __float_as_uint(w), mant = (b & 0x7fffffu) | 0x800000u;
    const u64 hi = u64(static_cast<uint32_t>(f >> 24)) * mant;
    const u64 lo = u64(static_cast<uint32_t>(f) & 0xffffffu) * mant;
    // w = mant 2^-(150 - e); what has no such mantissa is below 2^-126
    return ((hi << 10) + (lo >> 14)) >> min(136 - static_cast<int>(b >> 23), 63);
}

// the same shared object in block `rank` of the cluster (generic address)
template <typename P>
__device__ __forceinline__ P* peer(P* p, uint32_t rank) {
    u64 a;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
    return reinterpret_cast<P*>(a);
}

// cluster barrier of converged warps
__device__ __forceinline__ void cluster_join() {
    __syncwarp();
    cluster_sync();
}

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// maximum over the warp, by an integer reduction of order-preserving bits
__device__ __forceinline__ float warp_max(float v) {
    const int b = __float_as_int(v);
    const int k = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// Exclusive prefix of v and n over the block's threads, and the totals.  Not inlined, like
// the other serial parts of a row: they run once, and fetching their code is much of their
// time.
struct Scanned {
    u64 v, tv;
    uint32_t n, tn;
};
template <int THREADS>
__device__ __noinline__ Scanned block_scan(u64 v, uint32_t n, u64* part, uint32_t* part_n) {
    constexpr int kParts = THREADS / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 iv = v;
    uint32_t in = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const u64 ov = __shfl_up_sync(0xffffffffu, iv, off);
        const uint32_t on = __shfl_up_sync(0xffffffffu, in, off);
        if (lane >= off) iv += ov, in += on;
    }
    __syncthreads();
    if (lane == 31) part[warp] = iv, part_n[warp] = in;
    __syncthreads();
    // every warp scans the warps' sums for itself
    u64 pv = lane < kParts ? part[lane] : 0;
    uint32_t pn = lane < kParts ? part_n[lane] : 0;
#pragma unroll
    for (int off = 1; off < kParts; off <<= 1) {
        const u64 ov = __shfl_up_sync(0xffffffffu, pv, off);
        const uint32_t on = __shfl_up_sync(0xffffffffu, pn, off);
        if (lane >= off) pv += ov, pn += on;
    }
    Scanned r;
    r.tv = __shfl_sync(0xffffffffu, pv, kParts - 1);
    r.tn = __shfl_sync(0xffffffffu, pn, kParts - 1);
    const u64 bv = __shfl_sync(0xffffffffu, pv, warp - 1);
    const uint32_t bn = __shfl_sync(0xffffffffu, pn, warp - 1);
    r.v = (warp == 0 ? 0 : bv) + iv - v;
    r.n = (warp == 0 ? 0 : bn) + in - n;
    return r;
}

// ----------------------------------------------------------------------------- rows

// 16 bytes of a row from column c on, -inf past its end.  Not inlined where they come one by
// one: there are many such loads in code that is better short.
template <typename T>
__device__ __noinline__ uint4 load_single(const T* row, int V, int c) {
    constexpr int VEC = 16 / sizeof(T);
    alignas(16) T v[VEC];                // read as one
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = c + e < V ? row[c + e] : T(-INFINITY);
    return *reinterpret_cast<const uint4*>(v);
}
template <typename T>
__device__ __forceinline__ uint4 load_group(const T* row, int V, int c, bool vec) {
    constexpr int VEC = 16 / sizeof(T);
    if (vec && c + VEC <= V) return __ldg(reinterpret_cast<const uint4*>(row + c));
    return load_single(row, V, c);
}
template <typename T>
__device__ __forceinline__ float group_value(const uint4& g, int i) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&g);
    if (sizeof(T) == 4) return __uint_as_float(p[i]);
    return __uint_as_float((i & 1) ? (p[i / 2] & 0xffff0000u) : (p[i / 2] << 16));
}

// The 16 columns that a lane holds of a chunk, as they lie in memory: LOADS groups of VEC
// consecutive ones, group j of lane l at column (32 j + l) VEC of the chunk.
template <typename T>
struct Chunk {
    static constexpr int VEC = 16 / sizeof(T);
    static constexpr int LOADS = kLane / VEC;
    uint4 raw[LOADS];

    __device__ __forceinline__ static int column(int chunk, int j, int lane) {
        return chunk * kChunk + (j * 32 + lane) * VEC;
    }
    __device__ __forceinline__ void load(const T* row, int V, int chunk, int lane, bool vec) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) raw[j] = load_group(row, V, column(chunk, j, lane), vec);
    }
    // Four elements at a time, for loops whose code is better short: the first four, and the
    // others moved up.
    static constexpr int kQuads = kLane / 4;
    __device__ __forceinline__ void take(float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = get(e);
        uint32_t* p = reinterpret_cast<uint32_t*>(raw);
        constexpr int kWords = LOADS * 4, kStep = kWords / kQuads;
#pragma unroll
        for (int w = 0; w + kStep < kWords; ++w) p[w] = p[w + kStep];
    }
    __device__ __forceinline__ float get(int i) const {
        return group_value<T>(raw[i / VEC], i % VEC);
    }
};

// A warp's part of a ring of chunks in shared memory, on their way while another is worked on.
// Each lane copies just what it reads itself, so this needs no barrier: group j of slot s lies
// at (LOADS s + j) 32 + lane.  Two chunks of fp32: with three, an SM holds three blocks instead of
// four (67 instead of 54 us at [256, 151936]).
constexpr int kRing = 4096;              // bytes of a warp
template <typename T>
struct Ring {
    static constexpr int LOADS = Chunk<T>::LOADS, VEC = Chunk<T>::VEC;
    static constexpr int S = kRing / (kChunk * int(sizeof(T)));
    uint4* lane_base;

    __device__ __forceinline__ void fetch(int slot, const T* row, int V, int chunk, int lane,
                                          bool vec) const {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            uint4* to = lane_base + (slot * LOADS + j) * 32;
            const int c = Chunk<T>::column(chunk, j, lane);
            if (vec && c + VEC <= V) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)),
                             "l"(row + c)
                             : "memory");
            } else if (sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (c + e < V)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                         smem_u32(to) + 4 * e),
                                     "l"(row + c + e)
                                     : "memory");
                    else
                        reinterpret_cast<float*>(to)[e] = -INFINITY;
            } else {
                *to = load_group(row, V, c, false);
            }
        }
    }
    __device__ __forceinline__ void read(int slot, Chunk<T>& c) const {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) c.raw[j] = lane_base[(slot * LOADS + j) * 32];
    }
};
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest LEFT groups have arrived
template <int LEFT>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// A row's settings, from the scalars or its own.
struct Settings {
    float ch, cl;              // log2(e) / T in two floats
    SampleFraction u, top_p;
    float u_value, p_value;
    int64_t top_k;             // 0: off
    bool want_k, want_p, want_m, ok;
};
__device__ __forceinline__ Settings read_settings(const SampleArgs& a, int64_t row) {
    Settings s;
    s.ok = true;
    s.ch = a.ch;
    s.cl = a.cl;
    if (a.temperature_rows != nullptr) {
        const float t = a.temperature_rows[row];
        s.ok = t >= static_cast<float>(kSampleMinT) && t <= static_cast<float>(kSampleMaxT);
        constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596299e-8f;
        s.ch = __fdiv_rn(kLog2eHi, t);
        s.cl = (fmaf(-s.ch, t, kLog2eHi) + kLog2eLo) / t;
    }
    s.top_k = a.top_k_rows != nullptr ? a.top_k_rows[row] : a.top_k;
    s.ok = s.ok && s.top_k >= 0;
    s.want_k = s.top_k > 0 && s.top_k < a.V;
    s.top_p = a.top_p;
    s.p_value = a.top_p_value;
    if (a.top_p_rows != nullptr) {
        s.p_value = a.top_p_rows[row];
        s.ok = s.ok && s.p_value > 0.f;
        s.top_p = fraction(s.p_value);
    }
    s.want_p = s.p_value < 1.f;
    float m = a.min_p_value;
    if (a.min_p_rows != nullptr) {
        m = a.min_p_rows[row];
        s.ok = s.ok && m >= 0.f && m <= 1.f;
    }
    s.want_m = m > 0.f;
    s.u_value = a.uniforms[row];
    s.ok = s.ok && s.u_value >= 0.f && s.u_value < 1.f;
    s.u = fraction(s.u_value);
    return s;
}

// The key of the smallest float x with x >= m + T log(min_p).  fp64 arithmetic, at 1/64 of
// the rate of fp32's: called by one thread, and only with min_p on.
__device__ __noinline__ uint32_t min_p_key(const SampleArgs& a, int64_t row, float m) {
    double off = a.min_p_offset;
    if (a.temperature_rows != nullptr || a.min_p_rows != nullptr) {
        const double t = a.temperature_rows != nullptr ? a.temperature_rows[row] : a.temperature;
        off = t * log(a.min_p_rows != nullptr ? static_cast<double>(a.min_p_rows[row]) : a.min_p);
    }
    const double at = static_cast<double>(m) + off;
    const float f = static_cast<float>(at);
    return order_key(f) + (static_cast<double>(f) < at ? 1u : 0u);
}

template <typename T>
struct Row {
    const T* x;
    int V, nch, own, first, mine;        // chunks: all, a block's share, this block's
    bool vec;
    WeightScale ws;
    float scale;                         // bins per unit of distance
    int bits;
};
template <typename T>
__device__ __forceinline__ Row<T> make_row(const T* logits, const SampleArgs& a, int64_t row,
                                           const Settings& s, int nch, int own, int rank) {
    Row<T> r;
    r.x = logits + row * a.stride;
    r.V = a.V;
    r.nch = nch;
    r.own = own;
    r.first = rank * own;
    r.mine = max(0, min(own, nch - r.first));
    r.vec = a.vec_ok;
    r.bits = a.bits;
    r.ws.m = 0.f;
    r.ws.ch = s.ch;
    r.ws.cl = s.cl;
    r.ws.shift = 62 - a.bits;
    r.scale = s.ch * (kBins / kRange);
    return r;
}

// bounds of the exact total from the fast one; half a unit of each exact weight's own on top
__device__ __forceinline__ void total_bounds(u64 all, int V, u64& lo, u64& hi) {
    const u64 err =
        static_cast<u64>(static_cast<float>(all) * (kFastErr + 1.5e-11f)) + 2 * V + kFastUnits;
    lo = all > err ? all - err : 1;
    hi = all + err;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

__device__ __noinline__ void write_row(const SampleArgs& a, int64_t row, int64_t token, float logp,
                                       float kept_logp) {
    a.tokens[row] = token;
    if (a.logp != nullptr) a.logp[row] = logp;
    if (a.kept_logp != nullptr) a.kept_logp[row] = kept_logp;
}

// a row without a result, by one thread
__device__ __forceinline__ void write_failed(const SampleArgs& a, int64_t row, uint32_t bit) {
    write_row(a, row, -1, quiet_nan(), quiet_nan());
    if (a.err != nullptr) atomicOr(a.err, bit);
}

// logp = -t log 2 - log(sum), by one thread.  Sums are scaled by 2^bits, which is the
// largest weight: what is left after it goes to log1p, so a logp near 0 keeps its digits.
__device__ __noinline__ void write_drawn(const SampleArgs& a, int64_t row, int v, float x,
                                         WeightScale ws, u64 all, u64 kept) {
    float th, tl;
    scaled_distance(x, ws, th, tl);
    constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;
    const float zh = th * kLn2Hi;
    const float zl = fmaf(th, kLn2Hi, -zh) + fmaf(th, kLn2Lo, tl * kLn2Hi);
    const u64 one = u64(1) << (62 - ws.shift);
    const float unit = __uint_as_float(uint32_t(127 - (62 - ws.shift)) << 23);
    float logs[2];
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        logs[i] = -((zh + log1pf(static_cast<float>((i == 0 ? all : kept) - one) * unit)) + zl);
    write_row(a, row, v, logs[0], logs[1]);
}

// ----------------------------------------------------------------------------- scan

// Shared memory of the scan.
struct Shared0 {
    u64 table[kExpEntries];
    u64 part[kWarps];
    uint32_t part_n[kWarps];
    u64 at_w;
    uint32_t n_list, n_ids, flag, key_m;
    int at;
    // from here on first the ring of the pass over the row
    __align__(16) u64 order[kShort];     // the list, then sorted
    u64 w[kShort];
};

// Workspace: a header a row, whether the row goes on to the search, the chunks' maxima and
// sums, the segments' maxima (room for them as if logits were fp32).
enum : uint32_t { kRowDone, kRowSearch };
struct RowHeader {
    u64 all;                             // fast total of the weights
    float m;                             // maximum
};
__host__ __device__ constexpr size_t modes_offset(int64_t N) {
    return (size_t(N) * sizeof(RowHeader) + 255) / 256 * 256;
}
// Segments of a row: parts of a chunk each.  What one load of the warp covers (parts 0: one
// reduction gives their maximum), or, where top_k is more than half their number, what 32 / parts
// neighbouring lanes hold, with parts the power of two that makes twice top_k of them.  So the
// list has up to 1.4 top_k elements in rows in no particular order ([196, 32660] bf16 with top_k
// 279: 44 us, 97 with a search for each row; [64, 151936] fp32 with 600: 61 and 100).  Finer
// segments for all calls cost time ([256, 151936] bf16 with top_k 50 and top_p: 46.5 instead of
// 41.5 us with 32 parts).
__host__ __device__ constexpr int segments_of(int nch, int parts, size_t esize) {
    const int64_t n = int64_t(nch) * (parts > 0 ? parts : esize == 4 ? 4 : 2);
    return n <= kMaxSegments ? static_cast<int>(n) : 0;
}
int parts_of(int nch, int64_t top_k, size_t esize) {
    const int n = segments_of(nch, 0, esize);
    if (n == 0 || top_k <= n / 2 || top_k > kMaxShortK) return 0;
    int parts = esize == 4 ? 8 : 4;
    while (parts < 32 && int64_t(nch) * parts < 2 * top_k) parts *= 2;
    return parts;
}
// Floats between two rows' maxima of segments, a multiple of 4: one a load, or fewer than 4
// kMaxShortK parts (parts_of doubles them only below 2 top_k).
__host__ __device__ constexpr int64_t segs_stride(int64_t nch) {
    const int64_t most = nch * 4 > 4 * kMaxShortK ? nch * 4 : 4 * kMaxShortK;
    return ((nch * 32 < most ? nch * 32 : most) + 3) / 4 * 4;
}
__host__ __device__ constexpr size_t stats_offset(int64_t N) {
    return (modes_offset(N) + size_t(N) * sizeof(uint32_t) + 255) / 256 * 256;
}
__host__ __device__ constexpr size_t segs_offset(int64_t N, int nch) {
    return (stats_offset(N) + size_t(N) * nch * sizeof(float2) + 255) / 256 * 256;
}
__device__ __forceinline__ uint32_t* row_modes(const SampleArgs& a) {
    return reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.workspace) + modes_offset(a.N));
}
__device__ __forceinline__ float2* row_stats(const SampleArgs& a, int64_t row, int nch) {
    return reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) + stats_offset(a.N)) +
           row * nch;
}
__device__ __forceinline__ float* row_segs(const SampleArgs& a, int64_t row, int nch) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + segs_offset(a.N, nch)) +
           row * segs_stride(nch);
}

// log2(e) / T in two positive floats: a distance of -inf then stays one, where a negative or zero
// second part would make it NaN.
__device__ __forceinline__ float2 fast_scale(const Settings& s) {
    const float below = __int_as_float(__float_as_int(s.ch) - 1);
    return s.cl > 0.f ? make_float2(s.ch, s.cl) : make_float2(below, s.cl + (s.ch - below));
}

// Maximum and sum of a chunk.  The sum of 2^((x - max) c) leaves out one element of the maximum
// (and has its sign bit set) where no other lane comes within an eighth of that one's weight: a
// total is a sum of such parts plus those maxima's own weights, so a logp near 0 keeps its digits.
// (Elsewhere the sum is 9/8 or more, and what lies above 1 is off by 9 times its relative error at
// most.)  This follows from the chunk alone, so a total, and the logp from it, do not depend on how
// many blocks share a row.  Taking out every chunk's maximum costs more: [1024, 151936] bf16 with
// top_k 50 and top_p takes 108 us with a quarter, 106 with an eighth.
// ml: the lane's maximum; seg (GROUPS): the maxima of the warp's loads.
template <bool GROUPS, typename T>
__device__ __forceinline__ float2 chunk_stats(const Chunk<T>& c, float2 scale,
                                              float (&seg)[Chunk<T>::LOADS], float& ml) {
    constexpr int VEC = Chunk<T>::VEC, LOADS = Chunk<T>::LOADS;
    ml = -INFINITY;
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
        float v = c.get(j * VEC);
#pragma unroll
        for (int e = 1; e < VEC; ++e) v = fmaxf(v, c.get(j * VEC + e));
        ml = fmaxf(ml, v);
        if (GROUPS) m = fmaxf(m, seg[j] = warp_max(v));
    }
    if (!GROUPS) m = warp_max(ml);
    // a chunk of -inf has sum 0; NaN or +inf make it NaN
    const float mm = fmaxf(m, -3.402823466e38f);
    float2 s[kLane / 2];
#pragma unroll
    for (int e = 0; e < kLane / 2; ++e) {
        const float2 d = __fadd2_rn(make_float2(c.get(2 * e), c.get(2 * e + 1)),
                                    make_float2(-mm, -mm));
        const float2 t = __ffma2_rn(d, make_float2(scale.x, scale.x),
                                    __fmul2_rn(d, make_float2(scale.y, scale.y)));
        s[e] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
    }
    // the lanes near the maximum, its own among them; with NaN and infinities the sum is NaN or 0
    const uint32_t near = __ballot_sync(0xffffffffu, (ml - m) * scale.x >= -3.f);
    const bool apart = near != 0 && (near & (near - 1)) == 0;
    if (apart) {
        bool lead = near >> (threadIdx.x & 31) & 1u;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            float& w = e % 2 == 0 ? s[e / 2].x : s[e / 2].y;
            const bool hit = lead && c.get(e) == m;
            w = hit ? 0.f : w;
            lead = lead && !hit;
        }
    }
#pragma unroll
    for (int w = kLane / 4; w > 0; w >>= 1)
#pragma unroll
        for (int e = 0; e < w; ++e) s[e] = __fadd2_rn(s[e], s[e + w]);
    const float sum = warp_sum(s[0].x + s[0].y);
    return make_float2(m, apart ? -sum : sum);
}

// The draw without truncation from the fast weights; false where their error leaves the
// token open.
template <typename T>
__device__ bool fast_draw(const Row<T>& r, const float* cmax, const u64* cw, u64 all,
                          const Settings& s, const SampleArgs& a, int64_t row_i, Shared0& sh) {
    const int tid = threadIdx.x;
    const u64 target = part_of(s.u, all, false);
    const int each = (r.nch + kThreads - 1) / kThreads;
    const int c0 = min(r.nch, tid * each), c1 = min(r.nch, c0 + each);
    u64 w = 0;
    for (int c = c0; c < c1; ++c) w += cw[c];
    w = block_scan<kThreads>(w, 0, sh.part, sh.part_n).v;
    if (tid == 0) sh.flag = 0, sh.at = 0, sh.at_w = 0;
    __syncthreads();
    for (int c = c0; c < c1; ++c) {
        if (w <= target && target < w + cw[c]) sh.at = c, sh.at_w = w;
        w += cw[c];
    }
    __syncthreads();
    // the chunk's columns in order, two a thread
    const int chunk = sh.at, col = chunk * kChunk + 2 * tid;
    const float x0 = col < r.V ? load_one(r.x + col) : -INFINITY;
    const float x1 = col + 1 < r.V ? load_one(r.x + col + 1) : -INFINITY;
    const float m = cmax[chunk];
    const u64 top = fixed_weight(m, r.ws, sh.table);
    const float2 scale = fast_scale(s);
    const float d0 = x0 - m, d1 = x1 - m;
    const u64 w0 = scale_weight(ex2_approx(fmaf(d0, scale.x, d0 * scale.y)), top);
    const u64 w1 = scale_weight(ex2_approx(fmaf(d1, scale.x, d1 * scale.y)), top);
    const u64 lo = sh.at_w + block_scan<kThreads>(w0 + w1, 0, sh.part, sh.part_n).v;
    const u64 mid = lo + w0, hi = mid + w1;
    const float part = 2.f * s.u_value * (1.f - s.u_value) * kFastErr + 1.5e-11f;
    const u64 err = static_cast<u64>(static_cast<float>(all) * part) +
                    static_cast<u64>(static_cast<float>(cw[chunk]) * kSumErr) + r.V + kFastUnits;
    const bool hit0 = lo <= target && (lo == 0 || lo + err <= target) && target + err < mid;
    const bool hit1 = mid <= target && (mid == 0 || mid + err <= target) && target + err < hi;
    if (hit0 || hit1) {
        write_drawn(a, row_i, hit0 ? col : col + 1, hit0 ? x0 : x1, r.ws, all, all);
        sh.flag = 1;
    }
    __syncthreads();
    return sh.flag != 0;
}

// A value that enough segment maxima reach: at least `count` of them, or (need > 0) maxima of
// a weight of at least `need`.  Between the maximum and `low`, by bisection with a warp a
// trial: 3 rounds leave 1/729 of the range.  `low` itself if that is not enough, with
// found = false.
template <typename T>
__device__ float reach_value(const Row<T>& r, const float* smax, int nseg, int count, float need,
                             float low, bool& found, Shared0& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float hi = r.ws.m, lo = low;
    found = true;
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
        // warp w tries the (w + 1)-th of 9 parts below hi; the first round also tries low
        const float step = (hi - lo) * (1.f / (kWarps + 1));
        const float x = round == 0 && warp == kWarps - 1 ? low : hi - step * (warp + 1);
        int n = 0;
        float w = 0.f;
        if (need > 0.f) {
#pragma unroll 1
            for (int c = lane * 4; c < nseg; c += 128) {
                const float4 v = *reinterpret_cast<const float4*>(smax + c);
                w += v.x >= x ? ex2_approx((v.x - r.ws.m) * r.ws.ch) : 0.f;
                w += v.y >= x ? ex2_approx((v.y - r.ws.m) * r.ws.ch) : 0.f;
                w += v.z >= x ? ex2_approx((v.z - r.ws.m) * r.ws.ch) : 0.f;
                w += v.w >= x ? ex2_approx((v.w - r.ws.m) * r.ws.ch) : 0.f;
            }
        } else {
#pragma unroll 2
            for (int c = lane * 4; c < nseg; c += 128) {
                const float4 v = *reinterpret_cast<const float4*>(smax + c);
                n += (v.x >= x ? 1 : 0) + (v.y >= x ? 1 : 0) + (v.z >= x ? 1 : 0) +
                     (v.w >= x ? 1 : 0);
            }
        }
        const bool enough =
            need > 0.f ? warp_sum(w) >= need : __reduce_add_sync(0xffffffffu, n) >= count;
        __syncthreads();
        if (lane == 0) sh.part_n[warp] = enough ? 1u : 0u;
        __syncthreads();
        // the highest trial that is enough
        const unsigned who = __ballot_sync(0xffffffffu, lane < kWarps && sh.part_n[lane] != 0);
        const int first = who == 0 ? kWarps : __ffs(who) - 1;
        if (round == 0 && first >= kWarps - 1) {
            found = first < kWarps;
            if (!found) return low;
            hi = hi - step * (kWarps - 1);           // only low itself
            continue;
        }
        const float top = hi;
        if (first > 0) hi = top - step * first;
        if (first < kWarps) lo = top - step * (first + 1);
    }
    return lo;
}

// Sorts the first n <= kShort of (order, w) by descending order (all different): each element's
// place in its run is counted out by a thread, and its places in the other runs, sorted by then,
// are searched.  One run of all where they are few (to 512: 19.5 us instead of 22.5 for [16, 151936]
// with min_p 0.02), runs of 128 where they are many (68 instead of 102 us for [64, 151936] with top_k
// 700).  At these lengths that is quicker than a sorting network, whose steps each wait for the one
// before.  `order` is padded to a multiple of 4.
constexpr uint32_t kRun = 128;
template <bool RUNS>
__device__ __noinline__ void sort_by(uint32_t n, u64* order, u64* w) {
    constexpr int kPer = kShort / kThreads;
    const uint32_t padded = (n + 3) / 4 * 4;
    if (threadIdx.x < padded - n) order[n + threadIdx.x] = 0;
    __syncthreads();
    u64 me[kPer], mw[kPer];
    uint32_t place[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t i = threadIdx.x + q * kThreads, run = RUNS ? i / kRun * kRun : 0;
        me[q] = i < n ? order[i] : 0;
        mw[q] = i < n ? w[i] : 0;
        place[q] = run;
        // warps without elements of their own have nothing to count
        if ((i & ~31u) < n) {
            const uint32_t end = RUNS ? min(run + kRun, padded) : padded;
#pragma unroll 2
            for (uint32_t j = run; j < end; j += 4) {
                const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(order + j);
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(order + j + 2);
                place[q] += (a.x > me[q] ? 1u : 0u) + (a.y > me[q] ? 1u : 0u) +
                            (b.x > me[q] ? 1u : 0u) + (b.y > me[q] ? 1u : 0u);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        if (threadIdx.x + q * kThreads < n) order[place[q]] = me[q], w[place[q]] = mw[q];
    __syncthreads();
    if constexpr (RUNS) {
#pragma unroll
        for (int q = 0; q < kPer; ++q) place[q] %= kRun;
#pragma unroll 1
        for (uint32_t run = 0; run < n; run += kRun) {
            uint32_t at[kPer] = {0, 0, 0, 0};            // elements of the run that come before
#pragma unroll 1
            for (uint32_t step = kRun; step > 0; step >>= 1)
#pragma unroll
                for (int q = 0; q < kPer; ++q) {
                    const uint32_t k = run + at[q] + step - 1;
                    if (at[q] + step <= kRun && k < n && order[k] > me[q]) at[q] += step;
                }
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if ((threadIdx.x + q * kThreads) / kRun * kRun != run) place[q] += at[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (threadIdx.x + q * kThreads < n) order[place[q]] = me[q], w[place[q]] = mw[q];
        __syncthreads();
    }
}

__device__ __forceinline__ void sort_list(uint32_t n, u64* order, u64* w) {
    if (n > 512)
        sort_by<true>(n, order, w);
    else
        sort_by<false>(n, order, w);
}

// Lists the columns of the elements from a value on, out of the segments whose maximum reaches it:
// 16 bytes a thread, of a segment that is a load of the warp or (LANES) the groups of some lanes.
template <bool LANES, typename T>
__device__ __noinline__ void gather(const T* x, int V, bool vec, const uint16_t* ids, int n_ids,
                                    int parts, float tau_x, Shared0& sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int VEC = Chunk<T>::VEC, LOADS = Chunk<T>::LOADS, kAhead = 8;
    const int lg_wide = LANES ? 6 - __ffs(parts) : 5;
    const int lg_pieces = LANES ? lg_wide + __ffs(LOADS) - 1 : 5;
    const int total = n_ids << lg_pieces;
    const auto column = [&](int t) {
        const int seg = ids[t >> lg_pieces], k = t & ((1 << lg_pieces) - 1);
        if (!LANES) return (seg * 32 + k) * VEC;
        return Chunk<T>::column(seg >> (5 - lg_wide), k >> lg_wide,
                                ((seg & (parts - 1)) << lg_wide) + (k & ((1 << lg_wide) - 1)));
    };
#pragma unroll 1
    for (int t0 = tid & ~31; t0 < total; t0 += kAhead * kThreads) {
        uint4 raw[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int t = t0 + lane + q * kThreads;
            if (t < total) raw[q] = load_group(x, V, column(t), vec);
        }
        // bit q VEC + e: element e of group q
        u64 hits = 0;
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                hits |= u64(t0 + lane + q * kThreads < total && group_value<T>(raw[q], e) >= tau_x)
                        << (q * VEC + e);
        const uint32_t mine = __popcll(hits);
        uint32_t at = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, at, off);
            if (lane >= off) at += o;
        }
        uint32_t first = 0;
        if (lane == 31) first = atomicAdd(&sh.n_list, at);
        at += __shfl_sync(0xffffffffu, first, 31) - mine;
#pragma unroll 1
        for (; hits != 0; hits &= hits - 1, ++at) {
            const int e = __ffsll(hits) - 1;
            if (at < kShort) sh.order[at] = column(t0 + lane + e / VEC * kThreads) + e % VEC;
        }
    }
}

// Draws from the elements at or above a value, if they settle the boundary and are few.
template <typename T>
__device__ bool short_draw(const Row<T>& r, const Settings& s, const float* smax, uint16_t* ids,
                           int nseg, u64 all, const SampleArgs& a, int64_t row_i, Shared0& sh) {
    const int tid = threadIdx.x;
    if (tid == 0) {
        sh.n_list = 0, sh.n_ids = 0;
        sh.key_m = s.want_m ? min_p_key(a, row_i, r.ws.m) : 0;
    }
    // What min_p keeps is all that is needed where nothing refers to the weight of the first
    // top_k elements.
    const bool by_m = s.want_m && !(s.want_k && s.want_p);
    uint32_t tau = kKeyNegInf + 1;
    if (r.V > kShort && (s.want_k || s.want_p) && !(by_m && s.want_p)) {
        // a list of about -nseg log(1 - top_k / nseg) elements, if the row is in no order
        const bool few = s.want_k && s.top_k <= nseg / 2;
        if (s.want_k && !few && !by_m) return false;
        // between the maximum and what weighs nothing
        const float low = fmaxf(r.ws.m - 47.5f / r.ws.ch, -3.402823466e38f);
        const float need = s.p_value * 1.00001f * static_cast<float>(all) *
                           __uint_as_float(uint32_t(127 - r.bits) << 23);
        if (few || !s.want_k) {
            bool found;
            const float x = reach_value(r, smax, nseg, static_cast<int>(s.top_k),
                                        s.want_k ? 0.f : need, low, found, sh);
            if (!found && !s.want_k) return false;   // a wide nucleus
            tau = max(tau, order_key(x));
        }
    }
    __syncthreads();
    const uint32_t key_m = sh.key_m;
    if (by_m) tau = max(tau, key_m);
    const float tau_x = key_value(tau);
    for (int c = tid; c < nseg; c += kThreads)
        if (smax[c] >= tau_x) {
            const uint32_t at = atomicAdd(&sh.n_ids, 1u);
            if (at < kShort) ids[at] = static_cast<uint16_t>(c);
        }
    __syncthreads();
    const int n_ids = sh.n_ids;
    if (n_ids > kShort) return false;
    if (a.parts == 0)
        gather<false>(r.x, r.V, r.vec, ids, n_ids, 0, tau_x, sh);
    else
        gather<true>(r.x, r.V, r.vec, ids, n_ids, a.parts, tau_x, sh);
    __syncthreads();
    const uint32_t n = sh.n_list;
    if (n > kShort) return false;
#pragma unroll 1
    for (uint32_t i = tid; i < n; i += kThreads) {
        const uint32_t col = static_cast<uint32_t>(sh.order[i]);
        const float x = load_one(r.x + col);
        sh.order[i] = (u64(order_key(x)) << 32) | (0xffffffffu - col);
        sh.w[i] = fixed_weight(x, r.ws, sh.table);
    }
    sort_list(n, sh.order, sh.w);
    // thread t holds elements 4 t .. 4 t + 3 of the order
    constexpr int kPer = kShort / kThreads;
    const uint32_t i0 = kPer * tid;
    u64 w[kPer], b[kPer + 1], mine = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) w[q] = i0 + q < n ? sh.w[i0 + q] : 0, mine += w[q];
    const Scanned sum = block_scan<kThreads>(mine, 0, sh.part, sh.part_n);
    b[0] = sum.v;
#pragma unroll
    for (int q = 0; q < kPer; ++q) b[q + 1] = b[q] + w[q];
    uint32_t keep = n;
    u64 s_k = sum.tv;                                // fewer elements than top_k: all of them
    if (s.want_k && static_cast<u64>(s.top_k) < n) {
        keep = static_cast<uint32_t>(s.top_k);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            if (keep - 1 == i0 + q) sh.at_w = b[q + 1];
        __syncthreads();
        s_k = sh.at_w;
    }
    if (s.want_p) {
        u64 lo = s_k, hi = s_k;                      // exact, where the list holds all that counts
        const bool whole = s.want_k || (r.V <= kShort && !by_m);
        if (!whole) total_bounds(all, r.V, lo, hi);
        const u64 need_lo = max(u64(1), part_of(s.top_p, lo, true));
        const u64 need_hi = whole ? need_lo : max(u64(1), part_of(s.top_p, hi, true));
        if (need_hi > sum.tv && !by_m) return false;
        // the order's first elements before whose sum the need is not reached
        uint32_t n_lo = 0, n_hi = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            n_lo += i0 + q < n && b[q] < need_lo ? 1u : 0u;
            n_hi += i0 + q < n && b[q] < need_hi ? 1u : 0u;
        }
        const Scanned c = block_scan<kThreads>(n_hi, n_lo, sh.part, sh.part_n);
        if (c.tn != c.tv) return false;              // the total's error matters
        keep = min(keep, c.tn);
    }
    if (s.want_m) {
        const u64 cut = u64(key_m) << 32;
        uint32_t n_m = 0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) n_m += i0 + q < n && sh.order[i0 + q] >= cut ? 1u : 0u;
        keep = min(keep, block_scan<kThreads>(0, n_m, sh.part, sh.part_n).tn);
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        if (keep - 1 == i0 + q) sh.at_w = b[q + 1];
    // the kept elements by index: their order words become (~index, key)
    __syncthreads();
    const u64 kept = sh.at_w;
    const u64 target = part_of(s.u, kept, false);
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        if (i0 + q < keep) {
            const u64 o = sh.order[i0 + q];
            sh.order[i0 + q] = (o << 32) | (o >> 32);
        }
    __syncthreads();
    sort_list(keep, sh.order, sh.w);
    mine = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) w[q] = i0 + q < keep ? sh.w[i0 + q] : 0, mine += w[q];
    u64 run = block_scan<kThreads>(mine, 0, sh.part, sh.part_n).v;
    u64 drawn = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        if (run <= target && target < run + w[q]) drawn = sh.order[i0 + q];
        run += w[q];
    }
    if (drawn != 0)
        write_drawn(a, row_i, int(0xffffffffu - uint32_t(drawn >> 32)),
                    key_value(uint32_t(drawn)), r.ws, max(all, kept), kept);
    return true;
}

__host__ __device__ constexpr size_t scan_smem(int nch, int nseg) {
    const size_t ring = offsetof(Shared0, order) + kWarps * kRing;
    const size_t tail =
        sizeof(Shared0) + size_t(nch) * 12 + size_t(nseg) * 4 + kShort * 2 + 64;
    return ring > tail ? ring : tail;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    sample_scan_kernel(const T* __restrict__ logits, const SampleArgs a, int nch, int own,
                       int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared0& sh = *reinterpret_cast<Shared0*>(smem);
    u64* cw = reinterpret_cast<u64*>(smem + sizeof(Shared0));
    float* cmax = reinterpret_cast<float*>(cw + nch);
    const int nseg = segments_of(nch, a.parts, sizeof(T));   // 0: too many to be kept
    float* smax = reinterpret_cast<float*>(cw) + (nch * 3 + 3) / 4 * 4;
    uint16_t* ids = reinterpret_cast<uint16_t*>(smax + (nseg + 3) / 4 * 4);
    const int64_t row_i = blockIdx.x / ranks;
    const int rank = blockIdx.x % ranks;             // = the block's rank in its cluster
    // The block that finishes the row.  Not always the same one of its cluster: clusters that
    // follow each other on the same SMs would then finish their rows on the same few of them
    // (28.4 instead of 23.9 us at [64, 151936] with top_k and top_p).
    const bool lead = rank == static_cast<int>(row_i % ranks);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    RowHeader* head = static_cast<RowHeader*>(a.workspace) + row_i;
    float2* stats = row_stats(a, row_i, nch);
    if (lead)
        for (int i = tid; i < kExpEntries / 2; i += kThreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(sh.table + 2 * i)),
                         "l"(kExpTable.v + 2 * i)
                         : "memory");
    cp_commit();
    // what the stream did before is complete: the logits, and the last call's use of the workspace
    wait_previous(logits);
    if (a.mask != nullptr && a.mask[row_i] == 0) {
        cp_wait<0>();
        if (lead && tid == 0) {
            write_row(a, row_i, -1, 0.f, 0.f);
            row_modes(a)[row_i] = kRowDone;
        }
        return;
    }
    // the row is on its way while its settings are read
    const T* x = logits + row_i * a.stride;
    const int first = rank * own, share = max(0, min(own, nch - first));
    const Ring<T> ring{reinterpret_cast<uint4*>(sh.order) + warp * (kRing / 16) + lane};
    constexpr int S = Ring<T>::S;
#pragma unroll
    for (int q = 0; q < S; ++q) {
        if (warp + q * kWarps < share)
            ring.fetch(q, x, a.V, first + warp + q * kWarps, lane, a.vec_ok);
        cp_commit();
    }
    const Settings s = read_settings(a, row_i);
    if (!s.ok) {
        cp_wait<0>();
        if (lead && tid == 0) {
            write_failed(a, row_i, RLK_DEVERR_SAMPLE_PARAM);
            row_modes(a)[row_i] = kRowDone;
        }
        return;
    }
    Row<T> r = make_row(logits, a, row_i, s, nch, own, rank);
    const bool cut = s.want_k || s.want_p || s.want_m;
    float* segs = row_segs(a, row_i, nch);
    const float2 scale = fast_scale(s);
    int slot = 0;
#pragma unroll 1
    for (int i = warp; i < r.mine; i += kWarps) {
        cp_wait<S - 1>();
        Chunk<T> c;
        ring.read(slot, c);
        float seg[Chunk<T>::LOADS], ml;
        if (cut && a.parts == 0) {
            const float2 st = chunk_stats<true>(c, scale, seg, ml);
            if (lane == 0) {
                stats[r.first + i] = st;
#pragma unroll
                for (int j = 0; j < Chunk<T>::LOADS; ++j)
                    segs[(r.first + i) * Chunk<T>::LOADS + j] = seg[j];
            }
        } else {
            const float2 st = chunk_stats<false>(c, scale, seg, ml);
            if (lane == 0) stats[r.first + i] = st;
            if (cut) {
                const int wide = 32 / a.parts;       // lanes of a segment
#pragma unroll 1
                for (int off = wide >> 1; off > 0; off >>= 1)
                    ml = fmaxf(ml, __shfl_xor_sync(0xffffffffu, ml, off));
                if (lane % wide == 0) segs[(r.first + i) * a.parts + lane / wide] = ml;
            }
        }
        if (i + S * kWarps < r.mine)
            ring.fetch(slot, r.x, r.V, r.first + i + S * kWarps, lane, r.vec);
        cp_commit();
        slot = slot + 1 == S ? 0 : slot + 1;
    }
    // the other blocks are done once their part is out
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (!lead) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    float m = -INFINITY;
    bool bad = false;
    for (int i = tid; i < nch; i += kThreads) {
        const float2 st = stats[i];
        cmax[i] = st.x;
        cw[i] = __float_as_uint(st.y);
        m = fmaxf(m, st.x);
        bad |= st.y != st.y;
    }
    if (cut) {                               // padded to whole groups of 4 with -inf
#pragma unroll 2
        for (int i = tid * 4; i < nseg; i += kThreads * 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (i + 3 < nseg) v = *reinterpret_cast<const float4*>(segs + i);
            else v.x = segs[i], v.y = i + 1 < nseg ? segs[i + 1] : -INFINITY,
                 v.z = i + 2 < nseg ? segs[i + 2] : -INFINITY;
            *reinterpret_cast<float4*>(smax + i) = v;
        }
    }
    m = warp_max(m);
    if (lane == 0) sh.part_n[warp] = __float_as_uint(m);
    bad = __syncthreads_or(bad);
    m = warp_max(lane < kWarps ? __uint_as_float(sh.part_n[lane]) : -INFINITY);
    if (bad || m == -INFINITY) {
        if (tid == 0) {
            write_failed(a, row_i, RLK_DEVERR_LOGITS);
            row_modes(a)[row_i] = kRowDone;
        }
        return;
    }
    r.ws.m = m;
    u64 mine = 0;
#pragma unroll 1
    for (int i = tid; i < nch; i += kThreads) {
        const uint32_t st = static_cast<uint32_t>(cw[i]);
        const u64 top = fixed_weight(cmax[i], r.ws, sh.table);
        const u64 w = scale_weight(__uint_as_float(st & 0x7fffffffu), top) + (st >> 31 ? top : 0);
        cw[i] = w;
        mine += w;
    }
    const u64 all = block_scan<kThreads>(mine, 0, sh.part, sh.part_n).tv;   // its barriers publish cw
    const bool done = !cut ? fast_draw(r, cmax, cw, all, s, a, row_i, sh)
                           : nseg > 0 && short_draw(r, s, smax, ids, nseg, all, a, row_i, sh);
    if (tid == 0) {
        head->all = all;
        head->m = m;
        row_modes(a)[row_i] = done ? kRowDone : kRowSearch;
    }
}

// ----------------------------------------------------------------------------- search

// The rows to search of the batch base .. base + THREADS - 1 are dealt to groups of `group`
// blocks: every block counts them out of the rows' modes, and group g of G takes those whose
// number among them is g modulo G.  So they are spread evenly without a counter.  A group is a
// cluster, or (PARTED) a part of one where there are more rows than clusters.
struct Queue {
    uint32_t n;                          // rows of this block's group
    uint16_t at[kExact];                 // their places in the batch
};
// Returns the most rows that a group has.
template <int THREADS, bool PARTED>
__device__ uint32_t queue_rows(const uint32_t* modes, int N, int base, uint32_t ranks,
                               uint32_t& group, Queue& queue, u64* part, uint32_t* part_n) {
    const int tid = threadIdx.x;
    const bool hard = base + tid < N && modes[base + tid] == kRowSearch;
    if (!__syncthreads_or(hard)) return 0;
    if (tid == 0) queue.n = 0;
    const Scanned s = block_scan<THREADS>(0, hard ? 1 : 0, part, part_n);
    group = ranks;
    if (PARTED)
        while (group > 1 && s.tn > gridDim.x / group) group /= 2;
    const uint32_t groups = gridDim.x / group;
    if (hard && s.n % groups == blockIdx.x / group) {
        queue.at[s.n / groups] = static_cast<uint16_t>(tid);
        atomicAdd(&queue.n, 1u);
    }
    __syncthreads();
    return (s.tn + groups - 1) / groups;
}

// A step that block 0 asks of all blocks.  Elements are above, inside or below a window of
// values [key_value(klo), key_value(khi)].
enum : int { kHist, kCollect, kDone };
struct Cmd {
    int type;
    uint32_t klo, khi;
    int shift;        // kHist: bins of the keys, (khi - key) >> shift; -1: of the distance
    int by_weight;    // kHist: weights instead of counts, in bins of the distance 12-bit ones
    int list;         // kCollect: 1 lists the elements inside, 0 counts them per chunk
    int total;        // also the exact weight of all elements
};

// Shared memory of the search.
struct Shared {
    u64 table[kExpEntries];
    uint32_t key[kList], idx[kList];     // block 0: the merged list
    union {                              // of one step or the other
        struct {                         // the upper words: weights of keys
            uint32_t hist[kBins], hist_hi[kBins];
        };
        struct {
            uint32_t own_key[kList], own_idx[kList];   // this block's part of the list
        };
        struct {
            uint32_t cnt[kSelect], lo[kSelect], hi[kSelect];   // block 0, after the merge
        };
    };
    u64 part[kSearch / 32];
    uint32_t part_n[kSearch / 32];
    u64 own_above, own_total;            // exact weights, all own chunks
    uint32_t own_count;
    uint32_t n_list, n_few, key_m;
    Queue queue;
    // results of block-wide searches
    u64 at_w, width;
    uint32_t at_n;
    int at, at2;
    Cmd cmd;
};

// monotone in x; kBins and more: weight 0
template <typename T>
__device__ __forceinline__ float distance(float x, const Row<T>& r) {
    return fminf((r.ws.m - x) * r.scale, 2.f * kBins);
}

// The window as values: above is x > hi, inside lo <= x <= hi.  With no window (khi at or
// below -inf's key) all that is not -inf is above and nothing inside.
__device__ __forceinline__ void window_of(const Cmd& cmd, float& lo, float& hi) {
    const bool none = cmd.khi <= kKeyNegInf;
    lo = none ? INFINITY : key_value(max(cmd.klo, kKeyNegInf + 1));
    // the key between the negatives and 0 is no element's, but its value (-0) compares as 0
    const uint32_t khi = cmd.khi == 0x7fffffffu ? 0x7ffffffeu : cmd.khi;
    hi = none ? -INFINITY : khi > order_key(INFINITY) ? INFINITY : key_value(khi);
}

// a weight onto a sum in two words
__device__ __forceinline__ void add_weight(uint32_t* lo, uint32_t* hi, u64 w) {
    const uint32_t wl = static_cast<uint32_t>(w);
    const uint32_t old = atomicAdd(lo, wl);
    atomicAdd(hi, static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u));
}

// Histogram of the window.  Of keys: with the weights as integers, in the bins and above the window,
// so that the boundary's bin is certain however far apart its elements lie (codes relative to one
// value lose what is 13 bits below it: a window that spans a gap never closed).  About 9 us over 8
// blocks at V = 151936: shared-memory atomics and conversions bind it.
template <typename T>
__device__ __noinline__ void step_hist(const Row<T>& row, const Cmd& command, const float* cmax,
                                       Shared& sh) {
    const Row<T> r = row;                    // in registers for the loops
    const Cmd cmd = command;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kBins; i += kSearch) sh.hist[i] = sh.hist_hi[i] = 0;
    if (threadIdx.x == 0) sh.own_above = sh.own_total = 0;
    __syncthreads();
    const float unit = kRange / kBins;
    float lo, hi;
    window_of(cmd, lo, hi);
    u64 above = 0, all = 0;
    Chunk<T> next;                           // on its way while the one before is worked on
    if (warp < r.mine) next.load(r.x, r.V, r.first + warp, lane, r.vec);
#pragma unroll 1
    for (int i = warp; i < r.mine; i += kSearch / 32) {
        Chunk<T> c = next;
        if (i + kSearch / 32 < r.mine)
            next.load(r.x, r.V, r.first + i + kSearch / 32, lane, r.vec);
        const float top = cmax[r.first + i];
        if (distance(top, r) >= kBins || (cmd.shift >= 0 && !cmd.total && top < lo)) continue;
        if (cmd.shift < 0) {
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const float t = distance(c.get(e), r);
                const int b = static_cast<int>(t);
                const float q = cmd.by_weight ? rintf(4096.f * ex2_approx((b - t) * unit)) : 1.f;
                if (b < kBins) atomicAdd(&sh.hist[b], static_cast<uint32_t>(q));
            }
            continue;
        }
#pragma unroll 1
        for (int j = 0; j < Chunk<T>::kQuads; ++j) {
            float x[4];
            u64 w[4] = {0, 0, 0, 0};
            c.take(x);
            if (cmd.by_weight) {
                fixed_weights(make_float2(x[0], x[1]), r.ws, sh.table, w[0], w[1]);
                fixed_weights(make_float2(x[2], x[3]), r.ws, sh.table, w[2], w[3]);
            }
            all += (w[0] + w[1]) + (w[2] + w[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                above += x[e] > hi ? w[e] : 0;
                if (!(x[e] >= lo && x[e] <= hi)) continue;
                const uint32_t b = (cmd.khi - order_key(x[e])) >> cmd.shift;
                if (cmd.by_weight)
                    add_weight(&sh.hist[b], &sh.hist_hi[b], w[e]);
                else
                    atomicAdd(&sh.hist[b], 1u);
            }
        }
    }
    above = warp_sum(above);
    all = warp_sum(all);
    if (lane == 0 && above != 0) atomicAdd(&sh.own_above, above);
    if (lane == 0 && all != 0) atomicAdd(&sh.own_total, all);
    __syncthreads();
}

// Exact weight above the window, per chunk, and the elements inside it.  About 13 us over 8 blocks
// at V = 151936: the 64-bit arithmetic of the weights binds it.
template <typename T>
__device__ __noinline__ void step_collect(const Row<T>& row, const Cmd& command, const float* cmax,
                                          u64* own_w, uint32_t* own_n, Shared& sh) {
    const Row<T> r = row;                    // in registers for the loops
    const Cmd cmd = command;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.own_count = 0, sh.own_total = 0;
    __syncthreads();
    float lo, hi;
    window_of(cmd, lo, hi);
    const bool everything = hi == -INFINITY;
    u64 all = 0;
    Chunk<T> next;                           // on its way while the one before is worked on
    if (warp < r.mine) next.load(r.x, r.V, r.first + warp, lane, r.vec);
#pragma unroll 1
    for (int i = warp; i < r.mine; i += kSearch / 32) {
        Chunk<T> c = next;
        if (i + kSearch / 32 < r.mine)
            next.load(r.x, r.V, r.first + i + kSearch / 32, lane, r.vec);
        const float top = cmax[r.first + i];
        u64 w = 0;
        uint32_t n = 0;
        if (top >= lo || ((cmd.total || everything) && distance(top, r) < kBins)) {
            u64 sum = 0;
#pragma unroll 1
            for (int j = 0; j < Chunk<T>::kQuads; ++j) {
                float x[4];
                u64 we[4];
                c.take(x);
                fixed_weights(make_float2(x[0], x[1]), r.ws, sh.table, we[0], we[1]);
                fixed_weights(make_float2(x[2], x[3]), r.ws, sh.table, we[2], we[3]);
                sum += (we[0] + we[1]) + (we[2] + we[3]);
                if (everything) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w += x[e] > hi ? we[e] : 0;
                    if (!(x[e] >= lo && x[e] <= hi)) continue;
                    ++n;
                    if (!cmd.list) continue;
                    const uint32_t at = atomicAdd(&sh.own_count, 1u);
                    if (at < kList) {
                        const int v = j * 4 + e;
                        sh.own_key[at] = order_key(x[e]);
                        sh.own_idx[at] = Chunk<T>::column(r.first + i, v / Chunk<T>::VEC, lane) +
                                         v % Chunk<T>::VEC;
                    }
                }
            }
            all += sum;
            w = warp_sum(everything ? sum : w);
            n = cmd.list ? 0 : __reduce_add_sync(0xffffffffu, n);
        }
        if (lane == 0) own_w[i] = w, own_n[i] = n;
    }
    all = warp_sum(all);
    if (lane == 0 && all != 0) atomicAdd(&sh.own_total, all);
    __syncthreads();
}

// Selection in the merged list, whose keys lie in [lo, hi]: the key at which the count (or
// weight) of the elements from the top reaches `need` >= 1, and count and weight above that
// key.  A histogram of 1024 bins of the keys' range, then of the bin's, until a warp can order
// what is left (at once, nearly always): equal parts of the range keep the atomics of one bin
// few, where digits of the keys would not.
struct Selected {
    uint32_t key;
    u64 n, w;
};
template <typename T>
__device__ __noinline__ Selected list_select(const Row<T>& row, bool by_weight, u64 need,
                                             uint32_t lo, uint32_t hi, Shared& sh) {
    const WeightScale ws = row.ws;
    u64 n_up = 0, w_up = 0;
    int shift;
    if (threadIdx.x == 0) sh.n_few = 0;
#pragma unroll 1
    do {
        shift = max(0, 22 - __clz(hi - lo));         // (hi - lo) >> shift < 1024
        __syncthreads();
        for (int i = threadIdx.x; i < kSelect; i += kSearch) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < sh.n_list; i += kSearch) {
            const uint32_t k = sh.key[i];
            if (k < lo || k > hi) continue;
            const uint32_t b = (hi - k) >> shift;
            atomicAdd(&sh.cnt[b], 1u);
            add_weight(&sh.lo[b], &sh.hi[b], fixed_weight(key_value(k), ws, sh.table));
        }
        __syncthreads();
        // thread t holds bins 2 t and 2 t + 1, from the top down
        static_assert(kSelect == 2 * kSearch, "two bins a thread");
        const int b = 2 * threadIdx.x;
        const u64 w0 = (u64(sh.hi[b]) << 32) | sh.lo[b];
        const u64 w1 = (u64(sh.hi[b + 1]) << 32) | sh.lo[b + 1];
        const uint32_t n0 = sh.cnt[b], n1 = sh.cnt[b + 1];
        const Scanned s = block_scan<kSearch>(w0 + w1, n0 + n1, sh.part, sh.part_n);
        const u64 c0 = by_weight ? w_up + s.v : n_up + s.n;
        const u64 c1 = c0 + (by_weight ? w0 : u64(n0)), c2 = c1 + (by_weight ? w1 : u64(n1));
        if (c0 < need && c1 >= need)
            sh.at = b, sh.at_w = w_up + s.v, sh.at_n = static_cast<uint32_t>(n_up) + s.n;
        else if (c1 < need && c2 >= need)
            sh.at = b + 1, sh.at_w = w_up + s.v + w0,
            sh.at_n = static_cast<uint32_t>(n_up) + s.n + n0;
        __syncthreads();
        const uint32_t at = sh.at;
        w_up = sh.at_w;
        n_up = sh.at_n;
        const uint32_t top = hi - (at << shift);
        lo = max(lo, top - ((1u << shift) - 1));
        hi = top;
    } while (shift > 0 && sh.cnt[sh.at] > 32);
    if (shift == 0) {
        __syncthreads();
        return Selected{hi, n_up, w_up};
    }
    uint32_t* few = sh.lo;
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < sh.n_list; i += kSearch) {
        const uint32_t k = sh.key[i];
        if (k >= lo && k <= hi) few[atomicAdd(&sh.n_few, 1u)] = k;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t n = sh.n_few;
        const uint32_t k = threadIdx.x < n ? few[threadIdx.x] : 0;
        const u64 w = threadIdx.x < n ? fixed_weight(key_value(k), ws, sh.table) : 0;
        uint32_t n_above = 0, n_to = 0;
        u64 w_above = 0, w_to = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n; ++j) {
            const uint32_t kj = __shfl_sync(0xffffffffu, k, j);
            const u64 wj = __shfl_sync(0xffffffffu, w, j);
            n_above += kj > k ? 1u : 0u;
            n_to += kj >= k ? 1u : 0u;
            w_above += kj > k ? wj : 0;
            w_to += kj >= k ? wj : 0;
        }
        const u64 c0 = by_weight ? w_up + w_above : n_up + n_above;
        const u64 c1 = by_weight ? w_up + w_to : n_up + n_to;
        // lanes of equal keys write the same
        if (threadIdx.x < n && c0 < need && c1 >= need) {
            sh.at = static_cast<int>(k);
            sh.at_w = w_up + w_above;
            sh.at_n = static_cast<uint32_t>(n_up) + n_above;
        }
    }
    __syncthreads();
    const Selected r{static_cast<uint32_t>(sh.at), sh.at_n, sh.at_w};
    __syncthreads();
    return r;
}

// What block 0 carries from step to step (uniform over its threads).
struct Search {
    bool want_k, want_p;       // boundaries still to be found
    bool draw;                 // the next kCollect is the last
    bool exact;                // s_lo == s_hi is the exact weight that top_p refers to
    u64 n_above;               // count above the window (want_k)
    u64 s_lo, s_hi;            // bounds of the total that top_p refers to
    uint32_t key;              // the boundary so far
    u64 ties;
    uint32_t key_m;            // elements below are cut by min_p
    u64 top_k, all;
    SampleFraction top_p;

    __device__ u64 need(u64 total) const { return max(u64(1), part_of(top_p, total, true)); }
};

__device__ __forceinline__ Cmd make_hist0(bool by_weight) {
    return Cmd{kHist, 0u, 0xffffffffu, -1, by_weight ? 1 : 0, 0, 0};
}
// exact weights above a key, and the number of elements equal to it
__device__ __forceinline__ Cmd make_above(uint32_t key) {
    return Cmd{kCollect, key, key, 0, 0, 0, 0};
}

// the boundary is known up to min_p: the last step
__device__ __forceinline__ void ask_draw(Search& P, Cmd& cmd) {
    P.want_k = P.want_p = false;
    if (P.key_m > P.key) P.key = P.key_m - 1, P.ties = 0;
    P.draw = true;
    cmd = make_above(P.key);
}
// the top_p search from its beginning, or the end of the search without top_p
__device__ __forceinline__ void start_p(Search& P, Cmd& cmd) {
    if (!P.want_p) return ask_draw(P, cmd);
    cmd = make_hist0(true);
}
// a histogram of the window's keys
__device__ __forceinline__ void next_hist(Cmd& cmd) {
    cmd.type = kHist;
    const uint32_t span = cmd.khi - cmd.klo;
    cmd.shift = 0;
    while ((span >> cmd.shift) >= kBins) ++cmd.shift;
}
// the exact total, where this step formed it
__device__ __forceinline__ void take_total(Search& P, const Cmd& cmd, int ranks, Shared& sh) {
    if (!cmd.total) return;
    u64 t = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += k < ranks ? *peer(&sh.own_total, k) : 0;
    P.exact = true;
    P.s_lo = P.s_hi = P.all = t;
}

// The lowest key in [lo, hi] whose value lies in bin `bin` or above; hi's does.  One warp, 32
// trials at a time.
template <typename T>
__device__ __noinline__ uint32_t first_key(const Row<T>& r, uint32_t lo, uint32_t hi, int bin) {
    const uint32_t lane = threadIdx.x & 31;
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 32 + 1;
        const uint32_t k = min(hi, lo + step * lane);
        const bool in = static_cast<int>(distance(key_value(k), r)) <= bin;
        const int first = __ffs(__ballot_sync(0xffffffffu, in)) - 1;
        if (first == 0) return lo;
        if (first > 0) hi = min(hi, lo + step * first);
        lo = min(hi, lo + step * ((first < 0 ? 32 : first) - 1) + 1);
    }
    return hi;
}

// Narrows the window from the cluster's histograms and asks for the next step.
template <typename T>
__device__ __noinline__ void after_hist(const Row<T>& r, Search& P, Cmd& cmd, int ranks,
                                        Shared& sh) {
    constexpr int kPer = kBins / kSearch;
    static_assert(kPer == 4, "a thread takes 16 bytes of each histogram");
    const int b0 = threadIdx.x * kPer;
    const bool keys = cmd.shift >= 0;
    u64 q[kPer] = {0, 0, 0, 0}, weight[kPer];
    u64 above = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= ranks) break;
        const uint4 h = *reinterpret_cast<const uint4*>(peer(sh.hist, k) + b0);
        q[0] += h.x, q[1] += h.y, q[2] += h.z, q[3] += h.w;
        if (!keys) continue;
        above += *peer(&sh.own_above, k);
        if (!cmd.by_weight) continue;
        const uint4 hi = *reinterpret_cast<const uint4*>(peer(sh.hist_hi, k) + b0);
        q[0] += u64(hi.x) << 32, q[1] += u64(hi.y) << 32;
        q[2] += u64(hi.z) << 32, q[3] += u64(hi.w) << 32;
    }
    if (keys) take_total(P, cmd, ranks, sh);
    u64 mine = 0;
    const float unit = kRange / kBins;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        weight[i] = keys || !cmd.by_weight
                        ? q[i]
                        : __float2ull_rn(static_cast<float>(q[i]) *
                                         ex2_approx(-(b0 + i) * unit + (r.bits - 12)));
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += weight[i];
    const u64 before = block_scan<kSearch>(mine, 0, sh.part, sh.part_n).v;
    // the first bins at which the running sum surely may, and surely must, have reached the
    // need
    if (threadIdx.x == 0) sh.at = sh.at2 = kBins, sh.at_w = sh.width = 0;
    __syncthreads();
    u64 need_lo = P.top_k, need_hi = P.top_k, base = P.n_above;
    float err = 0.f;
    if (!P.want_k) {
        need_lo = P.need(P.s_lo);
        need_hi = P.need(P.s_hi);
        base = above;
        err = keys ? 0.f : kBinErr;
    }
    u64 run = before, at_before = 0;
    int first_may = kBins, first_must = kBins;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const u64 prev = run;
        run += weight[i];
        const u64 slack = err > 0.f ? static_cast<u64>(static_cast<float>(run) * err) + 4096 : 0;
        if (first_may == kBins && base + run + slack >= need_lo) {
            first_may = b0 + i;
            at_before = prev;
        }
        if (first_must == kBins && base + run >= need_hi + slack) first_must = b0 + i;
    }
    if (first_may < kBins) atomicMin(&sh.at, first_may);
    if (first_must < kBins) atomicMin(&sh.at2, first_must);
    __syncthreads();
    if (first_may < kBins && first_may == sh.at) sh.at_w = at_before;
    __syncthreads();
    const int at = sh.at, at2 = sh.at2;
    u64 skipped = sh.at_w;
    const int j1 = min(at, kBins - 1), j2 = max(j1, min(at2, kBins - 1));
    // elements of the new window, or their weight
    u64 est = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (b0 + i >= j1 && b0 + i <= j2) est += q[i];
    if (est != 0) atomicAdd(&sh.width, est);         // by few threads
    __syncthreads();
    est = sh.width;
    if (at == kBins) {
        // fewer elements of weight > 0 than top_k: nothing is cut.  (A weight is reached: the
        // bounds of total and bins hold.)
        P.key = kKeyNegInf;
        P.ties = 0;
        if (P.want_k) {
            P.want_k = false;
            start_p(P, cmd);
        } else {
            ask_draw(P, cmd);
        }
        return;
    }
    // the first top_k altogether, where the list holds them: top_p is then settled in it too
    if (cmd.by_weight && !keys) est = est / 3600 + 1;    // codes of the distance lie near 4096
    const bool whole = P.want_k && !keys && skipped + est <= kList;
    if (whole) skipped = 0;
    if (P.want_k) P.n_above += skipped;
    if (!keys) {
        // the keys of exactly these bins: the lowest of bin j2 or above, and the highest of
        // bin j1 or below
        const uint32_t bottom = kKeyNegInf + 1, top = order_key(r.ws.m);
        if (threadIdx.x < 32) {
            const uint32_t lo = first_key(r, bottom, top, j2);
            if (threadIdx.x == 0) sh.at = static_cast<int>(lo);
        } else if (threadIdx.x < 64) {
            const uint32_t hi = j1 == 0 || whole ? top : first_key(r, bottom, top, j1 - 1) - 1;
            if (threadIdx.x == 32) sh.at2 = static_cast<int>(hi);
        }
        __syncthreads();
        cmd.klo = static_cast<uint32_t>(sh.at);
        cmd.khi = static_cast<uint32_t>(sh.at2);
        __syncthreads();
    } else {
        const int64_t hi = int64_t(cmd.khi) - (int64_t(j1) << cmd.shift);
        const int64_t lo = int64_t(cmd.khi) - (int64_t(j2 + 1) << cmd.shift) + 1;
        cmd.klo = static_cast<uint32_t>(max(int64_t(cmd.klo), lo));
        cmd.khi = static_cast<uint32_t>(hi);
        if (cmd.by_weight) {             // at most so many of the least weight in it
            const u64 least = fixed_weight(key_value(cmd.klo), r.ws, sh.table);
            est = least > 0 ? est / least : u64(kList) + 1;
        }
    }
    if (cmd.klo == cmd.khi || est <= kList) {
        cmd.type = kCollect;
        cmd.list = cmd.klo == cmd.khi ? 0 : 1;
        return;
    }
    next_hist(cmd);
}

// Draws from the kept set: cw[c] holds the chunks' weight above the window, cn[c] the
// number of elements equal to P.key (list: both completed from the list here).
template <typename T>
__device__ __noinline__ void search_draw(const Row<T>& r, const Search& P, const Cmd& cmd, u64* cw,
                                         uint32_t* cn, const SampleArgs& a, int64_t row_i,
                                         SampleFraction u, Shared& sh) {
    const int tid = threadIdx.x;
    if (cmd.list) {
#pragma unroll 1
        for (uint32_t i = tid; i < sh.n_list; i += kSearch) {
            const int c = sh.idx[i] / kChunk;
            if (sh.key[i] > P.key)
                atomicAdd(&cw[c], fixed_weight(key_value(sh.key[i]), r.ws, sh.table));
            else if (sh.key[i] == P.key) atomicAdd(&cn[c], 1u);
        }
        __syncthreads();
    }
    const u64 wt = P.ties == 0 ? 0 : fixed_weight(key_value(P.key), r.ws, sh.table);
    const uint32_t ties = static_cast<uint32_t>(min(P.ties, u64(0xffffffffu)));
    const int each = (r.nch + kSearch - 1) / kSearch;
    const int c0 = min(r.nch, tid * each), c1 = min(r.nch, c0 + each);
    u64 w = 0;
    uint32_t n = 0;
    for (int c = c0; c < c1; ++c) w += cw[c], n += cn[c];
    const Scanned s = block_scan<kSearch>(w, n, sh.part, sh.part_n);
    w = s.v, n = s.n;
    const u64 kept = s.tv + min(s.tn, ties) * wt;
    // nothing cut: one total for both; otherwise the kept part is at most the whole
    const u64 all = P.key <= kKeyNegInf ? kept : max(P.all, kept);
    const u64 target = part_of(u, kept, false);
    if (tid == 0) sh.at = 0, sh.at_w = 0, sh.at_n = 0;
    __syncthreads();
    for (int c = c0; c < c1; ++c) {
        const u64 lo = w + min(n, ties) * wt, w_at = w;
        const uint32_t n_at = n;
        w += cw[c], n += cn[c];
        const u64 hi = w + min(n, ties) * wt;
        if (lo <= target && target < hi) sh.at = c, sh.at_w = w_at, sh.at_n = n_at;
    }
    __syncthreads();
    // the chunk's columns in order, one a thread
    static_assert(kSearch == kChunk, "a thread takes a column");
    const int col = sh.at * kChunk + tid;
    const float x = col < r.V ? load_one(r.x + col) : -INFINITY;
    const uint32_t k = order_key(x);
    const u64 we = k > P.key ? fixed_weight(x, r.ws, sh.table) : 0;
    const uint32_t tie = k == P.key ? 1 : 0;
    const u64 w_at = sh.at_w;
    const uint32_t n_at = sh.at_n;
    const Scanned in = block_scan<kSearch>(we, tie, sh.part, sh.part_n);
    const u64 lo = w_at + in.v + min(n_at + in.n, ties) * wt;
    const u64 hi = w_at + in.v + we + min(n_at + in.n + tie, ties) * wt;
    if (lo <= target && target < hi) write_drawn(a, row_i, col, x, r.ws, all, kept);
}

// All blocks' weights and counts per chunk, and their lists as one; sums in `above`,
// `inside`.  Returns the list's length, 0xffffffff if it does not fit.
template <typename T>
__device__ __noinline__ uint32_t merge(const Row<T>& r, const Cmd& cmd, u64* cw, uint32_t* cn,
                                       u64* own_w, uint32_t* own_n, int ranks, bool draws, u64& above,
                                       uint32_t& inside, Shared& sh) {
    u64 mine = 0;
    uint32_t n_mine = 0;
#pragma unroll 2
    for (int c = threadIdx.x; c < r.nch; c += kSearch) {
        const int k = c / r.own, i = c - k * r.own;
        const u64 w = peer(own_w, k)[i];
        const uint32_t n = peer(own_n, k)[i];
        cw[c] = w;
        cn[c] = n;
        mine += w;
        n_mine += n;
    }
    if (draws) {
        __syncthreads();
        return 0;
    }
    const Scanned s = block_scan<kSearch>(mine, n_mine, sh.part, sh.part_n);
    above = s.tv;
    inside = s.tn;
    if (!cmd.list) return 0;
    uint32_t start[9] = {0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        start[k + 1] = start[k] + (k < ranks ? *peer(&sh.own_count, k) : 0);
    const uint32_t n = start[8];
    const bool over = n > kList;
    if (!over)
#pragma unroll 2
        for (uint32_t i = threadIdx.x; i < n; i += kSearch) {
            int k = 0;
            uint32_t from = 0;
#pragma unroll
            for (int j = 1; j < 8; ++j)
                if (i >= start[j]) k = j, from = start[j];
            const uint32_t key = peer(sh.own_key, k)[i - from];
            sh.key[i] = key;
            sh.idx[i] = peer(sh.own_idx, k)[i - from];
        }
    if (threadIdx.x == 0) sh.n_list = over ? 0 : n;
    __syncthreads();
    return over ? 0xffffffffu : n;
}

// After a kCollect: the boundary, the draw, or the next step.  Returns true when done.
template <typename T>
__device__ __noinline__ bool after_collect(const Row<T>& r, Search& P, Cmd& cmd, u64* cw,
                                           uint32_t* cn, u64* own_w, uint32_t* own_n, int ranks,
                                           const SampleArgs& a, int64_t row_i, SampleFraction u,
                                           Shared& sh) {
    u64 above = 0;
    uint32_t inside = 0;
    const uint32_t n = merge(r, cmd, cw, cn, own_w, own_n, ranks, P.draw, above, inside, sh);
    if (P.draw) {
        search_draw(r, P, cmd, cw, cn, a, row_i, u, sh);
        return true;
    }
    take_total(P, cmd, ranks, sh);
    if (n == 0xffffffffu) {              // the list did not hold the window
        next_hist(cmd);
        return false;
    }
    const uint32_t key_top = min(cmd.khi, order_key(r.ws.m));
    u64 list_w = 0;
    if (cmd.list && (!P.want_k || P.top_k - P.n_above > n)) {
        u64 mine = 0;
        for (uint32_t i = threadIdx.x; i < n; i += kSearch)
            mine += fixed_weight(key_value(sh.key[i]), r.ws, sh.table);
        list_w = block_scan<kSearch>(mine, 0, sh.part, sh.part_n).tv;
    } else if (!cmd.list) {
        list_w = inside * fixed_weight(key_value(cmd.klo), r.ws, sh.table);
    }
    bool settled = false;                // the need lies in this window
    if (P.want_k) {
        const u64 left = P.top_k - P.n_above;
        u64 up_w = 0;
        if (cmd.list && left > n) {      // all that is not -inf
            P.key = kKeyNegInf;
            P.ties = 0;
            up_w = list_w;
        } else if (cmd.list) {
            const Selected at = list_select(r, false, left, cmd.klo, key_top, sh);
            P.key = at.key;
            P.ties = left - at.n;
            up_w = at.w;
        } else {
            P.key = cmd.klo;
            P.ties = left;
        }
        P.want_k = false;
        if (P.want_p) {
            const u64 wt = P.ties == 0 ? 0 : fixed_weight(key_value(P.key), r.ws, sh.table);
            P.exact = true;
            P.s_lo = P.s_hi = above + up_w + P.ties * wt;
            if (P.need(P.s_lo) <= above) {   // the nucleus ends above this window
                start_p(P, cmd);
                return false;
            }
            settled = true;
        }
    }
    if (P.want_p) {
        const u64 need = P.need(P.s_lo);     // exact by now
        if (need <= above || (!settled && need > above + list_w)) {
            // cannot be: the window was drawn around every total within its bounds
            P.key = kKeyNegInf;
            P.ties = 0;
            ask_draw(P, cmd);
            return false;
        }
        Selected at{cmd.klo, 0, 0};
        if (cmd.list) at = list_select(r, true, need - above, cmd.klo, key_top, sh);
        const u64 wt = fixed_weight(key_value(at.key), r.ws, sh.table);
        P.key = at.key;
        P.ties = wt == 0 ? 0 : (need - above - at.w + wt - 1) / wt;
        P.want_p = false;
    }
    if (P.key_m > P.key) {
        P.key = P.key_m - 1;
        P.ties = 0;
        // elements above the window are not told apart: min_p may cut among them
        if (!cmd.list || above != 0) {
            ask_draw(P, cmd);
            return false;
        }
    }
    search_draw(r, P, cmd, cw, cn, a, row_i, u, sh);
    return true;
}

// Floats and integers behind Shared in dynamic shared memory, for nch chunks of which a
// block owns `own`.
__host__ __device__ constexpr size_t search_smem(int nch, int own) {
    return sizeof(Shared) + size_t(nch) * 16 + size_t(own) * 12 + 16;
}

template <typename T>
__device__ __forceinline__ void search_row(const T* logits, const SampleArgs& a, int64_t row_i,
                                           int rank, int ranks, int nch, int own, u64* cw,
                                           u64* own_w, float* cmax, uint32_t* cn, uint32_t* own_n,
                                           Shared& sh) {
    const int tid = threadIdx.x;
    const RowHeader* head = static_cast<const RowHeader*>(a.workspace) + row_i;
    const Settings s = read_settings(a, row_i);
    Row<T> r = make_row(logits, a, row_i, s, nch, own, rank);
    r.ws.m = head->m;
    const float2* stats = row_stats(a, row_i, nch);
    for (int i = tid; i < nch; i += kSearch) cmax[i] = stats[i].x;
    if (tid == 0) sh.key_m = s.want_m ? min_p_key(a, row_i, r.ws.m) : 0;
    __syncthreads();

    Search P;
    P.want_k = s.want_k;
    P.want_p = s.want_p;
    P.draw = P.exact = false;
    P.n_above = 0;
    P.all = head->all;
    total_bounds(P.all, a.V, P.s_lo, P.s_hi);
    P.key = kKeyNegInf;
    P.ties = 0;
    P.key_m = sh.key_m;
    P.top_k = static_cast<u64>(s.top_k);
    P.top_p = s.top_p;
    Cmd cmd;
    if (!P.want_k && !P.want_p) {
        ask_draw(P, cmd);
    } else if (a.V <= kList) {           // the whole row fits the list
        cmd = Cmd{kCollect, kKeyNegInf + 1, 0xffffffffu, 0, 0, 1, 0};
    } else {
        cmd = make_hist0(!P.want_k);
    }
    cmd.total = P.want_p && !P.want_k && cmd.type == kCollect;
    // the blocks work on their chunks, block 0 decides what comes next
    for (int step = 0; step < kMaxSteps; ++step) {
        if (cmd.type == kHist)
            step_hist(r, cmd, cmax, sh);
        else
            step_collect(r, cmd, cmax, own_w, own_n, sh);
        cluster_join();
        if (rank == 0) {
            bool done = false;
            if (cmd.type == kHist)
                after_hist(r, P, cmd, ranks, sh);
            else
                done = after_collect(r, P, cmd, cw, cn, own_w, own_n, ranks, a, row_i, s.u, sh);
            if (done) cmd.type = kDone;
            // top_p refers to the exact total: formed on the way, in a pass that is made anyway
            cmd.total = P.want_p && !P.want_k && !P.exact &&
                        !(cmd.type == kHist && cmd.shift < 0);
            if (!done && step == kMaxSteps - 1 && tid == 0)
                write_failed(a, row_i, RLK_DEVERR_WAIT_TIMEOUT);
            __syncthreads();
            if (tid == 0) sh.cmd = cmd;
        }
        cluster_join();
        if (rank != 0) cmd = *peer(&sh.cmd, 0);
        if (cmd.type == kDone) break;
    }
    cluster_join();          // block 0's shared memory is read until here
}

template <typename T>
__global__ void __launch_bounds__(kSearch, 2)
    sample_search_kernel(const T* __restrict__ logits, const SampleArgs a, int nch, int own,
                         int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    u64* cw = reinterpret_cast<u64*>(smem + sizeof(Shared));     // all chunks: weight
    u64* own_w = cw + nch;                                       // own chunks
    float* cmax = reinterpret_cast<float*>(own_w + own);         // all chunks: maximum
    uint32_t* cn = reinterpret_cast<uint32_t*>(cmax + nch);      //             ties
    uint32_t* own_n = cn + nch;
    const int rank = blockIdx.x % ranks, tid = threadIdx.x;
    wait_previous(logits);               // the scan's results are complete
    const uint32_t* modes = row_modes(a);
    bool table = false;
    for (int base = 0; base < a.N; base += kSearch) {
        uint32_t group;
        const bool any = queue_rows<kSearch, false>(modes, a.N, base, ranks, group, sh.queue, sh.part,
                                                    sh.part_n) > 0;
        const uint32_t n = any ? sh.queue.n : 0;
        if (n > 0 && !table) {
            for (int i = tid; i < kExpEntries; i += kSearch) sh.table[i] = kExpTable.v[i];
            table = true;
        }
        for (uint32_t i = 0; i < n; ++i)
            search_row(logits, a, int64_t(base) + sh.queue.at[i], rank, ranks, nch, own, cw, own_w,
                       cmax, cn, own_n, sh);
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------- exact draw

// The second launch of a call without any truncation: its rows are those whose target lies near
// a border, few of them, and what counts is how soon each is done: 1024 threads a block, up to 8
// blocks a row (12 to 22 us for the 10 to 25 rows of [256, 151936]).  With more rows than clusters, a
// row gets fewer blocks ([1024, 151936] 139 us, 168 with 8 each).  Every weight of the row is
// formed exactly; a warp takes 128 columns at a time.
struct Shared1 {
    u64 table[kExpEntries];
    u64 part[kExact / 32];
    uint32_t part_n[kExact / 32];
    u64 at_w;
    int at;
    Queue queue;
};
__host__ __device__ constexpr size_t exact_smem(int nch) {
    return sizeof(Shared1) + size_t(nch) * 8 + 16;
}

template <typename T>
__global__ void __launch_bounds__(kExact, 1)
    sample_exact_kernel(const T* __restrict__ logits, const SampleArgs a, int nch, int, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared1& sh = *reinterpret_cast<Shared1*>(smem);
    u64* own_w = reinterpret_cast<u64*>(smem + sizeof(Shared1));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kExpEntries; i += kExact) sh.table[i] = kExpTable.v[i];
    wait_previous(logits);               // the scan's results are complete
    constexpr int kUnit = 128, kPerChunk = kChunk / kUnit, kAhead = 5, kUnits = kExact / 32;
    for (int base = 0; base < a.N; base += kExact) {
        uint32_t group = 1;
        const uint32_t n = queue_rows<kExact, true>(row_modes(a), a.N, base, ranks, group, sh.queue,
                                                    sh.part, sh.part_n);
        const int own = (nch + group - 1) / group;
        const uint32_t rank = blockIdx.x % group, first = blockIdx.x % ranks - rank;
        // the blocks of a cluster keep step: the last time a group may be without a row
        for (uint32_t q = 0; q < n; ++q) {
            const bool on = q < sh.queue.n;
            if (!on) {
                cluster_join();
                cluster_join();
                continue;
            }
            const int64_t row_i = int64_t(base) + sh.queue.at[q];
            const Settings s = read_settings(a, row_i);
            Row<T> r = make_row(logits, a, row_i, s, nch, own, rank);
            r.ws.m = (static_cast<const RowHeader*>(a.workspace) + row_i)->m;
            for (int i = tid; i < own; i += kExact) own_w[i] = 0;
            __syncthreads();
            const int units = r.mine * kPerChunk;
#pragma unroll 1
            for (int u0 = warp; u0 < units; u0 += kAhead * kUnits) {
                float x[kAhead][4];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int u = u0 + k * kUnits;
                    if (u >= units) break;
                    const int c = r.first * kChunk + u * kUnit + lane * 4;
                    if (sizeof(T) == 4 && r.vec && c + 4 <= r.V) {
                        const float4 v = __ldg(reinterpret_cast<const float4*>(r.x + c));
                        x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
                    } else if (sizeof(T) == 2 && r.vec && c + 4 <= r.V) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(r.x + c));
                        x[k][0] = __uint_as_float(v.x << 16);
                        x[k][1] = __uint_as_float(v.x & 0xffff0000u);
                        x[k][2] = __uint_as_float(v.y << 16);
                        x[k][3] = __uint_as_float(v.y & 0xffff0000u);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[k][e] = c + e < r.V ? load_one(r.x + c + e) : -INFINITY;
                    }
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int u = u0 + k * kUnits;
                    if (u >= units) break;
                    u64 w[4];
                    fixed_weights(make_float2(x[k][0], x[k][1]), r.ws, sh.table, w[0], w[1]);
                    fixed_weights(make_float2(x[k][2], x[k][3]), r.ws, sh.table, w[2], w[3]);
                    const u64 sum = warp_sum((w[0] + w[1]) + (w[2] + w[3]));
                    if (lane == 0) atomicAdd(&own_w[u / kPerChunk], sum);
                }
            }
            __syncthreads();
            cluster_join();
            if (rank == 0) {
                // the chunk, then the column, that u times the total falls on
                const int each = (nch + kExact - 1) / kExact;
                const int c0 = min(nch, tid * each), c1 = min(nch, c0 + each);
                u64 w = 0;
                for (int c = c0; c < c1; ++c) w += peer(own_w, first + c / own)[c % own];
                const Scanned t = block_scan<kExact>(w, 0, sh.part, sh.part_n);
                const u64 target = part_of(s.u, t.tv, false);
                if (tid == 0) sh.at = 0, sh.at_w = 0;
                __syncthreads();
                u64 run = t.v;
                for (int c = c0; c < c1; ++c) {
                    const u64 cw = peer(own_w, first + c / own)[c % own];
                    if (run <= target && target < run + cw) sh.at = c, sh.at_w = run;
                    run += cw;
                }
                __syncthreads();
                const int col = sh.at * kChunk + tid;
                const float x = tid < kChunk && col < r.V ? load_one(r.x + col) : -INFINITY;
                const u64 we = fixed_weight(x, r.ws, sh.table);
                const u64 lo = sh.at_w + block_scan<kExact>(we, 0, sh.part, sh.part_n).v;
                if (lo <= target && target < lo + we)
                    write_drawn(a, row_i, col, x, r.ws, t.tv, t.tv);
            }
            cluster_join();              // the blocks' sums are read until here
        }
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_rows(void (*kernel)(const T*, const SampleArgs, int, int, int),
                        const T* logits, const SampleArgs& a, int nch, int ranks, int clusters,
                        int threads, size_t smem, cudaStream_t stream) {
    const int own = (nch + ranks - 1) / ranks;
    // Always the most that any vocabulary needs: another thread's call with a smaller one may come
    // between this and the launch.
    constexpr int kMaxChunks = (1 << 22) / kChunk, kMost = 227 * 1024;
    static_assert(scan_smem(kMaxChunks, kMaxSegments) <= kMost && exact_smem(kMaxChunks) <= kMost &&
                      search_smem(kMaxChunks, (1 << 20) / kChunk) <= kMost,
                  "a block's shared memory");
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ranks;
    cluster.val.clusterDim.y = 1;
    cluster.val.clusterDim.z = 1;
    return launch_early(kernel, dim3(static_cast<unsigned>(clusters) * ranks), threads, smem,
                        stream, &cluster, logits, a, nch, own, ranks);
}

template <typename T>
cudaError_t launch_typed(const T* logits, const SampleArgs& args, cudaStream_t stream) {
    const int nch = (args.V + kChunk - 1) / kChunk;
    SampleArgs a = args;
    a.parts = parts_of(nch, a.top_k_rows != nullptr ? 0 : a.top_k, sizeof(T));
    const int nseg = segments_of(nch, a.parts, sizeof(T));
    const int ranks = nch >= 128 ? 8 : nch >= 64 ? 4 : nch >= 32 ? 2 : 1;
    if (int64_t(a.N) * ranks > 0x7fffffff) return cudaErrorInvalidValue;
    // As many blocks a row as run at the same time, four on each of 152 SMs: more of them, one
    // after the other, start anew with nothing on its way (with 8 at V = 151936, [256] fp32 takes
    // 56.5 instead of 53.8 us, [1024] 148 instead of 139, [1024] bf16 with top_k and top_p 145
    // instead of 96).
    int scan_ranks = ranks;
    while (scan_ranks > 1 && int64_t(a.N) * scan_ranks > 608) scan_ranks /= 2;
    cudaError_t e = launch_rows(sample_scan_kernel<T>, logits, a, nch, scan_ranks, a.N, kThreads,
                                scan_smem(nch, nseg), stream);
    if (e != cudaSuccess) return e;
    if (a.top_k_rows == nullptr && a.top_p_rows == nullptr && a.min_p_rows == nullptr &&
        (a.top_k == 0 || a.top_k >= a.V) && a.top_p_value >= 1.f && a.min_p_value == 0.f) {
        // One block on each of 152 SMs, which may come to weigh a whole row.
        return launch_rows(sample_exact_kernel<T>, logits, a, nch, ranks,
                           std::min(a.N, 152 / ranks), kExact, exact_smem(nch), stream);
    }
    // The search: two blocks on each of 152 SMs, and smaller clusters where more rows than clusters
    // are to be expected: nearly all rows where a wide nucleus is all that cuts, about a fifth where
    // each row brings its own settings, few otherwise.  V = 151936, top_p alone, with 8, 4, 2 and 1
    // blocks a row: fp32 [1] 56, 67, 94, 143 us; [64] 200, 164, 188, 276; [256] 735, 463, 420, 449;
    // bf16 [256] 672, 421, 355, 390.
    const bool own_settings =
        a.top_k_rows != nullptr || a.top_p_rows != nullptr || a.min_p_rows != nullptr;
    const bool listed =
        a.min_p_value > 0.f || (a.top_k > 0 && a.top_k <= nseg / 2);
    const int64_t expected = own_settings ? a.N / 4 : listed ? 0 : a.N;
    // A block's share stays below 2^20 columns, whose codes of 4096 would overflow a bin.
    const auto share = [nch](int blocks) { return (nch + blocks - 1) / blocks * kChunk; };
    int search_ranks = ranks;
    while (search_ranks > 2 && expected * search_ranks > 304 &&
           share(search_ranks / 2) < (1 << 20))
        search_ranks /= 2;
    return launch_rows(sample_search_kernel<T>, logits, a, nch, search_ranks,
                       std::min(a.N, 304 / search_ranks), kSearch,
                       search_smem(nch, (nch + search_ranks - 1) / search_ranks), stream);
}

}  // namespace

size_t sample_workspace(int64_t N, int64_t V) {
    const int nch = static_cast<int>((V + kChunk - 1) / kChunk);
    return segs_offset(N, nch) + size_t(N) * segs_stride(nch) * sizeof(float);
}

cudaError_t launch_sample(const void* logits, bool bf16, const SampleArgs& args,
                          cudaStream_t stream) {
    if (bf16)
        return launch_typed(static_cast<const __nv_bfloat16*>(logits), args, stream);
    return launch_typed(static_cast<const float*>(logits), args, stream);
}

}  // namespace rlk
