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
// Two launches.  The scan: a cluster of up to 8 blocks a row, a warp a chunk of 512
// columns; per chunk its maximum and an fp32 sum of 2^((x - chunk max) c), c = log2(e)/T,
// go to the workspace.  This is the only pass over HBM.  The cluster's block 0 then forms
// the chunks' weights as integers, in the same order whatever the split, and finishes the
// rows that need no further pass over all columns:
//
//   no truncation: the chunk and the element that u times the total falls on come from the
//   fast weights, together with a bound on their error (kFastErr); only when the target lies
//   within it of a border of the running sums -- some percent of the rows at V ~ 150k --
//   does the row go on to the search, which weighs it exactly.
//
//   truncation: elements from some value on are gathered from the chunks whose maximum
//   reaches it, and their order is counted out in place.  The value is one that K chunk
//   maxima reach (top_k), that chunk maxima of top_p of the total reach, or min_p's own; in
//   rows in no particular order few other elements reach it.
//
// The search takes the rows that are left (a wide nucleus, a large top_k, a row sorted by
// token, a target near a border), again a cluster a row: histograms of 2048 bins of the
// scaled distance from the maximum, then of the keys inside the remaining window, close in
// on the boundary until its window fits a list or is a single value.  Block 0 of the
// cluster decides each step; the blocks work on their own chunks in between.
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"
#include "weight_exp.cuh"

namespace rlk {

namespace {

typedef unsigned long long u64;

constexpr int kChunk = 512;              // columns of a chunk
constexpr int kLane = kChunk / 32;       // of a lane
constexpr int kBins = 2048;
constexpr int kList = 1024;              // elements of the search's list
constexpr int kShort = 512;              // of the scan's list, counted out in place
constexpr int kThreads = 256;
constexpr float kRange = 48.f;           // weights below 2^-48 round to 0 (bits <= 46)
constexpr int kMaxSteps = 32;            // far more than any row takes
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf)

// The fast weights' relative error, in units of 2^-24: 4 for ex2.approx, 9 roundings of a
// chunk's sum, and log(2) t_i (1 for x - max, 2 for the product with a rounded c) for each
// element: the weighted mean of t over 512 elements with sum s >= 1 is at most
// log2(512 / s) <= 9, so 19; another 9 between a chunk's sum and the sums of its parts.
// 42 in all, with the factor 2 u (1 - u) that a relative error of all weights leaves of
// sum(prefix) - u sum(all) at its zero.
constexpr float kFastErr = 42.f / 16777216.f;
constexpr float kBinErr = 1.f / 4096.f;  // of a histogram's weight: 12-bit codes

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
__device__ __forceinline__ u64 part_of(double f, u64 s, bool up) {
    u64 mant;
    int shift;
    bool rest;
    split_unit(f, mant, shift);
    const u64 r = mul_floor(mant, shift, s, rest);
    return r + (up && rest ? 1 : 0);
}
// floor(w * f) of a float 0 <= w <= 512 and an integer f <= 2^46, to 2^-40 of itself
__device__ __forceinline__ u64 scale_weight(float w, u64 f) {
    const uint32_t b = __float_as_uint(w);
    const int e = int(b >> 23);
    if (e == 0) return 0;
    const int shift = 150 - e - 6;             // w = mant 2^-(150 - e)
    if (shift > 63) return 0;
    return ((f >> 6) * u64((b & 0x7fffffu) | 0x800000u)) >> shift;
}

// the same shared object in block `rank` of the cluster (generic address)
template <typename P>
__device__ __forceinline__ P* peer(P* p, uint32_t rank) {
    u64 a;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(p)), "r"(rank));
    return reinterpret_cast<P*>(a);
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

// cluster barrier of converged warps
__device__ __forceinline__ void cluster_join() {
    __syncwarp();
    cluster_sync();
}

// ----------------------------------------------------------------------------- chunks

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
        for (int j = 0; j < LOADS; ++j) {
            const int c = column(chunk, j, lane);
            if (vec && c + VEC <= V) {
                raw[j] = __ldg(reinterpret_cast<const uint4*>(row + c));
            } else {
                T v[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = c + e < V ? row[c + e] : T(-INFINITY);
                raw[j] = *reinterpret_cast<const uint4*>(v);
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(raw);
            return __uint_as_float(p[i]);
        }
        const uint32_t* p = reinterpret_cast<const uint32_t*>(raw);
        return __uint_as_float((i & 1) ? (p[i / 2] & 0xffff0000u) : (p[i / 2] << 16));
    }
};

// A step that block 0 asks of all blocks.  Elements are above, inside or below a window:
// bins [b1, b2] of the scaled distance from the maximum, and keys [klo, khi] in them.
enum : int { kHist, kCollect, kDone };
struct Cmd {
    int type;
    int b1, b2;
    uint32_t klo, khi;
    int shift;        // kHist: bins of the keys, (khi - key) >> shift; -1: of the distance
    int by_weight;    // kHist: 12-bit weights instead of counts
    int list;         // kCollect: 1 lists the elements inside, 0 counts them per chunk
};

// Shared memory of the scan.
struct Shared0 {
    u64 table[kExpEntries];
    u64 w[kShort];
    uint32_t key[kShort], idx[kShort];
    u64 part[32];
    uint32_t part_n[32];
    u64 at_w;
    uint32_t n_list, n_ids, flag;
    int at;
};

// Workspace: a header a row, then the chunks' maxima and sums.
enum : uint32_t { kRowDone, kRowSearch };
struct RowHeader {
    u64 all;                             // fast total of the weights
    float m;                             // maximum
    uint32_t mode;
};
__host__ __device__ constexpr size_t stats_offset(int64_t N) {
    return (size_t(N) * sizeof(RowHeader) + 255) / 256 * 256;
}
__device__ __forceinline__ float2* row_stats(const SampleArgs& a, int64_t row, int nch) {
    return reinterpret_cast<float2*>(static_cast<uint8_t*>(a.workspace) + stats_offset(a.N)) +
           row * nch;
}

// Shared memory of the search.
struct Shared {
    u64 table[kExpEntries];
    u64 w[kList];                        // block 0: the merged list
    uint32_t key[kList], idx[kList];
    uint32_t own_key[kList], own_idx[kList];   // this block's part of it
    uint32_t hist[kBins];
    uint32_t cnt[256], lo[256], hi[256];
    u64 part[32];
    uint32_t part_n[32];
    u64 own_above;                       // exact weight above the window, all own chunks
    uint32_t own_count;
    uint32_t n_list;
    // results of block-wide searches
    u64 at_w;
    uint32_t at_n, at_n2;
    int at, at2;
    Cmd cmd;
};

// What a row's blocks know of it.
template <typename T>
struct Row {
    const T* x;
    int V, nch, own, first, mine;        // chunks: all, a block's share, this block's
    bool vec;
    WeightScale ws;
    float scale;                         // bins per unit of distance
    int bits;
};

template <int THREADS>
struct Block {
    static constexpr int kWarps = THREADS / 32;

    // exclusive prefix of v and n over the block's threads; totals in tv, tn
    template <typename S>
    __device__ static void scan(u64& v, uint32_t& n, u64& tv, uint32_t& tn, S& sh) {
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
        if (lane == 31) sh.part[warp] = iv, sh.part_n[warp] = in;
        __syncthreads();
        u64 bv = 0;
        uint32_t bn = 0;
        tv = 0, tn = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i == warp) bv = tv, bn = tn;
            tv += sh.part[i], tn += sh.part_n[i];
        }
        v = bv + iv - v;
        n = bn + in - n;
    }
};

template <typename T>
__device__ __forceinline__ int dist_bin(float x, const Row<T>& r) {
    // monotone in x; kBins and more: weight 0
    return static_cast<int>(fminf((r.ws.m - x) * r.scale, 2.f * kBins));
}

// ----------------------------------------------------------------------------- steps

// Histogram of the window; for windows of keys also the exact weight above it.
template <typename T, int THREADS>
__device__ void step_hist(const Row<T>& r, const Cmd& cmd, const float* cmax, Shared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kBins; i += THREADS) sh.hist[i] = 0;
    if (threadIdx.x == 0) sh.own_above = 0;
    __syncthreads();
    const float unit = kRange / kBins;
    const float x_hi = key_value(cmd.khi);
    u64 above = 0;
    for (int i = warp; i < r.mine; i += THREADS / 32) {
        const float top = cmax[r.first + i];
        if (dist_bin(top, r) > min(cmd.b2, kBins - 1) ||
            (cmd.shift >= 0 && order_key(top) < cmd.klo))
            continue;
        Chunk<T> c;
        c.load(r.x, r.V, r.first + i, lane, r.vec);
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const float x = c.get(e);
            const float t = fminf((r.ws.m - x) * r.scale, 2.f * kBins);
            const int b = static_cast<int>(t);
            if (b >= kBins || b > cmd.b2) continue;
            if (cmd.shift < 0) {
                const float q = cmd.by_weight ? rintf(4096.f * ex2_approx((b - t) * unit)) : 1.f;
                atomicAdd(&sh.hist[b], static_cast<uint32_t>(q));
                continue;
            }
            const uint32_t k = order_key(x);
            if (b < cmd.b1 || k > cmd.khi) {
                if (cmd.by_weight) above += fixed_weight(x, r.ws, sh.table);
            } else if (k >= cmd.klo) {
                const float q =
                    cmd.by_weight ? rintf(4096.f * ex2_approx((x - x_hi) * r.ws.ch)) : 1.f;
                atomicAdd(&sh.hist[(cmd.khi - k) >> cmd.shift], static_cast<uint32_t>(q));
            }
        }
    }
    above = warp_sum(above);
    if (lane == 0 && above != 0) atomicAdd(&sh.own_above, above);
    __syncthreads();
}

// Exact weight above the window, per chunk, and the elements inside it.
template <typename T, int THREADS>
__device__ void step_collect(const Row<T>& r, const Cmd& cmd, const float* cmax, u64* own_w,
                             uint32_t* own_n, Shared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) sh.own_count = 0;
    __syncthreads();
    for (int i = warp; i < r.mine; i += THREADS / 32) {
        const float top = cmax[r.first + i];
        u64 w = 0;
        uint32_t n = 0;
        if (dist_bin(top, r) <= cmd.b2 && order_key(top) >= cmd.klo) {
            Chunk<T> c;
            c.load(r.x, r.V, r.first + i, lane, r.vec);
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const float x = c.get(e);
                const int b = dist_bin(x, r);
                const uint32_t k = order_key(x);
                if (b > cmd.b2 || k < cmd.klo || k <= kKeyNegInf) continue;
                if (b < cmd.b1 || k > cmd.khi) {
                    w += fixed_weight(x, r.ws, sh.table);
                } else if (cmd.list) {
                    const uint32_t at = atomicAdd(&sh.own_count, 1u);
                    if (at < kList) {
                        sh.own_key[at] = k;
                        sh.own_idx[at] = Chunk<T>::column(r.first + i, e / Chunk<T>::VEC, lane) +
                                         e % Chunk<T>::VEC;
                    }
                } else {
                    ++n;
                }
            }
            w = warp_sum(w);
            n = warp_sum(n);
        }
        if (lane == 0) own_w[i] = w, own_n[i] = n;
    }
    __syncthreads();
}

// ----------------------------------------------------------------------------- block 0

// Radix selection in the merged list: the key at which the count (or weight) of the
// elements from the top reaches `need` >= 1, and what lies above that key.
template <int THREADS>
__device__ void list_select(bool by_weight, u64 need, Shared& sh, uint32_t& key, u64& above,
                            uint32_t& above_n, u64& above_w) {
    uint32_t prefix = 0;
    u64 n_up = 0, w_up = 0;
    for (int level = 3; level >= 0; --level) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += THREADS) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
        const uint32_t mask = level == 3 ? 0u : 0xffffffffu << (8 * (level + 1));
        for (uint32_t i = threadIdx.x; i < sh.n_list; i += THREADS) {
            const uint32_t k = sh.key[i];
            if ((k & mask) != prefix) continue;
            const uint32_t b = (k >> (8 * level)) & 255u;
            atomicAdd(&sh.cnt[b], 1u);
            const u64 w = sh.w[i];
            const uint32_t wl = static_cast<uint32_t>(w);
            const uint32_t old = atomicAdd(&sh.lo[b], wl);
            atomicAdd(&sh.hi[b], static_cast<uint32_t>(w >> 32) + (old + wl < old ? 1u : 0u));
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            // lane l holds bins 255 - 8 l .. 248 - 8 l, from the top down
            const int top = 255 - 8 * int(threadIdx.x);
            u64 w = 0;
            uint32_t n = 0;
            for (int j = 0; j < 8; ++j) {
                w += (u64(sh.hi[top - j]) << 32) | sh.lo[top - j];
                n += sh.cnt[top - j];
            }
            u64 iw = w;
            uint32_t in = n;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 ow = __shfl_up_sync(0xffffffffu, iw, off);
                const uint32_t on = __shfl_up_sync(0xffffffffu, in, off);
                if (threadIdx.x >= off) iw += ow, in += on;
            }
            const bool reached = by_weight ? w_up + iw >= need : n_up + in >= need;
            const unsigned who = __ballot_sync(0xffffffffu, reached);
            const int first = who == 0 ? 31 : __ffs(who) - 1;
            if (int(threadIdx.x) == first) {
                u64 cw = w_up + iw - w, cn = n_up + in - n;
                int b = top;
                for (int j = 0; j < 8; ++j, --b) {
                    const u64 bw = (u64(sh.hi[b]) << 32) | sh.lo[b];
                    if (j == 7 || (by_weight ? cw + bw : cn + sh.cnt[b]) >= need) break;
                    cw += bw;
                    cn += sh.cnt[b];
                }
                sh.at = b;
                sh.at_w = cw;
                sh.at_n = static_cast<uint32_t>(cn);
            }
        }
        __syncthreads();
        prefix |= uint32_t(sh.at) << (8 * level);
        w_up = sh.at_w;
        n_up = sh.at_n;
    }
    key = prefix;
    above = by_weight ? w_up : n_up;
    above_n = static_cast<uint32_t>(n_up);
    above_w = w_up;
    __syncthreads();
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ void write_row(const SampleArgs& a, int64_t row, int64_t token,
                                          float logp, float kept_logp) {
    a.tokens[row] = token;
    if (a.logp != nullptr) a.logp[row] = logp;
    if (a.kept_logp != nullptr) a.kept_logp[row] = kept_logp;
}

// log of sum / 2^bits; the largest weight is 2^bits, so sum >= 2^bits
__device__ __forceinline__ float log_of(u64 sum, int bits) {
    return log1pf(static_cast<float>(sum - (u64(1) << bits)) *
                  exp2f(static_cast<float>(-bits)));
}

__device__ __forceinline__ void write_drawn(const SampleArgs& a, int64_t row, int v, float x,
                                            float m, double temp, u64 all, u64 kept, int bits) {
    const double z = (static_cast<double>(x) - static_cast<double>(m)) / temp;
    write_row(a, row, v, static_cast<float>(z - log_of(all, bits)),
              static_cast<float>(z - log_of(kept, bits)));
}

// What block 0 carries from step to step (uniform over its threads).
struct Search {
    bool want_k, want_p;       // boundaries still to be found
    bool draw;                 // the next kCollect is the last
    bool sum;                  // the next kCollect is the exact total
    bool exact;                // s_lo == s_hi is the exact weight that top_p refers to
    int level;                 // histograms of this search so far
    u64 n_above;               // count above the window (want_k)
    u64 s_lo, s_hi;            // bounds of the total that top_p refers to
    uint32_t key;              // the boundary so far
    u64 ties;
    uint32_t key_m;            // elements below are cut by min_p
};

__device__ __forceinline__ Cmd make_hist0(bool by_weight) {
    return Cmd{kHist, 0, kBins - 1, 0u, 0xffffffffu, -1, by_weight ? 1 : 0, 0};
}
__device__ __forceinline__ Cmd make_above(uint32_t key) {
    return Cmd{kCollect, 0, 2 * kBins, key, key, 0, 0, 0};
}

template <typename T, int THREADS>
struct Sampler {
    typedef Block<THREADS> B;

    // Narrows the window from the histogram (merged over the cluster) and asks for the next
    // step.  P.level counts the histograms, this one included.
    __device__ static void after_hist(const Row<T>& r, Search& P, Cmd& cmd, double top_p,
                                      u64 top_k, uint32_t ranks, Shared& sh) {
        constexpr int kPer = kBins / THREADS;
        const int b0 = threadIdx.x * kPer;
        u64 q[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) q[i] = 0;
        u64 above = 0;
        for (uint32_t k = 0; k < ranks; ++k) {
            const uint32_t* h = peer(sh.hist, k);
#pragma unroll
            for (int i = 0; i < kPer; ++i) q[i] += h[b0 + i];
            above += *peer(&sh.own_above, k);
        }
        u64 mine = 0, total, qsum = 0;
        uint32_t dummy = 0, tn;
        const bool keys = cmd.shift >= 0, single = cmd.shift == 0;
        const float unit = kRange / kBins;
        const u64 w_hi = keys ? fixed_weight(fminf(key_value(cmd.khi), r.ws.m), r.ws, sh.table) : 0;
        u64 weight[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            qsum += q[i];
            if (!cmd.by_weight) {
                weight[i] = q[i];
            } else if (!keys) {
                weight[i] = __float2ull_rn(static_cast<float>(q[i]) *
                                           ex2_approx(-(b0 + i) * unit + (r.bits - 12)));
            } else if (single) {
                // one value a bin: its code tells the count, and the weight is exact
                const uint32_t k = cmd.khi - (b0 + i);
                weight[i] = 0;
                if (q[i] != 0) {
                    const float x = key_value(k);
                    const float code =
                        rintf(4096.f * ex2_approx((x - key_value(cmd.khi)) * r.ws.ch));
                    weight[i] = q[i] / static_cast<u64>(code) * fixed_weight(x, r.ws, sh.table);
                }
            } else {
                weight[i] = scale_weight(static_cast<float>(q[i]) * (1.f / 4096.f / 4096.f),
                                         w_hi) << 12;
            }
            mine += weight[i];
        }
        u64 before = mine;
        B::scan(before, dummy, total, tn, sh);
        // the first bins at which the running sum surely may, and surely must, have reached
        // the need
        if (threadIdx.x == 0) sh.at = sh.at2 = kBins, sh.at_w = 0, sh.at_n = 0;
        __syncthreads();
        u64 need_lo, need_hi, base;
        float err = 0.f;
        if (P.want_k) {
            need_lo = need_hi = top_k;
            base = P.n_above;
        } else {
            need_lo = max(u64(1), part_of(top_p, P.s_lo, true));
            need_hi = max(u64(1), part_of(top_p, P.s_hi, true));
            base = above;
            err = single ? 0.f : kBinErr;
        }
        u64 run = before;
        int first_may = kBins, first_must = kBins;
        u64 at_before = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const u64 prev = run;
            run += weight[i];
            const u64 slack = static_cast<u64>(static_cast<float>(run) * err) + (err > 0.f ? 4096 : 0);
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
        const bool found = sh.at < kBins;
        const int j1 = min(sh.at, kBins - 1), j2 = max(j1, min(sh.at2, kBins - 1));
        const u64 skipped = sh.at_w;
        // elements of the new window (codes of a window are near 4096 unless it is wide)
        u64 est = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (b0 + i >= j1 && b0 + i <= j2) est += q[i];
        u64 est_all;
        B::scan(est, dummy, est_all, tn, sh);
        if (cmd.by_weight) est_all = est_all / 3600 + 1;
        if (!found) {
            // fewer elements of weight > 0 than top_k: nothing is cut (a weight is always
            // reached)
            if (P.want_k) {
                P.want_k = false;
                P.key = kKeyNegInf;
                P.ties = 0;
                start_p(r, P, cmd, top_p);
            } else {
                P.draw = true;
                P.key = kKeyNegInf;
                P.ties = 0;
                finish(P, cmd);
            }
            return;
        }
        if (P.want_k) P.n_above += skipped;
        if (!keys) {
            cmd.b1 = j1;
            cmd.b2 = j2;
            const double s = r.scale, m = r.ws.m, pad = fabs(m) * 2.4e-7 + 1e-37;
            const double lo = m - (j2 + 1) / s * (1.0 + 1e-6) - pad;
            const double hi = m - j1 / s * (1.0 - 1e-6) + pad;
            cmd.klo = max(kKeyNegInf + 1, order_key(static_cast<float>(fmax(lo, -3.4028234663852886e38))) - 1);
            cmd.khi = min(order_key(r.ws.m), order_key(static_cast<float>(hi)) + 1);
        } else {
            const int64_t hi = int64_t(cmd.khi) - (int64_t(j1) << cmd.shift);
            const int64_t lo = int64_t(cmd.khi) - (int64_t(j2 + 1) << cmd.shift) + 1;
            cmd.klo = static_cast<uint32_t>(max(int64_t(cmd.klo), lo));
            cmd.khi = static_cast<uint32_t>(hi);
        }
        if (cmd.klo == cmd.khi || est_all <= kList) {
            cmd.type = kCollect;
            cmd.list = cmd.klo == cmd.khi ? 0 : 1;
            return;
        }
        next_hist(P, cmd);
    }

    // a histogram of the window's keys; without the exact total its error would not let the
    // window shrink much further
    __device__ static void next_hist(Search& P, Cmd& cmd) {
        ++P.level;
        if (!P.want_k && P.level > 2 && !P.exact) {
            P.sum = true;
            cmd = make_above(0u);
            return;
        }
        cmd.type = kHist;
        const uint32_t span = cmd.khi - cmd.klo;
        cmd.shift = 0;
        while ((span >> cmd.shift) >= kBins) ++cmd.shift;
    }

    // the top_p search from its beginning, or the end of the search without top_p
    __device__ static void start_p(const Row<T>& r, Search& P, Cmd& cmd, double top_p) {
        if (P.want_p) {
            P.level = 1;
            cmd = make_hist0(true);
        } else {
            finish(P, cmd);
        }
    }

    // the boundary is known up to min_p: the last step
    __device__ static void finish(Search& P, Cmd& cmd) {
        P.want_p = false;
        if (P.key_m > P.key) P.key = P.key_m - 1, P.ties = 0;
        P.draw = true;
        cmd = make_above(P.key);
    }

    // block 0: all blocks' weights and counts per chunk, and the merged list
    __device__ static uint32_t merge(const Row<T>& r, const Cmd& cmd, u64* cw, uint32_t* cn,
                                     u64* own_w, uint32_t* own_n, uint32_t ranks, u64& above,
                                     uint32_t& inside, Shared& sh) {
        u64 mine = 0;
        uint32_t n_mine = 0;
        for (int c = threadIdx.x; c < r.nch; c += THREADS) {
            const int k = c / r.own, i = c - k * r.own;
            const u64 w = peer(own_w, k)[i];
            const uint32_t n = peer(own_n, k)[i];
            cw[c] = w;
            cn[c] = n;
            mine += w;
            n_mine += n;
        }
        B::scan(mine, n_mine, above, inside, sh);
        if (!cmd.list) return 0;
        uint32_t n = 0;
        bool over = false;
        for (uint32_t k = 0; k < ranks; ++k) {
            const uint32_t m = *peer(&sh.own_count, k);
            if (n + m > kList) {
                over = true;
                break;
            }
            const uint32_t* pk = peer(sh.own_key, k);
            const uint32_t* pi = peer(sh.own_idx, k);
            for (uint32_t i = threadIdx.x; i < m; i += THREADS) {
                const uint32_t key = pk[i];
                sh.key[n + i] = key;
                sh.idx[n + i] = pi[i];
                sh.w[n + i] = fixed_weight(key_value(key), r.ws, sh.table);
            }
            n += m;
        }
        if (threadIdx.x == 0) sh.n_list = over ? 0 : n;
        __syncthreads();
        return over ? 0xffffffffu : n;
    }

    // Draws from the kept set: cw[c] holds the chunks' weight above the window, cn[c] the
    // number of elements equal to P.key (list: both completed from the list here).
    __device__ static void draw(const Row<T>& r, const Search& P, const Cmd& cmd, u64* cw,
                                uint32_t* cn, const SampleArgs& a, int64_t row_i, float u,
                                double temp, u64 all, Shared& sh) {
        const int tid = threadIdx.x;
        if (cmd.list) {
            for (uint32_t i = tid; i < sh.n_list; i += THREADS) {
                const int c = sh.idx[i] / kChunk;
                if (sh.key[i] > P.key) atomicAdd(&cw[c], sh.w[i]);
                else if (sh.key[i] == P.key) atomicAdd(&cn[c], 1u);
            }
            __syncthreads();
        }
        const u64 wt = P.ties == 0 ? 0 : fixed_weight(key_value(P.key), r.ws, sh.table);
        const uint32_t ties = static_cast<uint32_t>(min(P.ties, u64(0xffffffffu)));
        const int each = (r.nch + THREADS - 1) / THREADS;
        const int c0 = min(r.nch, tid * each), c1 = min(r.nch, c0 + each);
        u64 w = 0, tw;
        uint32_t n = 0, tn;
        for (int c = c0; c < c1; ++c) w += cw[c], n += cn[c];
        B::scan(w, n, tw, tn, sh);
        const u64 kept = tw + min(tn, ties) * wt;
        // nothing cut: one total for both; otherwise the kept part is at most the whole
        all = P.key <= kKeyNegInf ? kept : max(all, kept);
        const u64 target = part_of(static_cast<double>(u), kept, false);
        if (tid == 0) sh.at = 0, sh.at_w = 0, sh.at_n = 0;
        __syncthreads();
        for (int c = c0; c < c1; ++c) {
            const u64 lo = w + min(n, ties) * wt;
            w += cw[c], n += cn[c];
            const u64 hi = w + min(n, ties) * wt;
            if (lo <= target && target < hi) {
                sh.at = c;
                sh.at_w = w - cw[c];
                sh.at_n = n - cn[c];
            }
        }
        __syncthreads();
        if (tid >= 32) return;
        // one warp goes through the chunk in index order
        Chunk<T> c;
        const int chunk = sh.at;
        c.load(r.x, r.V, chunk, tid, r.vec);
        u64 run = sh.at_w;
        uint32_t seen = sh.at_n;
        constexpr int VEC = Chunk<T>::VEC;
#pragma unroll
        for (int j = 0; j < Chunk<T>::LOADS; ++j) {
            u64 we[VEC], sum = 0;
            uint32_t tie[VEC], tsum = 0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float x = c.get(j * VEC + e);
                const uint32_t k = order_key(x);
                we[e] = k > P.key ? fixed_weight(x, r.ws, sh.table) : 0;
                tie[e] = k == P.key ? 1u : 0u;
                sum += we[e];
                tsum += tie[e];
            }
            u64 iw = sum;
            uint32_t in = tsum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 ow = __shfl_up_sync(0xffffffffu, iw, off);
                const uint32_t on = __shfl_up_sync(0xffffffffu, in, off);
                if (tid >= off) iw += ow, in += on;
            }
            u64 w_at = run + iw - sum;
            uint32_t n_at = seen + in - tsum;
            run += __shfl_sync(0xffffffffu, iw, 31);
            seen += __shfl_sync(0xffffffffu, in, 31);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const u64 lo = w_at + min(n_at, ties) * wt;
                w_at += we[e];
                n_at += tie[e];
                const u64 hi = w_at + min(n_at, ties) * wt;
                if (lo <= target && target < hi)
                    write_drawn(a, row_i, Chunk<T>::column(chunk, j, tid) + e,
                                c.get(j * VEC + e), r.ws.m, temp, all, kept, r.bits);
            }
        }
    }

    // After a kCollect: the boundary, the draw, or the next step.  Returns true when done.
    __device__ static bool after_collect(const Row<T>& r, Search& P, Cmd& cmd, double top_p,
                                         u64 top_k, u64* cw, uint32_t* cn, u64* own_w,
                                         uint32_t* own_n, uint32_t ranks, const SampleArgs& a,
                                         int64_t row_i, float u, double temp, u64& all,
                                         Shared& sh) {
        u64 above;
        uint32_t inside;
        const uint32_t n = merge(r, cmd, cw, cn, own_w, own_n, ranks, above, inside, sh);
        if (P.draw) {
            draw(r, P, cmd, cw, cn, a, row_i, u, temp, all, sh);
            return true;
        }
        if (P.sum) {                         // the exact total: search again with it
            P.sum = false;
            P.exact = true;
            P.s_lo = P.s_hi = all = above;
            start_p(r, P, cmd, top_p);
            return false;
        }
        if (n == 0xffffffffu) {              // the list did not hold the window
            if (P.level == 0) {
                P.level = 1;
                cmd = make_hist0(!P.want_k);
            } else {
                next_hist(P, cmd);
            }
            return false;
        }
        u64 list_w = 0, dummy_w;
        uint32_t dummy_n = 0, tn;
        if (cmd.list) {
            u64 mine = 0;
            for (uint32_t i = threadIdx.x; i < n; i += THREADS) mine += sh.w[i];
            dummy_w = mine;
            B::scan(dummy_w, dummy_n, list_w, tn, sh);
        } else {
            list_w = inside * fixed_weight(key_value(cmd.klo), r.ws, sh.table);
        }
        uint32_t key, up_n;
        u64 up, up_w;
        if (P.want_k) {
            const u64 left = top_k - P.n_above;
            if (cmd.list && left > n) {      // all that is not -inf
                P.key = kKeyNegInf;
                P.ties = 0;
                up_w = list_w;
            } else if (cmd.list) {
                list_select<THREADS>(false, left, sh, key, up, up_n, up_w);
                P.key = key;
                P.ties = left - up;
            } else {
                P.key = cmd.klo;
                P.ties = left;
                up_w = 0;
            }
            P.want_k = false;
            if (P.want_p) {
                const u64 wt = fixed_weight(key_value(P.key), r.ws, sh.table);
                P.exact = true;
                P.s_lo = P.s_hi = above + up_w + P.ties * wt;
                const u64 need = max(u64(1), part_of(top_p, P.s_lo, true));
                if (need <= above) {         // the nucleus ends above this window
                    start_p(r, P, cmd, top_p);
                    return false;
                }
            }
        }
        if (P.want_p) {
            const u64 need_lo = max(u64(1), part_of(top_p, P.s_lo, true));
            const u64 need_hi = max(u64(1), part_of(top_p, P.s_hi, true));
            if (need_lo <= above || need_hi > above + list_w) {
                // outside the window: the guess was short, or the total's bounds straddle it
                if (P.level == 0) {
                    start_p(r, P, cmd, top_p);
                } else if (!P.exact) {
                    P.sum = true;
                    cmd = make_above(0u);
                } else {
                    // cannot happen: exact sums put the need into the window
                    P.key = kKeyNegInf;
                    P.ties = 0;
                    finish(P, cmd);
                }
                return false;
            }
            if (cmd.list) {
                list_select<THREADS>(true, need_lo - above, sh, key, up, up_n, up_w);
                const u64 wt = fixed_weight(key_value(key), r.ws, sh.table);
                const u64 lo = need_lo - above - up_w, hi = need_hi - above - up_w;
                const u64 t = wt == 0 ? 0 : (lo + wt - 1) / wt;
                P.key = key;
                P.ties = t;
                if (need_hi != need_lo && (wt == 0 || (hi + wt - 1) / wt != t)) {
                    P.sum = true;            // the total's error matters here
                    cmd = make_above(0u);
                    return false;
                }
            } else {
                const u64 wt = fixed_weight(key_value(cmd.klo), r.ws, sh.table);
                const u64 t = wt == 0 ? 0 : (need_lo - above + wt - 1) / wt;
                P.key = cmd.klo;
                P.ties = t;
                if (need_hi != need_lo && (wt == 0 || (need_hi - above + wt - 1) / wt != t)) {
                    P.sum = true;
                    cmd = make_above(0u);
                    return false;
                }
            }
            P.want_p = false;
        }
        if (P.key_m > P.key) {
            P.key = P.key_m - 1;
            P.ties = 0;
            // elements above the window are not told apart: min_p may cut among them
            if (!cmd.list || above != 0) {
                finish(P, cmd);
                return false;
            }
        }
        P.draw = true;
        draw(r, P, cmd, cw, cn, a, row_i, u, temp, all, sh);
        return true;
    }
};

// The draw without truncation from the fast weights; false where their error leaves the
// token open.
template <typename T>
__device__ bool fast_draw(const Row<T>& r, const float* cmax, const u64* cw, u64 all, float u,
                          const SampleArgs& a, int64_t row_i, double temp, Shared0& sh) {
    const int tid = threadIdx.x;
    const u64 target = part_of(static_cast<double>(u), all, false);
    const int each = (r.nch + kThreads - 1) / kThreads;
    const int c0 = min(r.nch, tid * each), c1 = min(r.nch, c0 + each);
    u64 w = 0, tw;
    uint32_t n = 0, tn;
    for (int c = c0; c < c1; ++c) w += cw[c];
    Block<kThreads>::scan(w, n, tw, tn, sh);
    if (tid == 0) sh.flag = 0, sh.at = 0, sh.at_w = 0;
    __syncthreads();
    for (int c = c0; c < c1; ++c) {
        if (w <= target && target < w + cw[c]) sh.at = c, sh.at_w = w;
        w += cw[c];
    }
    __syncthreads();
    if (tid < 32) {
        const u64 err = static_cast<u64>(static_cast<float>(all) * (2.f * u * (1.f - u) * kFastErr +
                                                                    1.5e-11f)) + 8192;
        Chunk<T> c;
        const int chunk = sh.at;
        c.load(r.x, r.V, chunk, tid, r.vec);
        const float m = cmax[chunk];
        const u64 top = fixed_weight(m, r.ws, sh.table);
        u64 run = sh.at_w;
        constexpr int VEC = Chunk<T>::VEC;
        bool sure = false;
#pragma unroll
        for (int j = 0; j < Chunk<T>::LOADS; ++j) {
            u64 we[VEC], sum = 0;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                we[e] = scale_weight(ex2_approx((c.get(j * VEC + e) - m) * r.ws.ch), top);
                sum += we[e];
            }
            u64 iw = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 ow = __shfl_up_sync(0xffffffffu, iw, off);
                if (tid >= off) iw += ow;
            }
            u64 at = run + iw - sum;
            run += __shfl_sync(0xffffffffu, iw, 31);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const u64 lo = at;
                at += we[e];
                if ((lo == 0 || lo + err <= target) && target + err < at && lo <= target) {
                    sure = true;
                    write_drawn(a, row_i, Chunk<T>::column(chunk, j, tid) + e,
                                c.get(j * VEC + e), r.ws.m, temp, all, all, r.bits);
                }
            }
        }
        if (__any_sync(0xffffffffu, sure) && tid == 0) sh.flag = 1;
    }
    __syncthreads();
    return sh.flag != 0;
}

// A row's settings.
struct Settings {
    double temp, top_p, min_p;
    int64_t top_k;
    float u;
    bool ok;
};
__device__ __forceinline__ Settings read_settings(const SampleArgs& a, int64_t row) {
    Settings s;
    s.temp = a.temperature_rows != nullptr ? a.temperature_rows[row] : a.temperature;
    s.top_k = a.top_k_rows != nullptr ? a.top_k_rows[row] : a.top_k;
    s.top_p = a.top_p_rows != nullptr ? a.top_p_rows[row] : a.top_p;
    s.min_p = a.min_p_rows != nullptr ? a.min_p_rows[row] : a.min_p;
    s.u = a.uniforms[row];
    s.ok = s.temp >= kSampleMinT && s.temp <= kSampleMaxT && s.top_k >= 0 && s.top_p > 0.0 &&
           s.min_p >= 0.0 && s.min_p <= 1.0 && s.u >= 0.f && s.u < 1.f;
    return s;
}

template <typename T>
__device__ __forceinline__ Row<T> make_row(const T* logits, const SampleArgs& a, int64_t row,
                                           double temp, int nch, int own, int rank) {
    Row<T> r;
    r.x = logits + row * a.stride;
    r.V = a.V;
    r.nch = nch;
    r.own = own;
    r.first = rank * own;
    r.mine = max(0, min(own, nch - r.first));
    r.vec = a.vec_ok;
    r.bits = a.bits;
    const double c = 1.4426950408889634074 / temp;
    r.ws.m = 0.f;
    r.ws.ch = static_cast<float>(c);
    r.ws.cl = static_cast<float>(c - static_cast<double>(r.ws.ch));
    r.ws.shift = 62 - a.bits;
    r.scale = r.ws.ch * (kBins / kRange);
    return r;
}

// the key of the smallest float x with x >= max + T log(min_p); 0 without min_p
__device__ __forceinline__ uint32_t min_p_key(const Settings& s, float m) {
    if (!(s.min_p > 0.0)) return 0;
    const double at = static_cast<double>(m) + s.temp * log(s.min_p);
    const float f = static_cast<float>(at);
    return order_key(f) + (static_cast<double>(f) < at ? 1u : 0u);
}

// bounds of the exact total from the fast one
__device__ __forceinline__ void total_bounds(u64 all, u64& lo, u64& hi) {
    const u64 err = static_cast<u64>(static_cast<float>(all) * (kFastErr + 1.5e-11f)) + 8192;
    lo = all > err ? all - err : 1;
    hi = all + err;
}

// A value that enough chunk maxima reach: at least `count` of them, or (need > 0) maxima of
// a weight of at least `need`.  Between the maximum and `low`, by bisection with a warp a
// trial: 4 rounds leave 1/6561 of the range.  `low` itself if that is not enough, with
// found = false.
template <typename T>
__device__ float reach_value(const Row<T>& r, const float* cmax, int count, float need, float low,
                             bool& found, Shared0& sh) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float hi = r.ws.m, lo = low;
    found = true;
    for (int round = 0; round < 4; ++round) {
        // warp w tries the (w + 1)-th of 9 parts below hi; the first round also tries low
        const float step = (hi - lo) / (kWarps + 1);
        const float x = round == 0 && warp == kWarps - 1 ? low : hi - step * (warp + 1);
        int n = 0;
        float w = 0.f;
        for (int c = lane; c < r.nch; c += 32) {
            const float v = cmax[c];
            if (v < x) continue;
            ++n;
            if (need > 0.f) w += ex2_approx((v - r.ws.m) * r.ws.ch);
        }
        const bool enough =
            need > 0.f ? warp_sum(w) >= need : __reduce_add_sync(0xffffffffu, n) >= count;
        __syncthreads();
        if (lane == 0) sh.part_n[warp] = enough ? 1u : 0u;
        __syncthreads();
        int first = 0;                               // the highest trial that is enough
        while (first < kWarps && sh.part_n[first] == 0) ++first;
        if (round == 0) {
            if (first == kWarps) {
                found = false;
                return low;
            }
            if (first == kWarps - 1) {               // only low itself
                hi = hi - step * (kWarps - 1);
                continue;
            }
        }
        const float top = hi;
        if (first > 0) hi = top - step * first;
        if (first < kWarps) lo = top - step * (first + 1);
    }
    return lo;
}

// Draws from the elements at or above a value, if they settle the boundary and are few.
// Block 0 of the scan.
template <typename T>
__device__ bool short_draw(const Row<T>& r, const Settings& s, const float* cmax, uint16_t* ids,
                           u64 all, const SampleArgs& a, int64_t row_i, Shared0& sh) {
    typedef Block<kThreads> B;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool want_k = s.top_k > 0 && s.top_k < r.V, want_p = s.top_p < 1.0;
    const uint32_t key_m = min_p_key(s, r.ws.m);
    uint32_t tau = kKeyNegInf + 1;
    if (r.V > kShort && (want_k || want_p)) {
        // between the maximum and 48 powers of two below it: what is lower weighs nothing
        const float low = static_cast<float>(
            fmax(static_cast<double>(r.ws.m) - kRange / static_cast<double>(r.ws.ch),
                 -3.4028234663852886e38));
        const float need = static_cast<float>(s.top_p * 1.00001 * static_cast<double>(all) /
                                              static_cast<double>(u64(1) << r.bits));
        if (want_k && s.top_k > r.nch * 9 / 10) return false;
        bool found;
        const float x = reach_value(r, cmax, static_cast<int>(s.top_k), want_k ? 0.f : need, low,
                                    found, sh);
        if (!found && !want_k) return false;         // a wide nucleus
        tau = max(tau, order_key(x));
    }
    // what min_p cuts is needed only where top_p counts it
    if (!want_p) tau = max(tau, key_m);
    if (tid == 0) sh.n_list = 0, sh.n_ids = 0;
    __syncthreads();
    for (int c = tid; c < r.nch; c += kThreads)
        if (order_key(cmax[c]) >= tau) ids[atomicAdd(&sh.n_ids, 1u)] = static_cast<uint16_t>(c);
    __syncthreads();
    const int n_ids = sh.n_ids;
    constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;
    for (int i0 = warp; i0 < n_ids; i0 += kAhead * (kThreads / 32)) {
        Chunk<T> ch[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int i = i0 + q * (kThreads / 32);
            if (i < n_ids) ch[q].load(r.x, r.V, ids[i], lane, r.vec);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int i = i0 + q * (kThreads / 32);
            if (i >= n_ids) break;
#pragma unroll
            for (int e = 0; e < kLane; ++e) {
                const float x = ch[q].get(e);
                const uint32_t k = order_key(x);
                if (k < tau) continue;
                const uint32_t at = atomicAdd(&sh.n_list, 1u);
                if (at < kShort) {
                    sh.w[at] = fixed_weight(x, r.ws, sh.table);
                    sh.key[at] = k;
                    sh.idx[at] = Chunk<T>::column(ids[i], e / Chunk<T>::VEC, lane) +
                                 e % Chunk<T>::VEC;
                }
            }
        }
    }
    __syncthreads();
    const uint32_t n = sh.n_list;
    if (n > kShort) return false;
    // each element's place in the order, and the weight before it
    constexpr int kPer = kShort / kThreads;
    uint32_t place[kPer];
    u64 before[kPer], list_w = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t i = tid + q * kThreads;
        place[q] = 0;
        before[q] = 0;
        if (i >= n) continue;
        const uint32_t k = sh.key[i], v = sh.idx[i];
        for (uint32_t j = 0; j < n; ++j) {
            const uint32_t kj = sh.key[j];
            if (kj > k || (kj == k && sh.idx[j] < v)) ++place[q], before[q] += sh.w[j];
        }
        list_w += sh.w[i];
    }
    u64 dummy_w = list_w;
    uint32_t dummy = 0, tn;
    B::scan(dummy_w, dummy, list_w, tn, sh);
    u64 need_lo = ~u64(0), need_hi = ~u64(0);
    u64 top_k = ~u64(0);
    if (want_k) {
        top_k = static_cast<u64>(s.top_k);
        if (tid == 0) sh.at_w = list_w;              // fewer elements than top_k: all of them
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
            const uint32_t i = tid + q * kThreads;
            if (i < n && place[q] == top_k - 1) sh.at_w = before[q] + sh.w[i];
        }
        __syncthreads();
        if (want_p) need_lo = need_hi = max(u64(1), part_of(s.top_p, sh.at_w, true));
    } else if (want_p) {
        u64 lo, hi;
        total_bounds(all, lo, hi);
        need_lo = max(u64(1), part_of(s.top_p, lo, true));
        need_hi = max(u64(1), part_of(s.top_p, hi, true));
        if (need_hi > list_w && r.V > kShort) return false;
        if (r.V <= kShort) need_lo = need_hi = max(u64(1), part_of(s.top_p, list_w, true));
    }
    // kept, by each bound of the total: where the two differ the search decides
    bool keep[kPer], open = false;
    u64 kept = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t i = tid + q * kThreads;
        keep[q] = i < n && place[q] < top_k && before[q] < need_lo && sh.key[i] >= key_m;
        open |= i < n && place[q] < top_k && before[q] >= need_lo && before[q] < need_hi &&
                sh.key[i] >= key_m;
        if (keep[q]) kept += sh.w[i];
    }
    if (__syncthreads_or(open)) return false;
    // cut elements weigh nothing from here on
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t i = tid + q * kThreads;
        if (i < n && !keep[q]) sh.w[i] = 0;
    }
    u64 kept_all;
    dummy_w = kept;
    B::scan(dummy_w, dummy, kept_all, tn, sh);
    const u64 target = part_of(static_cast<double>(s.u), kept_all, false);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const uint32_t i = tid + q * kThreads;
        if (i >= n || !keep[q]) continue;
        const uint32_t v = sh.idx[i];
        u64 run = 0;
        for (uint32_t j = 0; j < n; ++j)
            if (sh.idx[j] < v) run += sh.w[j];
        if (run <= target && target < run + sh.w[i])
            write_drawn(a, row_i, v, key_value(sh.key[i]), r.ws.m, s.temp, max(all, kept_all),
                        kept_all, r.bits);
    }
    return true;
}

__host__ __device__ constexpr size_t scan_smem(int nch) {
    return sizeof(Shared0) + size_t(nch) * 8 + size_t(nch) * 4 + size_t(nch) * 2 + 16;
}

// Maximum and sum of a chunk: the sum of 2^((x - max) c) without one element of the
// maximum (sign bit set) where `apart`, else of all.  A row's total is a sum of such parts
// plus the maximum's own weight, so a logp near 0 keeps its digits.
template <typename T>
__device__ __forceinline__ float2 chunk_stats(const Chunk<T>& c, float ch, float& best) {
    float ml = c.get(0);
#pragma unroll
    for (int e = 1; e < kLane; ++e) ml = fmaxf(ml, c.get(e));
    const float m = warp_max(ml);
    // a chunk of -inf has sum 0; NaN or +inf make it NaN
    const float mm = fmaxf(m, -3.402823466e38f);
    float s[kLane];
#pragma unroll
    for (int e = 0; e < kLane; ++e) s[e] = ex2_approx((c.get(e) - mm) * ch);
    // only a chunk that holds the warp's largest so far can hold the row's maximum
    const bool apart = m >= best && m < INFINITY && m > -INFINITY;
    if (apart) {
        best = m;
        bool lead = (threadIdx.x & 31) == __ffs(__ballot_sync(0xffffffffu, ml == m)) - 1;
#pragma unroll
        for (int e = 0; e < kLane; ++e) {
            const bool hit = lead && c.get(e) == m;
            s[e] = hit ? 0.f : s[e];
            lead = lead && !hit;
        }
    }
#pragma unroll
    for (int w = kLane / 2; w > 0; w >>= 1)
#pragma unroll
        for (int e = 0; e < w; ++e) s[e] += s[e + w];
    const float sum = warp_sum(s[0]);
    return make_float2(m, apart ? -sum : sum);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    sample_scan_kernel(const T* __restrict__ logits, const SampleArgs a, int nch, int own,
                       int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared0& sh = *reinterpret_cast<Shared0*>(smem);
    u64* cw = reinterpret_cast<u64*>(smem + sizeof(Shared0));
    float* cmax = reinterpret_cast<float*>(cw + nch);
    uint16_t* ids = reinterpret_cast<uint16_t*>(cmax + nch);
    const int64_t row_i = blockIdx.x / ranks;
    const int rank = blockIdx.x % ranks;             // = the block's rank in its cluster
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    RowHeader* head = static_cast<RowHeader*>(a.workspace) + row_i;
    float2* stats = row_stats(a, row_i, nch);
    if (a.mask != nullptr && a.mask[row_i] == 0) {
        if (rank == 0 && tid == 0) {
            write_row(a, row_i, -1, 0.f, 0.f);
            head->mode = kRowDone;
        }
        return;
    }
    const Settings s = read_settings(a, row_i);
    if (!s.ok) {
        if (rank == 0 && tid == 0) {
            write_row(a, row_i, -1, quiet_nan(), quiet_nan());
            if (a.err != nullptr) atomicOr(a.err, RLK_DEVERR_SAMPLE_PARAM);
            head->mode = kRowDone;
        }
        return;
    }
    Row<T> r = make_row(logits, a, row_i, s.temp, nch, own, rank);
    float best = -INFINITY;
    constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;
    for (int i0 = warp; i0 < r.mine; i0 += kAhead * (kThreads / 32)) {
        Chunk<T> c[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int i = i0 + q * (kThreads / 32);
            if (i < r.mine) c[q].load(r.x, r.V, r.first + i, lane, r.vec);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const int i = i0 + q * (kThreads / 32);
            if (i >= r.mine) break;
            const float2 st = chunk_stats(c[q], r.ws.ch, best);
            if (lane == 0) stats[r.first + i] = st;
        }
    }
    // the other blocks are done once their part is out
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    if (rank != 0) return;
    for (int i = tid; i < kExpEntries; i += kThreads) sh.table[i] = kExpTable.v[i];
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    float m = -INFINITY;
    bool bad = false;
    for (int i = tid; i < nch; i += kThreads) {
        const float2 st = stats[i];
        cmax[i] = st.x;
        m = fmaxf(m, st.x);
        bad |= st.y != st.y;
    }
    m = warp_max(m);
    if (lane == 0) sh.part_n[warp] = __float_as_uint(m);
    bad = __syncthreads_or(bad);
    for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, __uint_as_float(sh.part_n[i]));
    if (bad || m == -INFINITY) {
        if (tid == 0) {
            write_row(a, row_i, -1, quiet_nan(), quiet_nan());
            if (a.err != nullptr) atomicOr(a.err, RLK_DEVERR_LOGITS);
            head->mode = kRowDone;
        }
        return;
    }
    r.ws.m = m;
    u64 mine = 0, all;
    uint32_t dummy = 0, tn;
    for (int i = tid; i < nch; i += kThreads) {
        const float2 st = stats[i];
        u64 w = 0;
        if (st.x > -INFINITY) {
            const u64 top = fixed_weight(st.x, r.ws, sh.table);
            w = scale_weight(fabsf(st.y), top) + (__float_as_uint(st.y) >> 31 ? top : 0);
        }
        cw[i] = w;
        mine += w;
    }
    Block<kThreads>::scan(mine, dummy, all, tn, sh);     // its barriers also publish cw
    const bool cut = (s.top_k > 0 && s.top_k < a.V) || s.top_p < 1.0 || s.min_p > 0.0;
    const bool done = cut ? short_draw(r, s, cmax, ids, all, a, row_i, sh)
                          : fast_draw(r, cmax, cw, all, s.u, a, row_i, s.temp, sh);
    if (tid == 0) {
        head->all = all;
        head->m = m;
        head->mode = done ? kRowDone : kRowSearch;
    }
}

// Floats and integers behind Shared in dynamic shared memory, for nch chunks of which a
// block owns `own`.
__host__ __device__ constexpr size_t search_smem(int nch, int own) {
    return sizeof(Shared) + size_t(nch) * 16 + size_t(own) * 12 + 16;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3)
    sample_search_kernel(const T* __restrict__ logits, const SampleArgs a, int nch, int own,
                         int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    u64* cw = reinterpret_cast<u64*>(smem + sizeof(Shared));     // all chunks: weight
    u64* own_w = cw + nch;                                       // own chunks
    float* cmax = reinterpret_cast<float*>(own_w + own);         // all chunks: maximum
    uint32_t* cn = reinterpret_cast<uint32_t*>(cmax + nch);      //             ties
    uint32_t* own_n = cn + nch;
    const int64_t row_i = blockIdx.x / ranks;
    const int rank = blockIdx.x % ranks;
    const int tid = threadIdx.x;
    // the scan's results (also of earlier calls that shared the workspace) are complete
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const RowHeader* head = static_cast<const RowHeader*>(a.workspace) + row_i;
    if (head->mode != kRowSearch) return;
    const Settings s = read_settings(a, row_i);
    Row<T> r = make_row(logits, a, row_i, s.temp, nch, own, rank);
    r.ws.m = head->m;
    u64 all = head->all;
    const float2* stats = row_stats(a, row_i, nch);
    for (int i = tid; i < nch; i += kThreads) cmax[i] = stats[i].x;
    for (int i = tid; i < kExpEntries; i += kThreads) sh.table[i] = kExpTable.v[i];
    __syncthreads();

    Search P;
    P.want_k = s.top_k > 0 && s.top_k < a.V;
    P.want_p = s.top_p < 1.0;
    P.draw = P.sum = P.exact = false;
    P.level = 0;
    P.n_above = 0;
    total_bounds(all, P.s_lo, P.s_hi);
    P.key = kKeyNegInf;
    P.ties = 0;
    P.key_m = min_p_key(s, r.ws.m);
    Cmd cmd;
    if (!P.want_k && !P.want_p) {
        Sampler<T, kThreads>::finish(P, cmd);
    } else if (a.V <= kList) {
        cmd = Cmd{kCollect, 0, 2 * kBins, kKeyNegInf + 1, 0xffffffffu, 0, 0, 1};
    } else {
        P.level = 1;
        cmd = make_hist0(!P.want_k);
    }

    // the blocks work on their chunks, block 0 decides what comes next
    for (int step = 0; step < kMaxSteps; ++step) {
        if (cmd.type == kHist)
            step_hist<T, kThreads>(r, cmd, cmax, sh);
        else
            step_collect<T, kThreads>(r, cmd, cmax, own_w, own_n, sh);
        cluster_join();
        if (rank == 0) {
            bool done = false;
            if (cmd.type == kHist)
                Sampler<T, kThreads>::after_hist(r, P, cmd, s.top_p, static_cast<u64>(s.top_k),
                                                 ranks, sh);
            else
                done = Sampler<T, kThreads>::after_collect(r, P, cmd, s.top_p,
                                                           static_cast<u64>(s.top_k), cw, cn,
                                                           own_w, own_n, ranks, a, row_i, s.u,
                                                           s.temp, all, sh);
            if (done) cmd.type = kDone;
            if (!done && step == kMaxSteps - 1 && tid == 0) {
                write_row(a, row_i, -1, quiet_nan(), quiet_nan());
                if (a.err != nullptr) atomicOr(a.err, RLK_DEVERR_WAIT_TIMEOUT);
            }
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
cudaError_t launch_rows(void (*kernel)(const T*, const SampleArgs, int, int, int),
                        const T* logits, const SampleArgs& a, int nch, int ranks, size_t smem,
                        bool dependent, cudaStream_t stream) {
    const int own = (nch + ranks - 1) / ranks;
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, logits, a, nch, own, ranks);
}

template <typename T>
cudaError_t launch_typed(const T* logits, const SampleArgs& a, cudaStream_t stream) {
    const int nch = (a.V + kChunk - 1) / kChunk;
    const int ranks = nch >= 128 ? 8 : nch >= 64 ? 4 : nch >= 32 ? 2 : 1;
    if (int64_t(a.N) * ranks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaError_t e = launch_rows(sample_scan_kernel<T>, logits, a, nch, ranks, scan_smem(nch), false,
                                stream);
    if (e != cudaSuccess) return e;
    return launch_rows(sample_search_kernel<T>, logits, a, nch, ranks,
                       search_smem(nch, (nch + ranks - 1) / ranks), true, stream);
}

}  // namespace

size_t sample_workspace(int64_t N, int64_t V) {
    return stats_offset(N) + size_t(N) * size_t((V + kChunk - 1) / kChunk) * sizeof(float2);
}

cudaError_t launch_sample(const void* logits, bool bf16, const SampleArgs& args,
                          cudaStream_t stream) {
    if (bf16)
        return launch_typed(static_cast<const __nv_bfloat16*>(logits), args, stream);
    return launch_typed(static_cast<const float*>(logits), args, stream);
}

}  // namespace rlk
