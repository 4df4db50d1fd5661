// topk_kl.cu -- KL of the LM head against a teacher's top tokens: all but the GEMMs.
//
// "RL-Kernel Roadmap (2026)", backlog: distillation KL fused with lm_head.  A teacher that is
// not at hand as a head (rlk_linear_kl_fwd) sends K token ids a row and their log-weights a_k:
//
//   A = renormalize ? log sum_k exp a_k : 0,  q_k = exp(a_k - A),  Q = sum_k q_k
//   lp_k = s[t, id_k]/T - lse,  kl = sum_k q_k (a_k - A - lp_k)
//   dS[t,v] = (g_t / T) (Q_t p[t,v] - sum_{k: id_k = v} q_k)
//
// Forward: each row's tokens are put in order (launch_topk_list), the GEMM of the log-prob
// leaves the partials of lse and takes the listed logits from the same accumulators
// (launch_list_partials), and launch_topk_merge forms lse, logp and kl.  Backward: launch_topk_coef
// forms the coefficients; then per vocabulary chunk the dS GEMM, launch_topk_scatter for the listed
// entries, and the dh and dW GEMMs.  What bf16 leaves of the listed entries is taken along:
// launch_topk_dh starts dh with it, launch_topk_sort lists the entries by token and launch_topk_rows
// sums them for dW.
//
// A slot with a negative id is empty.  A row with an id >= V, or a log-weight that is NaN or
// +inf at an id, gives NaN and sets an error bit; the backward gives it no gradient.
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// A row's slots, one warp a row.  Sums run over each lane's slots in ascending order and a
// fixed tree: they depend on the row alone.
struct RowSlots {
    const int64_t* ids;
    const float* teacher;
    float shift;               // A
    uint32_t bad;              // error bits

    __device__ __forceinline__ RowSlots(const TopkSlots& s, int t, int lane)
        : ids(s.ids + static_cast<size_t>(t) * s.K),
          teacher(s.teacher + static_cast<size_t>(t) * s.K), shift(0.f), bad(0) {
        float m = -INFINITY;
        for (int j = lane; j < s.K; j += 32) {
            const int64_t id = ids[j];
            if (id < 0) continue;
            if (id >= s.V) bad |= RLK_DEVERR_TARGET_RANGE;
            const float a = teacher[j];
            if (!(a < INFINITY)) bad |= RLK_DEVERR_LOGITS;
            m = fmaxf(m, a);
        }
        bad = __reduce_or_sync(0xffffffffu, bad);
        if (bad != 0 || !s.renormalize) return;
        m = warp_max(m);
        if (m == -INFINITY) return;              // no weight at all: every q is 0
        float sum = 0.f;
        for (int j = lane; j < s.K; j += 32)
            if (ids[j] >= 0) sum += expf(teacher[j] - m);
        shift = m + logf(warp_sum(sum));
    }
    __device__ __forceinline__ float log_weight(int j) const { return teacher[j] - shift; }
};

// row i, by `threads` threads
__device__ __forceinline__ void copy_row(const CopyRows& c, int i, int thread, int threads) {
    if (c.h_to == nullptr) return;
    const int vecs = c.H / 8;
    const size_t from = static_cast<size_t>(i) * vecs;
    for (int j = thread; j < vecs; j += threads)
        static_cast<uint4*>(c.h_to)[from + j] = static_cast<const uint4*>(c.h)[from + j];
}

// ----------------------------------------------------------------------------- list

constexpr int kListThreads = 128;

// A block a GEMM row: its tokens in ascending order (Batcher's bitonic network), empty slots
// behind them, so that the GEMM's epilogue meets them as it walks the columns.
__global__ void __launch_bounds__(kListThreads)
    topk_list_kernel(const TopkSlots slots, const int* __restrict__ rows,
                     const int* __restrict__ n_rows, int num_chunks, int size,
                     int2* __restrict__ list, uint16_t* __restrict__ first, const CopyRows args) {
    __shared__ uint64_t key[kMaxTopK];
    TopkSlots s = slots;
    CopyRows copy = args;
    wait_previous(s.ids, rows, n_rows, copy.h);
    const int i = blockIdx.x;
    if (n_rows != nullptr && i >= *n_rows) return;
    copy_row(copy, i, threadIdx.x, kListThreads);
    const int64_t* ids = s.ids + static_cast<size_t>(rows != nullptr ? rows[i] : i) * s.K;
    for (int j = threadIdx.x; j < size; j += kListThreads) {
        const int64_t id = j < s.K ? ids[j] : -1;
        key[j] = (static_cast<uint64_t>(id >= 0 && id < s.V ? id : 0x7fffffff) << 32) | j;
    }
    __syncthreads();
    for (int run = 2; run <= size; run <<= 1) {
        for (int d = run >> 1; d > 0; d >>= 1) {
            for (int j = threadIdx.x; j < size; j += kListThreads) {
                const int o = j ^ d;
                if (o > j) {
                    const uint64_t a = key[j], b = key[o];
                    if ((a > b) == ((j & run) == 0)) {
                        key[j] = b;
                        key[o] = a;
                    }
                }
            }
            __syncthreads();
        }
    }
    for (int j = threadIdx.x; j < s.K; j += kListThreads)
        list[static_cast<size_t>(i) * s.K + j] =
            make_int2(static_cast<int>(key[j] >> 32), static_cast<int>(key[j] & 0xffffffffu));
    for (int c = threadIdx.x; c < num_chunks; c += kListThreads) {
        const uint64_t from = static_cast<uint64_t>(c) * kTileV << 32;
        int lo = 0, hi = s.K;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (key[mid] < from) lo = mid + 1; else hi = mid;
        }
        first[static_cast<size_t>(i) * num_chunks + c] = static_cast<uint16_t>(lo);
    }
}

// ----------------------------------------------------------------------------- lse, logp, kl

// lse of eight rows a block, a tile's partial to group tile mod 32 and ascending in it, then the
// groups in order; then a warp for each row's slots.
constexpr int kRows = 8, kGroups = 32;

__global__ void __launch_bounds__(kRows * kGroups)
    topk_merge_kernel(const TopkSlots args, const float2* __restrict__ partials, int num_chunks,
                      const int* __restrict__ pos_of, float k, float* __restrict__ kl,
                      float* __restrict__ lse, float* __restrict__ logp, uint32_t* err) {
    TopkSlots s = args;
    wait_previous(s.ids, s.teacher, s.mask, partials, pos_of, logp);
    __shared__ float s_m[kRows][kGroups + 1];
    __shared__ float s_s[kRows][kGroups + 1];
    const int t0 = blockIdx.x * kRows;
    {
        const int r = threadIdx.x % kRows, g = threadIdx.x / kRows;
        const int t = t0 + r;
        const bool live = t < s.N && (s.mask == nullptr || s.mask[t] != 0);
        const int i = !live ? 0 : (pos_of != nullptr ? pos_of[t] : t);
        float m = -INFINITY, sigma = 0.f;
        if (live) {
#pragma unroll 4
            for (int c = g; c < num_chunks; c += kGroups)
                m = fmaxf(m, partials[static_cast<size_t>(c) * s.N + i].x);
#pragma unroll 4
            for (int c = g; c < num_chunks; c += kGroups) {
                const float2 pc = partials[static_cast<size_t>(c) * s.N + i];
                sigma += pc.y * ex2_approx((pc.x - m) * k);
            }
        }
        s_m[r][g] = m;
        s_s[r][g] = sigma;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, a = threadIdx.x >> 5;
    {
        const int t = t0 + a;
        if (t >= s.N) return;
        float* lp = logp + static_cast<size_t>(t) * s.K;
        if (s.mask != nullptr && s.mask[t] == 0) {
            for (int j = lane; j < s.K; j += 32) lp[j] = 0.f;
            if (lane == 0) kl[t] = 0.f, lse[t] = 0.f;
            return;
        }
        // the row's largest logit, and log2 sum 2^((s - top) k)
        const float top = warp_max(s_m[a][lane]);
        const float log_sum = log2f(warp_sum(s_s[a][lane] * ex2_approx((s_m[a][lane] - top) * k)));
        if (lane == 0) lse[t] = fmaf(top, k, log_sum) * kLn2;
        const RowSlots slots(s, t, lane);
        if (slots.bad != 0) {
            for (int j = lane; j < s.K; j += 32) lp[j] = __int_as_float(0x7fc00000);
            if (lane == 0) {
                kl[t] = __int_as_float(0x7fc00000);
                if (err != nullptr) atomicOr(err, slots.bad);
            }
            return;
        }
        float sum = 0.f;
        for (int j = lane; j < s.K; j += 32) {
            if (slots.ids[j] < 0) {
                lp[j] = 0.f;
                continue;
            }
            // from the maximum, not from lse: a token near p = 1 keeps the digits of log p
            const float l = fmaf(lp[j] - top, k, -log_sum) * kLn2, la = slots.log_weight(j);
            lp[j] = l;
            if (la > -INFINITY) sum = fmaf(expf(la), la - l, sum);   // a weight of 0 counts 0
        }
        sum = warp_sum(sum);
        if (lane == 0) kl[t] = sum;
    }
}

// ----------------------------------------------------------------------------- entries of dS

constexpr int kCoefWarps = 4;

// A warp a GEMM row.  An id that a row lists more than once gets one entry, at its first slot,
// with the sum q of its weights.  Q p - q = (Q - q) p - q (1 - p) keeps its digits where p is
// near 1 and q near Q: 1 - p comes from expm1, and for the largest q of the row (no other can be
// near Q) Q - q is the sum of the others.
__global__ void __launch_bounds__(kCoefWarps * 32)
    topk_coef_kernel(const TopkSlots args, const float* __restrict__ grad,
                     const float* __restrict__ logp, const int* __restrict__ rows,
                     const int* __restrict__ n_rows, float temp, float* __restrict__ coef,
                     int* __restrict__ ids_out, float* __restrict__ val, const CopyRows copy_args,
                     uint32_t* err) {
    extern __shared__ int s_all[];
    TopkSlots s = args;
    CopyRows copy = copy_args;
    wait_previous(s.ids, s.teacher, grad, logp, rows, n_rows, copy.h);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* s_id = s_all + warp * 3 * s.K;
    float* s_q = reinterpret_cast<float*>(s_id + s.K);
    float* s_sum = s_q + s.K;                    // an id's weights together, at its first slot
    const int i = blockIdx.x * kCoefWarps + warp;
    if (i >= (n_rows != nullptr ? *n_rows : s.N)) return;
    copy_row(copy, i, lane, 32);
    const int t = rows != nullptr ? rows[i] : i;
    int* out_id = ids_out + static_cast<size_t>(i) * s.K;
    float* out_val = val + static_cast<size_t>(i) * s.K;
    const RowSlots slots(s, t, lane);
    if (slots.bad != 0) {
        for (int j = lane; j < s.K; j += 32) out_id[j] = -1;
        if (lane == 0) {
            coef[i] = 0.f;
            if (err != nullptr) atomicOr(err, slots.bad);
        }
        return;
    }
    for (int j = lane; j < s.K; j += 32) {
        const int id = slots.ids[j] < 0 ? -1 : static_cast<int>(slots.ids[j]);
        s_id[j] = id;
        s_q[j] = id < 0 ? 0.f : expf(slots.log_weight(j));
    }
    __syncwarp();
    float best = -1.f;
    int at = s.K;                                // the lane's largest sum and its slot
    for (int j = lane; j < s.K; j += 32) {
        const int id = s_id[j];
        float q = -1.f;
        if (id >= 0) {
            int first = j;
            q = 0.f;
            for (int e = 0; e < s.K; ++e)
                if (s_id[e] == id) {
                    first = min(first, e);
                    q += s_q[e];
                }
            if (first != j) q = -1.f;
        }
        s_sum[j] = q;
        if (q > best) best = q, at = j;
    }
    const float top = warp_max(best);
    at = __reduce_min_sync(0xffffffffu, best == top ? at : s.K);
    float others = 0.f;
    for (int j = lane; j < s.K; j += 32)
        if (j != at && s_sum[j] > 0.f) others += s_sum[j];
    others = warp_sum(others);
    const float mass = others + fmaxf(top, 0.f);
    const float gt = __fdiv_rn(grad[t], temp);
    if (lane == 0) coef[i] = gt * mass;
    for (int j = lane; j < s.K; j += 32) {
        const float q = s_sum[j];
        out_id[j] = q < 0.f ? -1 : s_id[j];
        if (q < 0.f) continue;
        const float lp = logp[static_cast<size_t>(t) * s.K + j];
        const float rest = j == at ? others : mass - q;
        out_val[j] = gt * fmaf(rest, expf(lp), q * expm1f(lp));
    }
}

// What rounding to bf16 leaves, exactly.
__device__ __forceinline__ float rest_of(float d) {
    return d - __bfloat162float(__float2bfloat16_rn(d));
}

// The chunk's listed entries, over what the GEMM wrote there.
template <bool LO>
__global__ void __launch_bounds__(256)
    topk_scatter_kernel(const int* __restrict__ ids, const float* __restrict__ val,
                        const int* __restrict__ n_rows, int N, int K, int c0, int width,
                        __nv_bfloat16* __restrict__ ds) {
    wait_previous(ids, val, n_rows, ds);
    const size_t count = static_cast<size_t>(n_rows != nullptr ? *n_rows : N) * K;
    const size_t step = static_cast<size_t>(gridDim.x) * 256;
    for (size_t e = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; e < count; e += step) {
        const int id = ids[e];
        if (id < c0 || id - c0 >= width) continue;
        const float d = val[e];
        __nv_bfloat16* at = ds + (e / K) * ((LO ? 2 : 1) * kBwdChunk) + (id - c0);
        at[0] = __float2bfloat16_rn(d);
        if (LO) at[kBwdChunk] = __float2bfloat16_rn(rest_of(d));
    }
}

// ----------------------------------------------------------------------------- what bf16 leaves

// acc += coef row, 8 columns
__device__ __forceinline__ void add_row(float coef, uint4 v, float (&acc)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(coef, __uint_as_float(w[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(coef, __uint_as_float(w[i] & 0xffff0000u), acc[2 * i + 1]);
    }
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
constexpr int kRowThreads = 256, kRowAhead = 8;

// dh_acc[i] = sum over the slots, ascending, of rest W[id]: a block a row and 2048 columns.  Bound by
// the rows of W it reads: N K H 2 bytes ([2048, 4096], K = 64: 1.07 GB in 132 us, 8.1 TB/s, some of
// them from L2).
__global__ void __launch_bounds__(kRowThreads)
    topk_dh_kernel(const int* __restrict__ ids, const float* __restrict__ val,
                   const int* __restrict__ n_rows, int N, int K, const uint4* __restrict__ weight,
                   int vecs, float* __restrict__ dh_acc) {
    __shared__ int s_id[kMaxTopK + kRowAhead];
    __shared__ float s_rest[kMaxTopK + kRowAhead];
    wait_previous(ids, val, n_rows, weight);
    const int i = blockIdx.x;
    if (i >= (n_rows != nullptr ? *n_rows : N)) return;
    for (int j = threadIdx.x; j < K + kRowAhead; j += kRowThreads) {
        const size_t at = static_cast<size_t>(i) * K + j;
        const int id = j < K ? ids[at] : -1;
        s_id[j] = id;
        s_rest[j] = id >= 0 ? rest_of(val[at]) : 0.f;
    }
    __syncthreads();
    const int c = blockIdx.y * kRowThreads + threadIdx.x;
    if (c >= vecs) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < K; j0 += kRowAhead) {
        uint4 v[kRowAhead];
#pragma unroll
        for (int q = 0; q < kRowAhead; ++q)
            if (s_id[j0 + q] >= 0) v[q] = __ldg(weight + static_cast<size_t>(s_id[j0 + q]) * vecs + c);
#pragma unroll
        for (int q = 0; q < kRowAhead; ++q)
            if (s_id[j0 + q] >= 0) add_row(s_rest[j0 + q], v[q], acc);
    }
    float4* to = reinterpret_cast<float4*>(dh_acc + (static_cast<size_t>(i) * vecs + c) * 8);
    to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// The same by vocabulary row: sums[place] = sum of rest h over its entries in ascending rows.  The h
// rows of some thousand tokens stay in L2.  Most rows have an entry or a few: a warp each, its
// entries fetched together.  Rows with more than kMany: a block for 256 columns, whose warps take an
// eighth of the entries each, added up in order.
constexpr int kMany = 32;

__global__ void __launch_bounds__(kRowThreads)
    topk_rows_kernel(const TopkRows r, int chunk, const uint4* __restrict__ hidden, int vecs) {
    const int lane = threadIdx.x & 31;
    const int count = r.counts[chunk].x, warps = gridDim.x * (kRowThreads / 32);
    uint4* sums = static_cast<uint4*>(r.sums);
    for (int p = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); p < count; p += warps) {
        const int v = r.list[chunk * kBwdChunk + p];
        const int e0 = r.first[v], n = r.last[v] - e0;
        if (n > kMany) continue;
        const int row = lane < n ? r.entry_row[e0 + lane] : 0;
        const float rest = lane < n ? r.entry_rest[e0 + lane] : 0.f;
        constexpr int kWide = 4;                 // groups of 256 columns at a time
        for (int cb = 0; cb < vecs; cb += 32 * kWide) {
            const int c0 = cb + lane;
            float acc[kWide][8] = {};
            for (int e = 0; e < n; e += 2) {
                uint4 h[2][kWide];
                float coef[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int er = __shfl_sync(0xffffffffu, row, min(e + q, n - 1));
                    coef[q] = __shfl_sync(0xffffffffu, rest, min(e + q, n - 1));
                    const uint4* from = hidden + static_cast<size_t>(er) * vecs;
#pragma unroll
                    for (int w = 0; w < kWide; ++w)
                        if (e + q < n && c0 + 32 * w < vecs) h[q][w] = __ldg(from + c0 + 32 * w);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int w = 0; w < kWide; ++w)
                        if (e + q < n && c0 + 32 * w < vecs) add_row(coef[q], h[q][w], acc[w]);
            }
#pragma unroll
            for (int w = 0; w < kWide; ++w)
                if (c0 + 32 * w < vecs)
                    sums[static_cast<size_t>(p) * vecs + c0 + 32 * w] =
                        make_uint4(pack(acc[w][0], acc[w][1]), pack(acc[w][2], acc[w][3]),
                                   pack(acc[w][4], acc[w][5]), pack(acc[w][6], acc[w][7]));
        }
    }
}

__global__ void __launch_bounds__(kRowThreads)
    topk_many_kernel(const TopkRows r, int chunk, const uint4* __restrict__ hidden, int vecs) {
    constexpr int kWarps = kRowThreads / 32;
    __shared__ float part[kWarps][32][8 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int count = r.counts[chunk].y, groups = (vecs + 31) / 32;
    for (int64_t job = blockIdx.x; job < static_cast<int64_t>(count) * groups; job += gridDim.x) {
        const int p = r.many[chunk * kBwdChunk + job / groups];
        const int c = static_cast<int>(job % groups) * 32 + lane;
        const int v = r.list[chunk * kBwdChunk + p];
        const int e0 = r.first[v], n = r.last[v] - e0;
        const int each = (n + kWarps - 1) / kWarps;
        const int from = e0 + min(n, warp * each), to = e0 + min(n, (warp + 1) * each);
        float acc[8] = {};
        if (c < vecs)
            for (int e = from; e < to; e += kRowAhead) {
                uint4 h[kRowAhead];
#pragma unroll
                for (int q = 0; q < kRowAhead; ++q)
                    if (e + q < to)
                        h[q] = __ldg(hidden + static_cast<size_t>(r.entry_row[e + q]) * vecs + c);
#pragma unroll
                for (int q = 0; q < kRowAhead; ++q)
                    if (e + q < to) add_row(r.entry_rest[e + q], h[q], acc);
            }
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][lane][i] = acc[i];
        __syncthreads();
        if (warp == 0 && c < vecs) {
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += part[w][lane][i];
            static_cast<uint4*>(r.sums)[static_cast<size_t>(p) * vecs + c] =
                make_uint4(pack(acc[0], acc[1]), pack(acc[2], acc[3]), pack(acc[4], acc[5]),
                           pack(acc[6], acc[7]));
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------- entries by token id
//
// A stable radix sort of (id, slot number) by id, 9 bits at a time from the lowest on: equal ids
// stay in ascending rows, so the sums of dW have one order.  A tile of 2048 pairs a block; each of
// its warps takes 256 consecutive ones, 32 at a time, and counts digits in its own row of shared
// memory, so that a pair's place follows from whole numbers alone.

constexpr int kRadix = 1 << kRadixBits, kSortThreads = 256, kSortWarps = kSortThreads / 32;
constexpr int kWarpPairs = kRadixTile / kSortWarps;

struct Pairs {
    const int* ids;                      // first pass: [E] by slot, -1: none
    const uint32_t* key;                 // later passes
    const uint32_t* slot;
    const int* n_rows;
    int64_t entries;
    int N, K, V;

    // entries without an id sort behind all others
    __device__ __forceinline__ uint32_t key_of(int64_t e) const {
        if (key != nullptr) return key[e];
        const int64_t live = static_cast<int64_t>(n_rows != nullptr ? *n_rows : N) * K;
        const int id = e < live ? ids[e] : -1;
        return static_cast<uint32_t>(id >= 0 ? id : V);
    }
};

__global__ void __launch_bounds__(kSortThreads)
    radix_count_kernel(const Pairs in, int shift, uint32_t* __restrict__ hist, int tiles) {
    __shared__ uint32_t s_n[kRadix];
    for (int d = threadIdx.x; d < kRadix; d += kSortThreads) s_n[d] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < kRadixTile; j += kSortThreads) {
        const int64_t e = static_cast<int64_t>(blockIdx.x) * kRadixTile + j;
        if (e < in.entries) atomicAdd(&s_n[(in.key_of(e) >> shift) & (kRadix - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kRadix; d += kSortThreads)
        hist[static_cast<size_t>(d) * tiles + blockIdx.x] = s_n[d];
}

// inclusive sum over the block's threads
template <int THREADS>
__device__ __forceinline__ uint32_t block_sum_scan(uint32_t v, uint32_t* part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += part[w];
    __syncthreads();
    return before + v;
}

// exclusive sums of n counts, in place, by one block
__global__ void __launch_bounds__(1024) radix_scan_kernel(uint32_t* hist, int64_t n) {
    __shared__ uint32_t part[32];
    __shared__ uint32_t s_total;
    uint32_t base = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 4096) {
        const int64_t i = i0 + threadIdx.x * 4;      // n is a multiple of 512
        uint4 v = i < n ? *reinterpret_cast<const uint4*>(hist + i) : uint4{};
        const uint32_t own = v.x + v.y + v.z + v.w;
        const uint32_t inc = base + block_sum_scan<1024>(own, part);
        if (threadIdx.x == 1023) s_total = inc;
        uint32_t run = inc - own;
        uint4 out;
        out.x = run, run += v.x;
        out.y = run, run += v.y;
        out.z = run, run += v.z;
        out.w = run;
        if (i < n) *reinterpret_cast<uint4*>(hist + i) = out;
        __syncthreads();
        base = s_total;
    }
}

__global__ void __launch_bounds__(kSortThreads)
    radix_place_kernel(const Pairs in, int shift, const uint32_t* __restrict__ hist, int tiles,
                       uint32_t* __restrict__ key_out, uint32_t* __restrict__ slot_out) {
    __shared__ uint32_t s_n[kSortWarps][kRadix];     // a warp's counts, then where its first goes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int d = threadIdx.x; d < kRadix * kSortWarps; d += kSortThreads) (&s_n[0][0])[d] = 0;
    __syncthreads();
    constexpr int kRounds = kWarpPairs / 32;
    uint32_t key[kRounds], rank[kRounds];
    const int64_t e0 = static_cast<int64_t>(blockIdx.x) * kRadixTile + warp * kWarpPairs + lane;
#pragma unroll
    for (int q = 0; q < kRounds; ++q) key[q] = e0 + q * 32 < in.entries ? in.key_of(e0 + q * 32) : 0;
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
        const bool there = e0 + q * 32 < in.entries;
        const uint32_t d = there ? (key[q] >> shift) & (kRadix - 1) : kRadix;
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        const int leader = __ffs(same) - 1;
        uint32_t before = 0;
        if (there && lane == leader) {
            before = s_n[warp][d];
            s_n[warp][d] = before + __popc(same);
        }
        rank[q] = __shfl_sync(0xffffffffu, before, leader) + __popc(same & ((1u << lane) - 1));
        __syncwarp();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kRadix; d += kSortThreads) {
        uint32_t run = hist[static_cast<size_t>(d) * tiles + blockIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t n = s_n[w][d];
            s_n[w][d] = run;
            run += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kRounds; ++q) {
        const int64_t e = e0 + q * 32;
        if (e >= in.entries) continue;
        const uint32_t to = s_n[warp][(key[q] >> shift) & (kRadix - 1)] + rank[q];
        key_out[to] = key[q];
        slot_out[to] = in.slot != nullptr ? in.slot[e] : static_cast<uint32_t>(e);
    }
}

// Each entry's GEMM row and remainder, in place of the sort's other buffers; where each token id's
// entries begin and end.
__global__ void __launch_bounds__(256)
    topk_entries_kernel(const uint32_t* __restrict__ key, const uint32_t* __restrict__ slot,
                        const float* __restrict__ val, int64_t entries, int K, uint32_t V,
                        int* __restrict__ row, float* __restrict__ rest, int* __restrict__ first,
                        int* __restrict__ last) {
    const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (e >= entries) return;
    const uint32_t v = key[e];
    if (v >= V) return;
    row[e] = static_cast<int>(slot[e] / static_cast<uint32_t>(K));
    rest[e] = rest_of(val[slot[e]]);
    if (e == 0 || key[e - 1] != v) first[v] = static_cast<int>(e);
    if (e + 1 == entries || key[e + 1] != v) last[v] = static_cast<int>(e) + 1;
}

// A block a vocabulary chunk: its rows that have entries, ascending; the places of those with many.
__global__ void __launch_bounds__(1024)
    topk_index_kernel(const int* __restrict__ first, const int* __restrict__ last, int V,
                      int* __restrict__ row_at, int* __restrict__ list, int* __restrict__ many,
                      int2* __restrict__ counts) {
    __shared__ uint32_t part[32];
    __shared__ uint32_t s_total, s_many;
    const int c0 = blockIdx.x * kBwdChunk, c1 = min(V, c0 + kBwdChunk);
    if (threadIdx.x == 0) s_many = 0;
    uint32_t base = 0;
    for (int b0 = c0; b0 < c1; b0 += 4096) {
        const int v0 = b0 + threadIdx.x * 4;
        int4 end = make_int4(0, 0, 0, 0);
        if (v0 + 3 < c1) {
            end = *reinterpret_cast<const int4*>(last + v0);
        } else {
            if (v0 < c1) end.x = last[v0];
            if (v0 + 1 < c1) end.y = last[v0 + 1];
            if (v0 + 2 < c1) end.z = last[v0 + 2];
        }
        const int ends[4] = {end.x, end.y, end.z, end.w};
        uint32_t own = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) own += ends[j] > 0;
        const uint32_t inc = base + block_sum_scan<1024>(own, part);
        if (threadIdx.x == 1023) s_total = inc;
        uint32_t at = inc - own;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (v0 + j >= c1) continue;
            const bool on = ends[j] > 0;
            row_at[v0 + j] = on ? static_cast<int>(at) : -1;
            if (!on) continue;
            list[c0 + at] = v0 + j;
            if (ends[j] - first[v0 + j] > kMany)
                many[c0 + atomicAdd(&s_many, 1u)] = static_cast<int>(at);   // in no order: each by itself
            ++at;
        }
        __syncthreads();
        base = s_total;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        counts[blockIdx.x] = make_int2(static_cast<int>(base), static_cast<int>(s_many));
}

}  // namespace

cudaError_t launch_topk_list(const TopkSlots& slots, const int* rows, const int* n_rows,
                             int num_chunks, int2* list, uint16_t* first, const CopyRows& copy,
                             cudaStream_t stream) {
    int size = 2;
    while (size < slots.K) size *= 2;
    return launch_early(topk_list_kernel, dim3(slots.N), kListThreads, 0, stream, nullptr, slots,
                        rows, n_rows, num_chunks, size, list, first, copy);
}

cudaError_t launch_topk_merge(const TopkSlots& slots, const float2* partials, int num_chunks,
                              const int* pos_of, float k, float* kl, float* lse, float* logp,
                              uint32_t* err, cudaStream_t stream) {
    return launch_early(topk_merge_kernel, dim3((slots.N + kRows - 1) / kRows), kRows * kGroups, 0,
                        stream, nullptr, slots, partials, num_chunks, pos_of, k, kl, lse, logp, err);
}

cudaError_t launch_topk_coef(const TopkSlots& slots, const float* grad, const float* logp,
                             const int* rows, const int* n_rows, float temp, float* coef,
                             int* ids, float* val, const CopyRows& copy, uint32_t* err,
                             cudaStream_t stream) {
    static_assert(kCoefWarps * 12 * kMaxTopK <= 48 * 1024, "a block's shared memory");
    return launch_early(topk_coef_kernel, dim3((slots.N + kCoefWarps - 1) / kCoefWarps),
                        kCoefWarps * 32, static_cast<size_t>(kCoefWarps) * 12 * slots.K, stream,
                        nullptr, slots, grad, logp, rows, n_rows, temp, coef, ids, val, copy, err);
}

cudaError_t launch_topk_scatter(const int* ids, const float* val, const int* n_rows, int N, int K,
                                int c0, int width, void* ds, bool lo, cudaStream_t stream) {
    const size_t blocks = (static_cast<size_t>(N) * K + 255) / 256, most = 152 * 8;
    const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(ds);
    return launch_early(lo ? topk_scatter_kernel<true> : topk_scatter_kernel<false>, dim3(grid), 256,
                        0, stream, nullptr, ids, val, n_rows, N, K, c0, width, to);
}

cudaError_t launch_topk_dh(const int* ids, const float* val, const int* n_rows, int N, int K,
                           const void* weight, int H, float* dh_acc, cudaStream_t stream) {
    const int vecs = H / 8;
    const dim3 grid(N, (vecs + kRowThreads - 1) / kRowThreads);
    return launch_early(topk_dh_kernel, grid, kRowThreads, 0, stream, nullptr, ids, val, n_rows, N, K,
                        static_cast<const uint4*>(weight), vecs, dh_acc);
}

cudaError_t launch_topk_rows(const TopkRows& rows, int chunk, const void* hidden, int H,
                             cudaStream_t stream) {
    const int vecs = H / 8, blocks = (rows.places + kRowThreads / 32 - 1) / (kRowThreads / 32);
    const uint4* h = static_cast<const uint4*>(hidden);
    topk_rows_kernel<<<blocks < 152 * 8 ? blocks : 152 * 8, kRowThreads, 0, stream>>>(rows, chunk, h,
                                                                                      vecs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    topk_many_kernel<<<152 * 8, kRowThreads, 0, stream>>>(rows, chunk, h, vecs);
    return cudaGetLastError();
}

cudaError_t launch_topk_sort(const TopkKlBwdLayout& lay, uint8_t* ws, const int* n_rows, int N, int K,
                             int V, TopkRows* out, cudaStream_t stream) {
    const int64_t entries = static_cast<int64_t>(N) * K;
    const int tiles = static_cast<int>(lay.tiles);
    uint32_t* key[2];
    uint32_t* slot[2];
    for (int i = 0; i < 2; ++i) {
        key[i] = reinterpret_cast<uint32_t*>(ws + lay.key_off[i]);
        slot[i] = reinterpret_cast<uint32_t*>(ws + lay.slot_off[i]);
    }
    uint32_t* hist = reinterpret_cast<uint32_t*>(ws + lay.hist_off);
    Pairs in{reinterpret_cast<const int*>(ws + lay.ids_off), nullptr, nullptr, n_rows, entries, N, K, V};
    int at = 0;
    for (int shift = 0; shift < 32 && (V >> shift) != 0; shift += kRadixBits, at ^= 1) {
        radix_count_kernel<<<tiles, kSortThreads, 0, stream>>>(in, shift, hist, tiles);
        radix_scan_kernel<<<1, 1024, 0, stream>>>(hist, static_cast<int64_t>(tiles) * kRadix);
        radix_place_kernel<<<tiles, kSortThreads, 0, stream>>>(in, shift, hist, tiles, key[at],
                                                               slot[at]);
        in.key = key[at];
        in.slot = slot[at];
    }
    int* first = reinterpret_cast<int*>(ws + lay.first_off);
    int* last = reinterpret_cast<int*>(ws + lay.last_off);
    int* row = reinterpret_cast<int*>(key[at]);          // the buffers that the last pass read
    float* rest = reinterpret_cast<float*>(slot[at]);
    const int chunks = (V + kBwdChunk - 1) / kBwdChunk;
    cudaError_t e = cudaMemsetAsync(last, 0, static_cast<size_t>(V) * 4, stream);
    if (e != cudaSuccess) return e;
    topk_entries_kernel<<<static_cast<unsigned>((entries + 255) / 256), 256, 0, stream>>>(
        in.key, in.slot, reinterpret_cast<const float*>(ws + lay.val_off), entries, K,
        static_cast<uint32_t>(V), row, rest, first, last);
    int* row_at = reinterpret_cast<int*>(ws + lay.at_off);
    int* list = reinterpret_cast<int*>(ws + lay.list_off);
    int* many = reinterpret_cast<int*>(ws + lay.many_off);
    int2* counts = reinterpret_cast<int2*>(ws + lay.counts_off);
    topk_index_kernel<<<chunks, 1024, 0, stream>>>(first, last, V, row_at, list, many, counts);
    *out = TopkRows{row, rest, first, last, row_at, list, many, counts, ws + lay.sums_off,
                    static_cast<int>(lay.places)};
    return cudaGetLastError();
}

}  // namespace rlk
