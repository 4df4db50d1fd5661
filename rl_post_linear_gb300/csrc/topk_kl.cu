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
// entries, and the dh and dW GEMMs.
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

// The chunk's listed entries, over what the GEMM wrote there.
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
        const __nv_bfloat16 hi = __float2bfloat16_rn(d);
        __nv_bfloat16* at = ds + (e / K) * (2 * kBwdChunk) + (id - c0);
        at[0] = hi;
        at[kBwdChunk] = __float2bfloat16_rn(d - __bfloat162float(hi));
    }
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
                                int c0, int width, void* ds, cudaStream_t stream) {
    const size_t blocks = (static_cast<size_t>(N) * K + 255) / 256, most = 152 * 8;
    const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
    return launch_early(topk_scatter_kernel, dim3(grid), 256, 0, stream, nullptr, ids, val, n_rows, N,
                        K, c0, width, static_cast<__nv_bfloat16*>(ds));
}

}  // namespace rlk
