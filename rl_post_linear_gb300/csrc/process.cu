// process.cu -- penalties for repeated tokens, biases and masks on logits.
//
// What a rollout does to a row of logits x_v before it draws from it (the logits that
// rlk_sample_logits takes).  With a row's tokens (the prompt, then what was drawn), c_v how
// often v was drawn, repetition penalty r, frequency penalty f, presence penalty p:
//
//   x = x > 0 ? x / r : x r          where v is among the row's tokens
//   x = x - f c_v - p                where c_v > 0
//   x = x + sum of the biases of v   (ascending slots)
//   x = -inf                         where the mask's bit of v is 0
//
// A block takes a range of columns of one row.  It counts the row's tokens that fall into its
// range in a table in shared memory (whole numbers, so the order of the atomics does not
// matter), then streams its columns once.
#include <cuda_bf16.h>

#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

constexpr int kThreads = 256;
constexpr int kColumns = 8192;           // of a block
// a column's word in the table
constexpr uint32_t kInPrompt = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& to, float v) { to = v; }
__device__ __forceinline__ void put(__nv_bfloat16& to, float v) { to = __float2bfloat16_rn(v); }

template <typename T>
__global__ void __launch_bounds__(kThreads) process_kernel(const ProcessArgs a, int ranges) {
    constexpr int VEC = 16 / sizeof(T);
    extern __shared__ uint32_t table[];          // [kColumns], then the biases' ids
    int* bias_id = reinterpret_cast<int*>(table + kColumns);
    const int row = blockIdx.x / ranges, range = blockIdx.x % ranges;
    if (a.mask != nullptr && a.mask[row] == 0) return;
    const int tid = threadIdx.x;
    const int c0 = range * kColumns, cols = min(kColumns, a.V - c0);
    const float rep = a.repetition_rows != nullptr ? a.repetition_rows[row] : a.repetition;
    const float freq = a.frequency_rows != nullptr ? a.frequency_rows[row] : a.frequency;
    const float pres = a.presence_rows != nullptr ? a.presence_rows[row] : a.presence;
    uint32_t bad = 0;
    if (!(rep > 0.f && rep < INFINITY) || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY))
        bad = RLK_DEVERR_SAMPLE_PARAM;
    int64_t len = 0, prompt = 0;
    if (a.tokens != nullptr) {
        len = a.lengths != nullptr ? a.lengths[row] : a.width;
        prompt = a.prompt_lengths != nullptr ? a.prompt_lengths[row] : 0;
        if (prompt < 0 || len < prompt || len > a.width) {
            bad |= RLK_DEVERR_SAMPLE_PARAM;
            len = prompt = 0;
        }
    }
    const bool listed = len > 0 || a.bias > 0;
    if (listed) {
        for (int i = tid; i < kColumns; i += kThreads) table[i] = 0;
        __syncthreads();
        const int64_t* tokens = a.tokens + static_cast<int64_t>(row) * a.tokens_stride;
        for (int64_t i = tid; i < len; i += kThreads) {
            const int64_t id = tokens[i];
            if (id >= a.V) bad |= RLK_DEVERR_TARGET_RANGE;
            if (id < c0 || id >= c0 + cols) continue;
            if (i < prompt)
                atomicOr(&table[id - c0], kInPrompt);
            else
                atomicAdd(&table[id - c0], 1u);
        }
        for (int i = tid; i < a.bias; i += kThreads) {
            const int64_t id = a.bias_ids[static_cast<int64_t>(row) * a.bias + i];
            if (id >= a.V) bad |= RLK_DEVERR_TARGET_RANGE;
            const bool mine = id >= c0 && id < c0 + cols;
            bias_id[i] = mine ? static_cast<int>(id) - c0 : -1;
            if (mine) atomicOr(&table[id - c0], kBiased);
        }
    }
    if (bad != 0 && range == 0 && a.err != nullptr) atomicOr(a.err, bad);
    const bool broken = __syncthreads_or(bad != 0) != 0;

    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + c0;
    T* out = static_cast<T*>(a.out) + row * a.out_stride + c0;
    const int32_t* allowed =
        a.allowed != nullptr ? a.allowed + row * a.allowed_stride + c0 / 32 : nullptr;
    const float* bias = a.bias_values + static_cast<int64_t>(row) * a.bias;
    for (int c = tid * VEC; c < cols; c += kThreads * VEC) {
        const bool whole = c + VEC <= cols;
        alignas(16) T v[VEC];
        if (a.x_vec && whole) {
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(x + c);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c + e < cols) v[e] = x[c + e];
        }
        const uint32_t bits =
            allowed != nullptr ? static_cast<uint32_t>(allowed[c / 32]) >> (c % 32) : ~0u;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float f = to_f32(v[e]);
            const uint32_t w = listed && c + e < cols ? table[c + e] : 0;
            if (w != 0) {
                if ((w & ~kBiased) != 0) f = f > 0.f ? __fdiv_rn(f, rep) : f * rep;
                const uint32_t n = w & kCount;
                if (n != 0) f = fmaf(-freq, static_cast<float>(n), f) - pres;
                if (w & kBiased) {
                    float sum = 0.f;
                    for (int i = 0; i < a.bias; ++i)
                        if (bias_id[i] == c + e) sum += bias[i];
                    f += sum;
                }
            }
            if (!((bits >> e) & 1u)) f = -INFINITY;
            if (broken) f = __int_as_float(0x7fc00000);
            put(v[e], f);
        }
        if (a.out_vec && whole) {
            *reinterpret_cast<uint4*>(out + c) = *reinterpret_cast<const uint4*>(v);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c + e < cols) out[c + e] = v[e];
        }
    }
}

}  // namespace

cudaError_t launch_process(const ProcessArgs& a, bool bf16, cudaStream_t stream) {
    const int ranges = (a.V + kColumns - 1) / kColumns;
    const int64_t blocks = static_cast<int64_t>(a.N) * ranges;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const size_t smem = kColumns * 4 + static_cast<size_t>(a.bias) * 4;   // at most 48 KB
    static_assert(kColumns * 4 + kMaxBias * 4 <= 48 * 1024, "a block's shared memory");
    const unsigned grid = static_cast<unsigned>(blocks);
    if (bf16)
        process_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(a, ranges);
    else
        process_kernel<float><<<grid, kThreads, smem, stream>>>(a, ranges);
    return cudaGetLastError();
}

}  // namespace rlk
