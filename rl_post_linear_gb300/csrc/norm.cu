// norm.cu -- layer norm and RMS norm, forward and backward.
//
// The final norm in front of the LM head ("RL-Kernel Roadmap (2026)", WS1:
// batch-invariant RMSNorm forward and backward next to the batch-invariant
// log-prob).  Row t of x has H columns, fp32 or bf16; all arithmetic is fp32:
//
//   mean = sum x / H (layer norm; 0 for RMS norm)
//   rstd = 1 / sqrt( sum (x - mean)^2 / H + eps )
//   y    = (x - mean) rstd w + b
//
// The variance is summed from the centred values, so a large mean costs no
// digits.  Backward, with xh = (x - mean) rstd and g = dy w:
//
//   dx = rstd ( g - mean_H(g) - xh mean_H(g xh) )     (no mean_H(g) for RMS norm)
//   dw = sum_t dy xh      db = sum_t dy
//
// Both directions are bound by HBM: x in, y out; x and dy in, dx out.  A block takes row
// after row and holds one in registers between its reductions, so each is read once; the
// next rows are on their way into shared memory meanwhile (cp.async, a row or two ahead).
// Each thread copies just what it reads itself, so this needs no barrier.  Measured (bf16;
// the bytes that have to move over the time, against the 6.8 TB/s of a plain copy): layer
// norm [8192, 4096] 23.8 us, 5.6 TB/s, and 39.3 us, 5.1 TB/s, backward with dw and db; RMS
// norm [16384, 7168] with a fifth masked 69.3 us, 6.1 TB/s, and 112 us, 5.5 TB/s.  One row or
// 64 take 2.0 to 2.5 us, about what a launch costs.
//
// Columns are dealt in groups of 8: thread j of the row's `threads` owns groups j and
// j + threads and folds them in that order, then a fixed shuffle tree and the warps in
// order.  The number of threads follows from H alone, and the way a group is copied (16
// bytes at a time, 4 bytes, or element by element, as the rows are aligned) does not change
// the order: a row's results do not depend on N, its position, the mask or the alignment.
//
// dw and db: block b of a number of blocks fixed by N and H takes rows b, b + blocks, ...
// in ascending order, adds them up in registers (each thread its own columns)
// and writes one fp32 partial row; a second launch adds the partial rows in a
// fixed tree (4 to 5 us by itself).  No atomics: bitwise reproducible.
#include <cuda_bf16.h>

#include <algorithm>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

constexpr int kGroup = 8;   // columns of one group

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Two columns at a time: sm_100's paired fp32 instructions, each half rounded as the single
// instruction rounds.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// One group of 8 columns as it lies in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
        const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) w[e / 2] |= uint32_t(__ldcs(q + e)) << (16 * (e & 1));
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        f[0] = make_float2(bf_lo(a.x), bf_hi(a.x)), f[1] = make_float2(bf_lo(a.y), bf_hi(a.y));
        f[2] = make_float2(bf_lo(a.z), bf_hi(a.z)), f[3] = make_float2(bf_lo(a.w), bf_hi(a.w));
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        f[0] = bf_lo(a.x), f[1] = bf_hi(a.x), f[2] = bf_lo(a.y), f[3] = bf_hi(a.y);
        f[4] = bf_lo(a.z), f[5] = bf_hi(a.z), f[6] = bf_lo(a.w), f[7] = bf_hi(a.w);
    }
};
template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void load_some(const float* p, int n) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < n ? __ldcs(p + e) : 0.f;
        a = make_float4(w[0], w[1], w[2], w[3]);
        b = make_float4(w[4], w[5], w[6], w[7]);
    }
    __device__ __forceinline__ void unpack(float2 (&f)[4]) const {
        f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};

// valid columns of the group that starts at column c
__device__ __forceinline__ int valid_cols(int c, int H) { return min(kGroup, max(0, H - c)); }

template <typename T>
__device__ __forceinline__ void load_group(Raw<T>& r, const T* row, int c, int H, bool vec) {
    const int n = valid_cols(c, H);
    if (n == kGroup && vec)
        r.load(row + c);
    else if (n > 0)
        r.load_some(row + c, n);
    else
        r.zero();
}

__device__ __forceinline__ void store_group(__nv_bfloat16* row, int c, int H, bool vec,
                                            const float (&f)[8]) {
    const int n = valid_cols(c, H);
    if (n == kGroup && vec) {
        __stcs(reinterpret_cast<uint4*>(row + c),
               make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                          pack_bf16(f[6], f[7])));
        return;
    }
#pragma unroll
    for (int e = 0; e < kGroup; ++e)
        if (e < n) row[c + e] = __float2bfloat16_rn(f[e]);
}
__device__ __forceinline__ void store_group(float* row, int c, int H, bool vec,
                                            const float (&f)[8]) {
    const int n = valid_cols(c, H);
    // whole sectors at once where the rows allow it ([4096, 4096] RMS norm 21.4 instead of 22.9 us)
    if (n == kGroup && (reinterpret_cast<uintptr_t>(row) & 31) == 0) {
        asm volatile("st.global.cs.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + c),
                     "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]),
                     "f"(f[7])
                     : "memory");
        return;
    }
    if (n == kGroup && vec) {
        __stcs(reinterpret_cast<float4*>(row + c), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(row + c) + 1, make_float4(f[4], f[5], f[6], f[7]));
        return;
    }
#pragma unroll
    for (int e = 0; e < kGroup; ++e)
        if (e < n) row[c + e] = f[e];
}

template <typename T>
__device__ __forceinline__ void store_group(T* row, int c, int H, bool vec, const float2 (&f)[4]) {
    const float v[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
    store_group(row, c, H, vec, v);
}
template <typename T>
__device__ __forceinline__ void zero_row(T* row, int H, bool vec) {
    const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int c = threadIdx.x * kGroup; c < H; c += blockDim.x * kGroup)
        store_group(row, c, H, vec, z);
}

// weight / bias group: read by every row, so kept in L1 (default caching)
__device__ __forceinline__ void param_group(const void* p, bool bf16, bool vec, int c, int H,
                                            float (&f)[8]) {
    const int n = valid_cols(c, H);
    if (bf16) {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + c;
        if (n == kGroup && vec) {
            Raw<__nv_bfloat16> r;
            r.a = __ldg(reinterpret_cast<const uint4*>(q));
            r.unpack(f);
            return;
        }
#pragma unroll
        for (int e = 0; e < kGroup; ++e) f[e] = e < n ? __bfloat162float(q[e]) : 0.f;
    } else {
        const float* q = static_cast<const float*>(p) + c;
        if (n == kGroup && vec) {
            Raw<float> r;
            r.a = __ldg(reinterpret_cast<const float4*>(q));
            r.b = __ldg(reinterpret_cast<const float4*>(q) + 1);
            r.unpack(f);
            return;
        }
#pragma unroll
        for (int e = 0; e < kGroup; ++e) f[e] = e < n ? __ldg(q + e) : 0.f;
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sums over the block's threads, in every thread: lanes by a shuffle tree, then the warps by
// another one.  `slot` alternates between consecutive calls, so one barrier a call suffices.
template <int MAXT>
__device__ __forceinline__ float row_sum(float a, float2 (*slots)[32], int& slot) {
    a = warp_sum(a);
    if (blockDim.x == 32) return a;
    float2* s = slots[slot];
    slot ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5].x = a;
    __syncthreads();
    a = lane < (blockDim.x >> 5) ? s[lane].x : 0.f;
#pragma unroll
    for (int off = MAXT / 64; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    return __shfl_sync(0xffffffffu, a, 0);
}
template <int MAXT>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*slots)[32], int& slot) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (blockDim.x == 32) return make_float2(a, b);
    float2* s = slots[slot];
    slot ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = lane < (blockDim.x >> 5) ? s[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int off = MAXT / 64; off > 0; off >>= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, off);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, off);
    }
    return make_float2(__shfl_sync(0xffffffffu, t.x, 0), __shfl_sync(0xffffffffu, t.y, 0));
}

// A partial row of dw or db holds element e of the i-th group of thread t at place
// (8 i + e) threads + t, whose column is 8 (t + i threads) + e.
__host__ __device__ constexpr int64_t part_len(int64_t H, int threads) {
    return (H + threads * kGroup - 1) / (threads * kGroup) * (threads * kGroup);
}

// Copies of a group into shared memory: how the rows are aligned.
enum : int { kCopy16, kCopy4, kCopyPlain };

__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int bytes, bool wide) {
    // The rest of the 16 (4) bytes is filled with zeros.  Through L1: the two halves of a group of
    // fp32 come one after the other, and the second finds its sectors there (fp32 [4096, 4096] a
    // quarter less time than past L1, bf16 the same either way).
    if (wide)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                     : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest LEFT groups have arrived
template <int LEFT>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Groups of a thread: two keep the forward at 64 registers and the backward at 128 (with
// four, [8192, 4096] takes 37.8 instead of 23.8 us, its backward 56 instead of 39).
constexpr int kGroups = 2;
// Rows that a block has in shared memory, the one it works on among them.  The forward gains
// nothing from a third row (24 us at [8192, 4096] either way, but 89 instead of 69 us at
// [16384, 7168] with a fifth masked), the backward nothing from a fourth (39.7 and 39.3 us,
// 114 and 112).
template <typename T, int MAXT, int TENSORS>
__host__ __device__ constexpr int stages_of() {
    return TENSORS == 1 ? 2 : MAXT == 512 || sizeof(T) == 2 ? 3 : 1;
}

// A thread's part of a ring of rows in shared memory: `stages` slots of kGroups groups.
// 16-byte piece p of slot s lies at (s pieces + p) threads + tid, so the threads of a warp
// touch neighbouring pieces.
template <typename T>
struct Ring {
    static constexpr int kPieces = kGroups * kGroup * sizeof(T) / 16;
    uint4* base;
    __device__ __forceinline__ uint4* piece(int stage, int p) const {
        return base + (stage * kPieces + p) * blockDim.x + threadIdx.x;
    }
    // fit: as at the forward kernel below
    __device__ __forceinline__ void fetch(const T* row, int stage, int H, int mode,
                                          int fit) const {
        constexpr int kPerGroup = kPieces / kGroups, kElems = kGroup / kPerGroup;
        if (fit == 2) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
                cp_async(smem_u32(piece(stage, p)),
                         row + (threadIdx.x + p / kPerGroup * blockDim.x) * kGroup +
                             p % kPerGroup * kElems,
                         16, true);
            return;
        }
        if (fit == 1) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
                const int c = (threadIdx.x + p / kPerGroup * blockDim.x) * kGroup;
                cp_async(smem_u32(piece(stage, p)), c < H ? row + c + p % kPerGroup * kElems : row,
                         c < H ? 16 : 0, true);
            }
            return;
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const int c = (threadIdx.x + p / kPerGroup * blockDim.x) * kGroup +
                          p % kPerGroup * kElems;
            const int n = min(kElems, max(0, H - c));
            const T* src = n > 0 ? row + c : row;
            const uint32_t dst = smem_u32(piece(stage, p));
            if (mode == kCopy16) {
                cp_async(dst, src, n * int(sizeof(T)), true);
            } else if (mode == kCopy4 && sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < kElems; ++e)
                    cp_async(dst + 4 * e, e < n ? src + e : row, e < n ? 4 : 0, false);
            } else {
                alignas(16) T v[kElems];             // read as one piece
#pragma unroll
                for (int e = 0; e < kElems; ++e) v[e] = e < n ? src[e] : T(0.f);
                *piece(stage, p) = *reinterpret_cast<const uint4*>(v);
            }
        }
    }
    __device__ __forceinline__ Raw<T> group(int stage, int i) const;
};
template <>
__device__ __forceinline__ Raw<__nv_bfloat16> Ring<__nv_bfloat16>::group(int stage, int i) const {
    Raw<__nv_bfloat16> r;
    r.a = *piece(stage, i);
    return r;
}
template <>
__device__ __forceinline__ Raw<float> Ring<float>::group(int stage, int i) const {
    Raw<float> r;
    r.a = *reinterpret_cast<const float4*>(piece(stage, 2 * i));
    r.b = *reinterpret_cast<const float4*>(piece(stage, 2 * i + 1));
    return r;
}

// mask byte of a row: 0 past the end
__device__ __forceinline__ int mask_byte(const uint8_t* mask, int row, int N) {
    return row >= N ? 0 : mask == nullptr ? 1 : __ldg(mask + row);
}

// The forward of a row in registers: two block reductions for layer norm, one for RMS norm, and
// two blocks or more of up to 512 threads on an SM, so that one reduces while another moves data.
// FIT: every row starts on 16 bytes and H is 16 columns for each thread (2), so that no column
// needs a test, or whole groups (1), so that a group does; otherwise (0) each column.  The
// arithmetic is the same (bf16 [8000, 1664] 13.5 us with 1, 15.1 with 0).
template <typename T, bool CENTER, int MAXT, int FIT>
__global__ void __launch_bounds__(MAXT, MAXT == 1024 ? 1 : 2)
    norm_fwd_kernel(const NormArgs a, int x_mode, float inv_h) {
    constexpr int S = stages_of<T, MAXT, 1>();
    extern __shared__ uint4 ring_smem[];
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int tid = threadIdx.x, H = a.H;
    const bool out_vec = FIT > 0 || a.out_vec;
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.out);
    const uint8_t* mask = a.mask;
    const void *weight = a.weight, *bias = a.bias;
    wait_previous(x, mask, weight, bias);
    const Ring<T> ring{ring_smem};
    // Row indices leave room for S more steps below 2^31.  S - 1 rows are on their way before
    // the first is waited for; `bits` says which of them are active, `next` whether the row
    // after them is.
    const int step = gridDim.x;
    int row = blockIdx.x, next;
    uint32_t bits = 0;
    const T* ahead = x + row * a.x_stride;           // the row to fetch next
    T* yr = y + row * a.out_stride;
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
        if (mask_byte(mask, row + k * step, a.N)) {
            ring.fetch(ahead, k, H, x_mode, FIT);
            bits |= 1u << k;
        }
        cp_commit();
        ahead += step * a.x_stride;
    }
    next = mask_byte(mask, row + (S - 1) * step, a.N);
    float2 w[kGroups][4], b[kGroups][4];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int c = (tid + i * blockDim.x) * kGroup;
        float v[8];
        param_group(weight, a.w_bf16, a.w_vec, c, H, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = make_float2(v[2 * e], v[2 * e + 1]), b[i][e] = both(0.f);
        if (bias != nullptr) {
            param_group(bias, a.w_bf16, a.w_vec, c, H, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) b[i][e] = make_float2(v[2 * e], v[2 * e + 1]);
        }
    }
    int stage = 0;
    for (; row < a.N; row += step, yr += step * a.out_stride) {
        if (next) {
            ring.fetch(ahead, stage == 0 ? S - 1 : stage - 1, H, x_mode, FIT);
            bits |= 1u << (S - 1);
        }
        cp_commit();
        ahead += step * a.x_stride;
        next = mask_byte(mask, row + S * step, a.N);
        const bool on = bits & 1u;
        bits >>= 1;
        const int at = stage;
        stage = stage + 1 == S ? 0 : stage + 1;
        if (!on) {
            zero_row(yr, H, out_vec);
            if (tid == 0) {
                if (a.mean_out != nullptr) a.mean_out[row] = 0.f;
                if (a.rstd_out != nullptr) a.rstd_out[row] = 0.f;
            }
            continue;
        }
        cp_wait<S - 1>();
        float2 f[kGroups][4], s = both(0.f);
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            ring.group(at, i).unpack(f[i]);
            if (CENTER)
#pragma unroll
                for (int e = 0; e < 4; ++e) s = __fadd2_rn(s, f[i][e]);   // columns past H hold 0
        }
        if (CENTER) mean = row_sum<MAXT>(s.x + s.y, slots, slot) * inv_h;
        float2 q = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int n = valid_cols((tid + i * blockDim.x) * kGroup, H);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (CENTER) {
                    f[i][e] = __fadd2_rn(f[i][e], both(-mean));
                    if (FIT == 1 && n == 0) f[i][e] = both(0.f);
                    if (FIT == 0 && 2 * e >= n) f[i][e].x = 0.f;
                    if (FIT == 0 && 2 * e + 1 >= n) f[i][e].y = 0.f;
                }
                q = __ffma2_rn(f[i][e], f[i][e], q);
            }
        }
        const float var = row_sum<MAXT>(q.x + q.y, slots, slot) * inv_h;
        const float rstd = rsqrtf(var + a.eps);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = (tid + i * blockDim.x) * kGroup;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[i][e] = __ffma2_rn(__fmul2_rn(f[i][e], both(rstd)), w[i][e], b[i][e]);
            if (FIT == 2 || c < H) store_group(yr, c, FIT > 0 ? c + kGroup : H, out_vec, f[i]);
        }
        if (tid == 0) {
            if (a.mean_out != nullptr) a.mean_out[row] = mean;
            if (a.rstd_out != nullptr) a.rstd_out[row] = rstd;
        }
    }
}

// Rows too wide for registers (H > 16384): the same sums, with the row read again, from L2
// mostly, for each step.
template <typename T, bool CENTER>
__global__ void __launch_bounds__(1024)
    norm_fwd_wide_kernel(const T* __restrict__ x, int64_t x_stride, bool x_vec,
                         const void* __restrict__ weight, const void* __restrict__ bias,
                         bool w_bf16, bool w_vec, const uint8_t* __restrict__ mask, int N, int H,
                         float inv_h, float eps, T* __restrict__ y, int64_t y_stride, bool y_vec,
                         float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int64_t row = blockIdx.x;
    T* yr = y + row * y_stride;
    const T* xr = x + row * x_stride;
    const int c0 = threadIdx.x * kGroup;
    constexpr int kStep = 1024 * kGroup;
    const bool live = mask == nullptr || mask[row] != 0;
    float mean = 0.f, rstd = 0.f;
    Raw<T> raw;
    if (live) {
        if (CENTER) {
            float s = 0.f;
            for (int c = c0; c < H; c += kStep) {
                float f[8];
                load_group(raw, xr, c, H, x_vec);
                raw.unpack(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += f[e];
            }
            mean = row_sum<1024>(s, slots, slot) * inv_h;
        }
        float q = 0.f;
        for (int c = c0; c < H; c += kStep) {
            float f[8];
            load_group(raw, xr, c, H, x_vec);
            raw.unpack(f);
            const int n = valid_cols(c, H);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = f[e] - mean;
                if (e < n) q = fmaf(d, d, q);
            }
        }
        const float var = row_sum<1024>(q, slots, slot) * inv_h;
        rstd = rsqrtf(var + eps);
    }
    for (int c = c0; c < H; c += kStep) {
        float f[8] = {0, 0, 0, 0, 0, 0, 0, 0}, w[8], b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (live) {
            load_group(raw, xr, c, H, x_vec);
            raw.unpack(f);
            param_group(weight, w_bf16, w_vec, c, H, w);
            if (bias != nullptr) param_group(bias, w_bf16, w_vec, c, H, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[e], b[e]);
        }
        store_group(yr, c, H, y_vec, f);
    }
    if (threadIdx.x == 0) {
        if (mean_out != nullptr) mean_out[row] = mean;
        if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
}

// ----------------------------------------------------------------------------- backward

// The backward of a row in registers, with the block's part of dw and db: 64 floats a thread for
// the two tensors' groups, w and the sums, hence one block of 512 threads (or two of 256) on an
// SM.  One reduction of both means.
template <typename T, bool CENTER, int MAXT, int FIT>
__global__ void __launch_bounds__(MAXT, 1)
    norm_bwd_kernel(const NormArgs a, int x_mode, int dy_mode, float inv_h,
                    float* __restrict__ dw_part, float* __restrict__ db_part) {
    constexpr int S = stages_of<T, MAXT, 2>();
    extern __shared__ uint4 ring_smem[];
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int tid = threadIdx.x, H = a.H;
    const bool out_vec = FIT > 0 || a.out_vec;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.out);
    const uint8_t* mask = a.mask;
    const void* weight = a.weight;
    wait_previous(x, dy, mask, weight);
    const Ring<T> rx{ring_smem}, rg{ring_smem + S * Ring<T>::kPieces * blockDim.x};
    const int step = gridDim.x;
    int row = blockIdx.x, next;
    uint32_t bits = 0;
    const T* x_ahead = x + row * a.x_stride;
    const T* g_ahead = dy + row * a.dy_stride;
    T* dxr = dx + row * a.out_stride;
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
        if (mask_byte(mask, row + k * step, a.N)) {
            rx.fetch(x_ahead, k, H, x_mode, FIT);
            rg.fetch(g_ahead, k, H, dy_mode, FIT);
            bits |= 1u << k;
        }
        cp_commit();
        x_ahead += step * a.x_stride;
        g_ahead += step * a.dy_stride;
    }
    next = mask_byte(mask, row + (S - 1) * step, a.N);
    float2 w[kGroups][4], dw[kGroups][4], db[kGroups][4];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        float v[8];
        param_group(weight, a.w_bf16, a.w_vec, (tid + i * blockDim.x) * kGroup, H, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[i][e] = make_float2(v[2 * e], v[2 * e + 1]);
            dw[i][e] = db[i][e] = both(0.f);
        }
    }
    // the statistics of a row are read one row early
    float rstd_next = a.rstd[row], mean_next = CENTER ? a.mean[row] : 0.f;
    int stage = 0;
    for (; row < a.N; row += step, dxr += step * a.out_stride) {
        if (next) {
            const int to = stage == 0 ? S - 1 : stage - 1;
            rx.fetch(x_ahead, to, H, x_mode, FIT);
            rg.fetch(g_ahead, to, H, dy_mode, FIT);
            bits |= 1u << (S - 1);
        }
        cp_commit();
        x_ahead += step * a.x_stride;
        g_ahead += step * a.dy_stride;
        next = mask_byte(mask, row + S * step, a.N);
        const bool on = bits & 1u;
        bits >>= 1;
        const int at = stage;
        stage = stage + 1 == S ? 0 : stage + 1;
        const float rstd = rstd_next, mean = mean_next;
        if (row + step < a.N) {
            rstd_next = a.rstd[row + step];
            if (CENTER) mean_next = a.mean[row + step];
        }
        if (!on) {
            zero_row(dxr, H, out_vec);
            continue;
        }
        cp_wait<S - 1>();
        float2 xh[kGroups][4], g[kGroups][4], s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            rx.group(at, i).unpack(xh[i]);
            rg.group(at, i).unpack(g[i]);       // dy past H is 0: these columns add nothing
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (CENTER) xh[i][e] = __fadd2_rn(xh[i][e], both(-mean));
                xh[i][e] = __fmul2_rn(xh[i][e], both(rstd));
                dw[i][e] = __ffma2_rn(g[i][e], xh[i][e], dw[i][e]);
                if (CENTER) db[i][e] = __fadd2_rn(db[i][e], g[i][e]);
                g[i][e] = __fmul2_rn(g[i][e], w[i][e]);
                if (CENTER) s1 = __fadd2_rn(s1, g[i][e]);
                s2 = __ffma2_rn(g[i][e], xh[i][e], s2);
            }
        }
        float2 t;
        if (CENTER)
            t = row_sum<MAXT>(s1.x + s1.y, s2.x + s2.y, slots, slot);
        else
            t = make_float2(0.f, row_sum<MAXT>(s2.x + s2.y, slots, slot));
        const float m1 = t.x * inv_h, m2 = t.y * inv_h;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int c = (tid + i * blockDim.x) * kGroup;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (CENTER) g[i][e] = __fadd2_rn(g[i][e], both(-m1));
                g[i][e] = __fmul2_rn(__ffma2_rn(xh[i][e], both(-m2), g[i][e]), both(rstd));
            }
            if (FIT == 2 || c < H) store_group(dxr, c, FIT > 0 ? c + kGroup : H, out_vec, g[i]);
        }
    }
    // the block's partial row, in the order of part_len: neighbouring threads write
    // neighbouring floats
    const int64_t out = int64_t(blockIdx.x) * (blockDim.x * kGroups * 8) + tid;
#pragma unroll
    for (int i = 0; i < kGroups * 4; ++i) {
        const float2 vw = dw[i / 4][i % 4], vb = db[i / 4][i % 4];
        const int64_t at = out + 2 * i * blockDim.x;
        if (dw_part != nullptr) dw_part[at] = vw.x, dw_part[at + blockDim.x] = vw.y;
        if (CENTER && db_part != nullptr) db_part[at] = vb.x, db_part[at + blockDim.x] = vb.y;
    }
}

// Rows too wide for registers: the partial sums live in the block's partial row itself.
template <typename T, bool CENTER>
__global__ void __launch_bounds__(1024)
    norm_bwd_wide_kernel(const T* __restrict__ x, int64_t x_stride, const T* __restrict__ dy,
                         int64_t dy_stride, bool in_vec, const void* __restrict__ weight,
                         bool w_bf16, bool w_vec, const float* __restrict__ mean_in,
                         const float* __restrict__ rstd_in, const uint8_t* __restrict__ mask,
                         int N, int H, float inv_h, T* __restrict__ dx, int64_t dx_stride,
                         bool dx_vec, float* __restrict__ dw_part, float* __restrict__ db_part) {
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int c0 = threadIdx.x * kGroup;
    constexpr int kStep = 1024 * kGroup;
    // each thread owns its columns, and their places in the partial row, throughout
    const int64_t at = int64_t(blockIdx.x) * part_len(H, 1024) + threadIdx.x;
    for (int c = c0; c < H; c += kStep)
        for (int e = 0; e < 8; ++e) {
            const int64_t k = at + (int64_t(c / kStep) * 8 + e) * 1024;
            if (dw_part != nullptr) dw_part[k] = 0.f;
            if (CENTER && db_part != nullptr) db_part[k] = 0.f;
        }
    Raw<T> rx, rg;
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
        T* dxr = dx + row * dx_stride;
        const T* xr = x + row * x_stride;
        const T* gr = dy + row * dy_stride;
        if (mask != nullptr && mask[row] == 0) {
            const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int c = c0; c < H; c += kStep) store_group(dxr, c, H, dx_vec, z);
            continue;
        }
        const float rstd = rstd_in[row];
        const float mean = CENTER ? mean_in[row] : 0.f;
        float s1 = 0.f, s2 = 0.f;
        for (int c = c0; c < H; c += kStep) {
            float xf[8], gf[8], w[8];
            load_group(rx, xr, c, H, in_vec);
            load_group(rg, gr, c, H, in_vec);
            rx.unpack(xf);
            rg.unpack(gf);
            param_group(weight, w_bf16, w_vec, c, H, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xf[e] - mean) * rstd;
                const float g = gf[e] * w[e];
                if (CENTER) s1 += g;
                s2 = fmaf(g, xh, s2);
                const int64_t k = at + (int64_t(c / kStep) * 8 + e) * 1024;
                if (dw_part != nullptr) dw_part[k] = fmaf(gf[e], xh, dw_part[k]);
                if (CENTER && db_part != nullptr) db_part[k] += gf[e];
            }
        }
        const float2 t = row_sum<1024>(s1, s2, slots, slot);
        const float m1 = t.x * inv_h, m2 = t.y * inv_h;
        for (int c = c0; c < H; c += kStep) {
            float xf[8], gf[8], w[8];
            load_group(rx, xr, c, H, in_vec);
            load_group(rg, gr, c, H, in_vec);
            rx.unpack(xf);
            rg.unpack(gf);
            param_group(weight, w_bf16, w_vec, c, H, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xf[e] - mean) * rstd;
                const float d = fmaf(gf[e], w[e], CENTER ? -m1 : 0.f);
                xf[e] = fmaf(-xh, m2, d) * rstd;
            }
            store_group(dxr, c, H, dx_vec, xf);
        }
    }
}

// Column sums of the partial rows: 32 places a block, 32 threads a place (each every 32nd
// partial row, ascending), then the 32 in order.  P = 0 writes zeros.  Launched early: its
// blocks wait for the partial rows.
__global__ void __launch_bounds__(1024)
    norm_dw_merge_kernel(const float* __restrict__ dw_part, const float* __restrict__ db_part,
                         int P, int len, int threads, int H, bool bf16,
                         void* __restrict__ dweight, void* __restrict__ dbias) {
    wait_previous(dw_part, db_part);
    const float* part = blockIdx.y == 0 ? dw_part : db_part;
    void* out = blockIdx.y == 0 ? dweight : dbias;
    if (out == nullptr) return;
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int pos = blockIdx.x * 32 + x;             // len is a multiple of 32
    const int r = pos / threads;                     // the place's column: see part_len
    const int64_t c = (int64_t(r >> 3) * threads + pos % threads) * kGroup + (r & 7);
    float a = 0.f;
    if (c < H) {
        // ten loads at a time, added in ascending order
        for (int p = q; p < P; p += 320) {
            float v[10];
#pragma unroll
            for (int k = 0; k < 10; ++k)
                v[k] = p + 32 * k < P ? part[int64_t(p + 32 * k) * len + pos] : 0.f;
#pragma unroll
            for (int k = 0; k < 10; ++k) a += v[k];
        }
    }
    s[q][x] = a;
    __syncthreads();
    if (q != 0 || c >= H) return;
#pragma unroll 8
    for (int k = 1; k < 32; ++k) a += s[k][x];
    if (bf16)
        static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(a);
    else
        static_cast<float*>(out)[c] = a;
}

// The widest row that stays in registers.
constexpr int kMaxRegH = 1024 * kGroups * kGroup;

// Blocks on an SM: the forward holds 64 registers a thread, the backward up to 128.
int fwd_blocks_per_sm(int threads) { return std::max(1, std::min(16, 1024 / std::max(threads, 32))); }
int bwd_blocks_per_sm(int threads) { return std::max(1, std::min(16, 512 / std::max(threads, 32))); }

// The threads of a row follow from H alone; 0: the wide kernels.
int threads_of(int64_t H) {
    if (H > kMaxRegH) return 0;
    const int64_t half = (H + kGroups * kGroup - 1) / (kGroups * kGroup);
    return static_cast<int>((half + 31) / 32 * 32);
}

// Blocks (= partial rows) of the backward and floats of a partial row: fixed by H and N.  As many
// as run at the same time, but from 152 on each takes four rows or more, so that the partial rows
// stay a small part of the traffic (bf16 [1600, 1024] 7.3 us, 10.0 with a row a block; [4000, 256]
// 8.1 and 10.7; [800, 4096] 9.5 and 9.2).
struct Parts {
    int threads, blocks;
    int64_t len;
};
Parts bwd_parts(int64_t N, int64_t H) {
    const int t = threads_of(H);
    const int64_t most = 152 * (t == 0 ? 1 : bwd_blocks_per_sm(t));
    const int64_t blocks = std::min<int64_t>(most, std::max<int64_t>(152, N / 4));
    return {t == 0 ? 1024 : t, static_cast<int>(std::min<int64_t>(N, blocks)),
            part_len(H, t == 0 ? 1024 : t * kGroups)};
}

int copy_mode(const void* p, int64_t stride, size_t esize) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a % 16 == 0 && size_t(stride) * esize % 16 == 0) return kCopy16;
    return esize == 4 ? kCopy4 : kCopyPlain;
}

// A block's shared memory beyond 48 KB is asked for: always the most that the kernel may need, as
// another thread's call with narrower rows may come between this and the launch.
template <typename F>
cudaError_t allow_smem(F kernel, size_t smem, size_t most) {
    if (smem <= 47 * 1024) return cudaSuccess;      // with the static part below 48 KB
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(most));
}

int fit_of(const NormArgs& a, int threads) {
    if (!a.in_vec || !a.out_vec || a.H % kGroup != 0) return 0;
    return a.H == threads * kGroups * kGroup ? 2 : 1;
}

template <typename T, bool CENTER, int MAXT>
cudaError_t run_fwd(const NormArgs& a, int threads, cudaStream_t stream) {
    const int fit = fit_of(a, threads);
    auto kernel = fit == 2   ? norm_fwd_kernel<T, CENTER, MAXT, 2>
                  : fit == 1 ? norm_fwd_kernel<T, CENTER, MAXT, 1>
                             : norm_fwd_kernel<T, CENTER, MAXT, 0>;
    constexpr size_t each = kGroups * kGroup * sizeof(T) * stages_of<T, MAXT, 1>();
    const size_t smem = threads * each;
    const cudaError_t e = allow_smem(kernel, smem, MAXT * each);
    if (e != cudaSuccess) return e;
    const int blocks = std::min(a.N, a.sms * fwd_blocks_per_sm(threads));
    return launch_early(kernel, dim3(blocks), threads, smem, stream, nullptr, a,
                        copy_mode(a.x, a.x_stride, sizeof(T)), 1.f / static_cast<float>(a.H));
}

template <typename T, bool CENTER>
cudaError_t fwd_dispatch(const NormArgs& a, cudaStream_t stream) {
    const int t = threads_of(a.H);
    if (t == 0) {
        norm_fwd_wide_kernel<T, CENTER><<<a.N, 1024, 0, stream>>>(
            static_cast<const T*>(a.x), a.x_stride, a.in_vec, a.weight, a.bias, a.w_bf16, a.w_vec,
            a.mask, a.N, a.H, 1.f / static_cast<float>(a.H), a.eps, static_cast<T*>(a.out),
            a.out_stride, a.out_vec, a.mean_out, a.rstd_out);
        return cudaGetLastError();
    }
    return t <= 512 ? run_fwd<T, CENTER, 512>(a, t, stream) : run_fwd<T, CENTER, 1024>(a, t, stream);
}

template <typename T, bool CENTER, int MAXT>
cudaError_t run_bwd(const NormArgs& a, int threads, int blocks, float* dwp, float* dbp,
                    cudaStream_t stream) {
    const int fit = fit_of(a, threads);
    auto kernel = fit == 2   ? norm_bwd_kernel<T, CENTER, MAXT, 2>
                  : fit == 1 ? norm_bwd_kernel<T, CENTER, MAXT, 1>
                             : norm_bwd_kernel<T, CENTER, MAXT, 0>;
    constexpr size_t each = kGroups * kGroup * sizeof(T) * 2 * stages_of<T, MAXT, 2>();
    const size_t smem = threads * each;
    const cudaError_t e = allow_smem(kernel, smem, MAXT * each);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3(blocks), threads, smem, stream, nullptr, a,
                        copy_mode(a.x, a.x_stride, sizeof(T)),
                        copy_mode(a.dy, a.dy_stride, sizeof(T)), 1.f / static_cast<float>(a.H), dwp,
                        dbp);
}

template <typename T, bool CENTER>
cudaError_t bwd_dispatch(const NormArgs& a, int blocks, float* dwp, float* dbp,
                         cudaStream_t stream) {
    const int t = threads_of(a.H);
    if (t == 0) {
        norm_bwd_wide_kernel<T, CENTER><<<blocks, 1024, 0, stream>>>(
            static_cast<const T*>(a.x), a.x_stride, static_cast<const T*>(a.dy), a.dy_stride,
            a.in_vec, a.weight, a.w_bf16, a.w_vec, a.mean, a.rstd, a.mask, a.N, a.H,
            1.f / static_cast<float>(a.H), static_cast<T*>(a.out), a.out_stride, a.out_vec, dwp,
            dbp);
        return cudaGetLastError();
    }
    return t <= 512 ? run_bwd<T, CENTER, 512>(a, t, blocks, dwp, dbp, stream)
                    : run_bwd<T, CENTER, 1024>(a, t, blocks, dwp, dbp, stream);
}

}  // namespace

size_t norm_bwd_workspace(int64_t N, int64_t H, bool center) {
    const Parts p = bwd_parts(N, H);
    return align_up(size_t(p.blocks) * p.len * sizeof(float), 256) * (center ? 2 : 1) + 256;
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool center, cudaStream_t stream) {
    if (a.bf16)
        return center ? fwd_dispatch<__nv_bfloat16, true>(a, stream)
                      : fwd_dispatch<__nv_bfloat16, false>(a, stream);
    return center ? fwd_dispatch<float, true>(a, stream) : fwd_dispatch<float, false>(a, stream);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool center, cudaStream_t stream) {
    const Parts p = bwd_parts(a.N, a.H);
    const size_t plane = align_up(size_t(p.blocks) * p.len * sizeof(float), 256);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    float* dwp = a.dweight != nullptr ? reinterpret_cast<float*>(ws) : nullptr;
    float* dbp = a.dbias != nullptr ? reinterpret_cast<float*>(ws + plane) : nullptr;
    if (a.N > 0) {
        cudaError_t e;
        if (a.bf16)
            e = center ? bwd_dispatch<__nv_bfloat16, true>(a, p.blocks, dwp, dbp, stream)
                       : bwd_dispatch<__nv_bfloat16, false>(a, p.blocks, dwp, dbp, stream);
        else
            e = center ? bwd_dispatch<float, true>(a, p.blocks, dwp, dbp, stream)
                       : bwd_dispatch<float, false>(a, p.blocks, dwp, dbp, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(p.len / 32), a.dbias != nullptr ? 2 : 1);
    return launch_early(norm_dw_merge_kernel, grid, 1024, 0, stream, nullptr,
                        static_cast<const float*>(dwp), static_cast<const float*>(dbp),
                        a.N > 0 ? p.blocks : 0, static_cast<int>(p.len), p.threads, a.H, a.w_bf16,
                        a.dweight, a.dbias);
}

}  // namespace rlk
