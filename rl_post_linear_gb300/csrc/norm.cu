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
// Both directions are bound by HBM: x in, y out; x and dy in, dx out.  A row
// stays in the registers of its threads between its two reductions, so it is
// read once.  Columns are dealt in groups of 8: thread j of the row's THREADS
// owns groups j, j + THREADS, ...  and folds them in that order, then a fixed
// shuffle tree and the warps in order.  THREADS and the groups a thread holds
// follow from H alone, and the way a group is loaded (one or two 16-byte
// loads, or element by element where rows are not 16-byte aligned or the
// group crosses H) does not change the order: a row's results do not depend
// on N, its position, the mask or the alignment.
//
// dw and db: block b of a fixed number of blocks takes rows b, b + blocks, ...
// in ascending order, adds them up in registers (each thread its own columns)
// and writes one fp32 partial row; a second launch adds the partial rows in a
// fixed tree.  No atomics: bitwise reproducible.
#include <cuda_bf16.h>

#include <algorithm>

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
    if (n == kGroup && vec) {
        __stcs(reinterpret_cast<float4*>(row + c), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(row + c) + 1, make_float4(f[4], f[5], f[6], f[7]));
        return;
    }
#pragma unroll
    for (int e = 0; e < kGroup; ++e)
        if (e < n) row[c + e] = f[e];
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

// Sums of a and b over the row's THREADS threads, in every thread: lanes by a shuffle
// tree, warps in order.  `slot` alternates between consecutive calls, so one barrier a
// call suffices.
template <int THREADS>
__device__ __forceinline__ float2 row_sum(float a, float b, float2 (*slots)[32], int& slot) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (THREADS == 32) return make_float2(a, b);
    float2* s = slots[slot];
    slot ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    float2 t = s[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) {
        t.x += s[w].x;
        t.y += s[w].y;
    }
    return t;
}

// A partial row of dw or db holds element e of the i-th group of thread t at place
// (8 i + e) threads + t, whose column is 8 (t + i threads) + e.
__host__ __device__ constexpr int64_t part_len(int64_t H, int threads) {
    return (H + threads * kGroup - 1) / (threads * kGroup) * (threads * kGroup);
}

// Rows a block of the register kernels works on side by side.
__host__ __device__ constexpr int rows_of(int threads) { return threads == 32 ? 4 : 1; }

template <typename T, bool CENTER, int THREADS, int GROUPS>
__global__ void __launch_bounds__(THREADS * rows_of(THREADS))
    norm_fwd_kernel(const T* __restrict__ x, int64_t x_stride, bool x_vec,
                    const void* __restrict__ weight, const void* __restrict__ bias, bool w_bf16,
                    bool w_vec, const uint8_t* __restrict__ mask, int N, int H, float inv_h,
                    float eps, T* __restrict__ y, int64_t y_stride, bool y_vec,
                    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = int64_t(blockIdx.x) * rows_of(THREADS) + (THREADS == 32 ? threadIdx.x >> 5 : 0);
    if (row >= N) return;
    T* yr = y + row * y_stride;
    if (mask != nullptr && mask[row] == 0) {
        const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int c = tid * kGroup; c < H; c += THREADS * kGroup) store_group(yr, c, H, y_vec, z);
        if (tid == 0) {
            if (mean_out != nullptr) mean_out[row] = 0.f;
            if (rstd_out != nullptr) rstd_out[row] = 0.f;
        }
        return;
    }
    const T* xr = x + row * x_stride;
    Raw<T> raw[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
        load_group(raw[i], xr, (tid + i * THREADS) * kGroup, H, x_vec);
    float mean = 0.f;
    if (CENTER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            float f[8];
            raw[i].unpack(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += f[e];     // columns past H hold 0
        }
        mean = row_sum<THREADS>(s, 0.f, slots, slot).x * inv_h;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        float f[8];
        raw[i].unpack(f);
        const int n = valid_cols((tid + i * THREADS) * kGroup, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = f[e] - mean;
            if (e < n) q = fmaf(d, d, q);
        }
    }
    const float var = row_sum<THREADS>(q, 0.f, slots, slot).x * inv_h;
    const float rstd = 1.f / sqrtf(var + eps);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
        const int c = (tid + i * THREADS) * kGroup;
        if (c >= H) break;
        float f[8], w[8], b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        raw[i].unpack(f);
        param_group(weight, w_bf16, w_vec, c, H, w);
        if (bias != nullptr) param_group(bias, w_bf16, w_vec, c, H, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, w[e], b[e]);
        store_group(yr, c, H, y_vec, f);
    }
    if (tid == 0) {
        if (mean_out != nullptr) mean_out[row] = mean;
        if (rstd_out != nullptr) rstd_out[row] = rstd;
    }
}

// Rows too wide for registers: the same sums, with the row read again for each step.
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
            mean = row_sum<1024>(s, 0.f, slots, slot).x * inv_h;
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
        const float var = row_sum<1024>(q, 0.f, slots, slot).x * inv_h;
        rstd = 1.f / sqrtf(var + eps);
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

template <typename T, bool CENTER, int THREADS, int GROUPS>
__global__ void __launch_bounds__(THREADS * rows_of(THREADS))
    norm_bwd_kernel(const T* __restrict__ x, int64_t x_stride, const T* __restrict__ dy,
                    int64_t dy_stride, bool in_vec, const void* __restrict__ weight, bool w_bf16,
                    bool w_vec, const float* __restrict__ mean_in,
                    const float* __restrict__ rstd_in, const uint8_t* __restrict__ mask, int N,
                    int H, float inv_h, T* __restrict__ dx, int64_t dx_stride, bool dx_vec,
                    float* __restrict__ dw_part, float* __restrict__ db_part) {
    __shared__ float2 slots[2][32];
    int slot = 0;
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int sub = THREADS == 32 ? threadIdx.x >> 5 : 0;
    float dw[GROUPS * 8], db[CENTER ? GROUPS * 8 : 1];
#pragma unroll
    for (int i = 0; i < GROUPS * 8; ++i) {
        dw[i] = 0.f;
        if (CENTER) db[i] = 0.f;
    }
    const int64_t step = int64_t(gridDim.x) * rows_of(THREADS);
    for (int64_t row = int64_t(blockIdx.x) * rows_of(THREADS) + sub; row < N; row += step) {
        T* dxr = dx + row * dx_stride;
        if (mask != nullptr && mask[row] == 0) {
            const float z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int c = tid * kGroup; c < H; c += THREADS * kGroup)
                store_group(dxr, c, H, dx_vec, z);
            continue;
        }
        Raw<T> rx[GROUPS], rg[GROUPS];
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int c = (tid + i * THREADS) * kGroup;
            load_group(rx[i], x + row * x_stride, c, H, in_vec);
            load_group(rg[i], dy + row * dy_stride, c, H, in_vec);
        }
        const float rstd = rstd_in[row];
        const float mean = CENTER ? mean_in[row] : 0.f;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int c = (tid + i * THREADS) * kGroup;
            if (c >= H) break;
            float xf[8], gf[8], w[8];
            rx[i].unpack(xf);
            rg[i].unpack(gf);          // dy past H is 0, so these columns add nothing
            param_group(weight, w_bf16, w_vec, c, H, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xf[e] - mean) * rstd;
                const float g = gf[e] * w[e];
                if (CENTER) s1 += g;
                s2 = fmaf(g, xh, s2);
                dw[i * 8 + e] = fmaf(gf[e], xh, dw[i * 8 + e]);
                if (CENTER) db[i * 8 + e] += gf[e];
            }
        }
        const float2 t = row_sum<THREADS>(s1, s2, slots, slot);
        const float m1 = t.x * inv_h, m2 = t.y * inv_h;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int c = (tid + i * THREADS) * kGroup;
            if (c >= H) break;
            float xf[8], gf[8], w[8];
            rx[i].unpack(xf);
            rg[i].unpack(gf);
            param_group(weight, w_bf16, w_vec, c, H, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (xf[e] - mean) * rstd;
                float d = fmaf(gf[e], w[e], CENTER ? -m1 : 0.f);
                xf[e] = fmaf(-xh, m2, d) * rstd;
            }
            store_group(dxr, c, H, dx_vec, xf);
        }
    }
    if (dw_part == nullptr && db_part == nullptr) return;
    // the block's partial row, in the order of part_len: neighbouring threads write
    // neighbouring floats.  Rows worked on side by side are added in order first.
    const int64_t at = int64_t(blockIdx.x) * (THREADS * GROUPS * 8);
    if (THREADS != 32) {
#pragma unroll
        for (int i = 0; i < GROUPS * 8; ++i) {
            if (dw_part != nullptr) dw_part[at + i * THREADS + tid] = dw[i];
            if (CENTER && db_part != nullptr) db_part[at + i * THREADS + tid] = db[i];
        }
    } else {
        __shared__ float acc[2][THREADS == 32 ? 32 * GROUPS * 8 : 1];
        for (int r = 0; r < rows_of(THREADS); ++r) {
            if (sub == r) {
#pragma unroll
                for (int i = 0; i < GROUPS * 8; ++i) {
                    const int k = i * 32 + tid;
                    acc[0][k] = r == 0 ? dw[i] : acc[0][k] + dw[i];
                    if (CENTER) acc[1][k] = r == 0 ? db[i] : acc[1][k] + db[i];
                }
            }
            __syncthreads();
        }
        for (int k = threadIdx.x; k < 32 * GROUPS * 8; k += blockDim.x) {
            if (dw_part != nullptr) dw_part[at + k] = acc[0][k];
            if (CENTER && db_part != nullptr) db_part[at + k] = acc[1][k];
        }
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

// Column sums of the partial rows: 32 places a block, 16 threads a place (each every 16th
// partial row, ascending), then the 16 in order.  P = 0 writes zeros.
__global__ void __launch_bounds__(512)
    norm_dw_merge_kernel(const float* __restrict__ dw_part, const float* __restrict__ db_part,
                         int P, int len, int threads, int H, bool bf16,
                         void* __restrict__ dweight, void* __restrict__ dbias) {
    const float* part = blockIdx.y == 0 ? dw_part : db_part;
    void* out = blockIdx.y == 0 ? dweight : dbias;
    if (out == nullptr) return;
    __shared__ float s[16][33];
    const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int pos = blockIdx.x * 32 + x;             // len is a multiple of 32
    const int r = pos / threads;                     // the place's column: see part_len
    const int64_t c = (int64_t(r >> 3) * threads + pos % threads) * kGroup + (r & 7);
    float a = 0.f;
    if (c < H)
        for (int p = q; p < P; p += 16) a += part[int64_t(p) * len + pos];
    s[q][x] = a;
    __syncthreads();
    if (q != 0 || c >= H) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) a += s[k][x];
    if (bf16)
        static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(a);
    else
        static_cast<float*>(out)[c] = a;
}

// The widest row that stays in registers (512 threads of 4 groups).
constexpr int kMaxRegH = 512 * 4 * kGroup;

struct BwdPlan {
    int threads, groups, blocks;   // groups: 0 for the wide kernel
    int64_t len;                   // floats of a partial row
};

// Fixed by H and N alone.  The number of blocks fills the GPU with what the registers
// allow (two accumulators a column) and keeps the partial rows small.
BwdPlan bwd_plan(int64_t N, int64_t H) {
    BwdPlan p;
    if (H <= 1024) p = {32, H <= 256 ? 1 : H <= 512 ? 2 : 4, 608, 0};
    else if (H <= 4096) p = {128, H <= 2048 ? 2 : 4, 608, 0};
    else if (H <= 8192) p = {256, 4, 304, 0};
    else if (H <= kMaxRegH) p = {512, 4, 152, 0};
    else p = {1024, 0, 152, 0};
    const int rows = rows_of(p.threads);
    p.blocks = static_cast<int>(std::min<int64_t>((N + rows - 1) / rows, p.blocks));
    p.len = p.groups > 0 ? int64_t(p.threads) * p.groups * kGroup : part_len(H, p.threads);
    return p;
}

template <typename T, bool CENTER>
cudaError_t fwd_dispatch(const NormArgs& a, cudaStream_t stream) {
    const float inv_h = 1.f / static_cast<float>(a.H);
    const T* x = static_cast<const T*>(a.x);
    T* y = static_cast<T*>(a.out);
#define RLK_NORM_FWD(TH, G)                                                                       \
    norm_fwd_kernel<T, CENTER, TH, G>                                                             \
        <<<(a.N + rows_of(TH) - 1) / rows_of(TH), TH * rows_of(TH), 0, stream>>>(                 \
            x, a.x_stride, a.in_vec, a.weight, a.bias, a.w_bf16, a.w_vec, a.mask, a.N, a.H,       \
            inv_h, a.eps, y, a.out_stride, a.out_vec, a.mean_out, a.rstd_out)
    if (a.H <= 256) RLK_NORM_FWD(32, 1);
    else if (a.H <= 512) RLK_NORM_FWD(32, 2);
    else if (a.H <= 1024) RLK_NORM_FWD(32, 4);
    else if (a.H <= 2048) RLK_NORM_FWD(128, 2);
    else if (a.H <= 4096) RLK_NORM_FWD(128, 4);
    else if (a.H <= 8192) RLK_NORM_FWD(256, 4);
    else if (a.H <= kMaxRegH) RLK_NORM_FWD(512, 4);
    else
        norm_fwd_wide_kernel<T, CENTER><<<a.N, 1024, 0, stream>>>(
            x, a.x_stride, a.in_vec, a.weight, a.bias, a.w_bf16, a.w_vec, a.mask, a.N, a.H, inv_h,
            a.eps, y, a.out_stride, a.out_vec, a.mean_out, a.rstd_out);
#undef RLK_NORM_FWD
    return cudaGetLastError();
}

template <typename T, bool CENTER>
cudaError_t bwd_dispatch(const NormArgs& a, const BwdPlan& p, float* dwp, float* dbp,
                         cudaStream_t stream) {
    const float inv_h = 1.f / static_cast<float>(a.H);
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.out);
#define RLK_NORM_BWD(TH, G)                                                                       \
    norm_bwd_kernel<T, CENTER, TH, G><<<p.blocks, TH * rows_of(TH), 0, stream>>>(                 \
        x, a.x_stride, dy, a.dy_stride, a.in_vec, a.weight, a.w_bf16, a.w_vec, a.mean, a.rstd,    \
        a.mask, a.N, a.H, inv_h, dx, a.out_stride, a.out_vec, dwp, dbp)
    switch (p.threads * 8 + p.groups) {
        case 32 * 8 + 1: RLK_NORM_BWD(32, 1); break;
        case 32 * 8 + 2: RLK_NORM_BWD(32, 2); break;
        case 32 * 8 + 4: RLK_NORM_BWD(32, 4); break;
        case 128 * 8 + 2: RLK_NORM_BWD(128, 2); break;
        case 128 * 8 + 4: RLK_NORM_BWD(128, 4); break;
        case 256 * 8 + 4: RLK_NORM_BWD(256, 4); break;
        case 512 * 8 + 4: RLK_NORM_BWD(512, 4); break;
        default:
            norm_bwd_wide_kernel<T, CENTER><<<p.blocks, 1024, 0, stream>>>(
                x, a.x_stride, dy, a.dy_stride, a.in_vec, a.weight, a.w_bf16, a.w_vec, a.mean,
                a.rstd, a.mask, a.N, a.H, inv_h, dx, a.out_stride, a.out_vec, dwp, dbp);
    }
#undef RLK_NORM_BWD
    return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_workspace(int64_t N, int64_t H, bool center) {
    const BwdPlan p = bwd_plan(N, H);
    return align_up(size_t(p.blocks) * p.len * sizeof(float), 256) * (center ? 2 : 1) + 256;
}

cudaError_t launch_norm_fwd(const NormArgs& a, bool center, cudaStream_t stream) {
    if (a.bf16)
        return center ? fwd_dispatch<__nv_bfloat16, true>(a, stream)
                      : fwd_dispatch<__nv_bfloat16, false>(a, stream);
    return center ? fwd_dispatch<float, true>(a, stream) : fwd_dispatch<float, false>(a, stream);
}

cudaError_t launch_norm_bwd(const NormArgs& a, bool center, cudaStream_t stream) {
    const BwdPlan p = bwd_plan(a.N, a.H);
    const size_t plane = align_up(size_t(p.blocks) * p.len * sizeof(float), 256);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    float* dwp = a.dweight != nullptr ? reinterpret_cast<float*>(ws) : nullptr;
    float* dbp = a.dbias != nullptr ? reinterpret_cast<float*>(ws + plane) : nullptr;
    if (a.N > 0) {
        cudaError_t e;
        if (a.bf16)
            e = center ? bwd_dispatch<__nv_bfloat16, true>(a, p, dwp, dbp, stream)
                       : bwd_dispatch<__nv_bfloat16, false>(a, p, dwp, dbp, stream);
        else
            e = center ? bwd_dispatch<float, true>(a, p, dwp, dbp, stream)
                       : bwd_dispatch<float, false>(a, p, dwp, dbp, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.dweight == nullptr && a.dbias == nullptr) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(p.len / 32), a.dbias != nullptr ? 2 : 1);
    norm_dw_merge_kernel<<<grid, 512, 0, stream>>>(dwp, dbp, p.blocks, static_cast<int>(p.len),
                                                   p.threads, a.H, a.w_bf16, a.dweight, a.dbias);
    return cudaGetLastError();
}

}  // namespace rlk
