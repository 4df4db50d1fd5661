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
// Bound by HBM for many rows, by latency for few.  A block copies a range of columns through the
// mask; it counts the row's tokens that fall into the range in a table in shared memory (16 bits a
// column) while its first loads are on their way.  Where tokens and biases are few (1 to kSparse
// columns, at most), the first to name a column also puts it on a list, and the block reads the
// list's logits while it copies, and changes them behind a barrier: [64, 129280] bf16 with a mask,
// 512 tokens and 64 biases 11.7 us, by a look into the table for each column 13.9.  Where they are
// many that look costs less, and the changed value is taken from the loaded ones: [33, 50021] with
// 20000 tokens 16 us, by the list 31.
//
// Few rows get ranges for all SMs and 1024 threads a block.  Many rows get ranges of kRange columns
// and 256 threads: [1024, 32003] fp32 with 1000 tokens 62 us.  Each block reads all of its row's
// tokens, so a long vocabulary with few tokens takes two launches, the copy and a block for each
// row's listed columns, which counts while the copy ends: [256, 151936] fp32 with 500 tokens 55 us, in
// ranges 60; with 4096 71 and 70; with 15000 121 and 100; [1024, 32003] with 500 61 and 52.  The
// same launch changes rows in place, where nothing else is copied.  It counts up to kFew tokens
// and biases in a hash table of the columns; more in a table of 16 bits a column, part by part of
// the row, where the thread that takes a column's word out of the table changes that column.
// Counting a share of the tokens into the tables of a cluster's blocks was slower, since a text's few
// common tokens all fall into one table.  Counts are whole numbers, so the order of the atomics does
// not matter.  A row with more drawn tokens than 14 bits count gets 32 bits a column.
//
// Measured: [1, 151936] fp32 with 2000 tokens 6.9 us; the 71 above are the copy's 48 and the listed
// columns' 22, whose lines have left L2.
//
// Groups of 16 bytes follow the alignment of the output row.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "ptx.cuh"
#include "rlk_internal.h"

namespace rlk {

namespace {

constexpr int kFew = 4096;               // tokens and biases that the hash table takes
constexpr int kFewWords = 4 * kFew;      // for two slots each
constexpr int kWords = 40960;            // of any other table: a block has an SM to itself
constexpr int kRoom = 16;                // columns of a table in front of a range and behind it
constexpr int kRange = 24576;            // columns of a block where there are many rows
constexpr int kSparse = 32;              // columns for each token and bias, where these are few
constexpr int kMaxNarrow = 0x3fff;       // drawn tokens that 16 bits a column count
constexpr int kUnroll = 4;               // groups a thread has on their way
constexpr int kTokens = 4;               // and tokens
constexpr int kHeld = 2;                 // and listed columns

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& to, float v) { to = v; }
__device__ __forceinline__ void put(__nv_bfloat16& to, float v) { to = __float2bfloat16_rn(v); }

// narrow: two columns a word, 14 bits of count each; wide: one, 30 bits.  Above the count a bit
// for biased columns and one for those among the prompt.
struct Table {
    uint32_t* words;
    bool wide;

    __device__ __forceinline__ int width() const { return wide ? 32 : 16; }
    __device__ __forceinline__ uint32_t* word(int i) const { return words + (wide ? i : i >> 1); }
    __device__ __forceinline__ int shift(int i) const { return wide ? 0 : (i & 1) * 16; }
    // whether nothing had named the column
    __device__ __forceinline__ bool add(int i, bool drawn) const {
        const uint32_t old = drawn ? atomicAdd(word(i), 1u << shift(i))
                                   : atomicOr(word(i), 1u << (shift(i) + width() - 1));
        return (wide ? old : old >> shift(i) & 0xffffu) == 0;
    }
    __device__ __forceinline__ bool mark_biased(int i) const {
        const uint32_t old = atomicOr(word(i), 1u << (shift(i) + width() - 2));
        return (wide ? old : old >> shift(i) & 0xffffu) == 0;
    }
    __device__ __forceinline__ uint32_t get(int i) const {
        return wide ? words[i] : reinterpret_cast<const uint16_t*>(words)[i];
    }
    // bit i: column at + i of VEC is listed; at is a multiple of VEC
    template <int VEC>
    __device__ __forceinline__ uint32_t listed(int at) const {
        uint32_t bits = 0;
        if (wide) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) bits |= words[at + i] != 0 ? 1u << i : 0u;
        } else {
            uint32_t w[VEC / 2];
            if constexpr (VEC == 4)
                *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(words + at / 2);
            else
                *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(words + at / 2);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                bits |= (w[i] & 0xffffu) != 0 ? 1u << 2 * i : 0u;
                bits |= (w[i] >> 16) != 0 ? 2u << 2 * i : 0u;
            }
        }
        return bits;
    }
    // the column's word, which is 0 from then on
    __device__ __forceinline__ uint32_t take(int i) const {
        const uint32_t own = wide ? ~0u : 0xffffu << shift(i);
        if ((*static_cast<volatile uint32_t*>(word(i)) & own) == 0) return 0;
        return (atomicAnd(word(i), ~own) & own) >> shift(i);
    }
};

// The biases by column: open addressing, 2 slots and more for each.  A column that several biases
// name is marked, and gets their sum in ascending slots.
constexpr uint32_t kFree = 0xffffffffu, kTwice = 0x80000000u;
__device__ __forceinline__ uint32_t hashed(uint32_t c) { return c * 0x9e3779b1u >> 8; }
struct Biases {
    uint32_t* key;
    float* value;
    uint32_t mask;                       // of the number of slots, a power of two

    __device__ __forceinline__ Biases(uint32_t* at, int slots)
        : key(at), value(reinterpret_cast<float*>(at + slots)), mask(slots - 1) {}
    __device__ __forceinline__ void insert(uint32_t c, float b) const {
        for (uint32_t h = hashed(c) & mask;; h = (h + 1) & mask) {
            const uint32_t old = atomicCAS(key + h, kFree, c);
            if (old == kFree) {
                value[h] = b;
                return;
            }
            if ((old & ~kTwice) == c) {
                atomicOr(key + h, kTwice);
                return;
            }
        }
    }
    __device__ __forceinline__ float find(uint32_t c) const {
        uint32_t h = hashed(c) & mask;
        while ((key[h] & ~kTwice) != c) h = (h + 1) & mask;
        return value[h];
    }
    // between two barriers; a warp for each marked slot
    template <int THREADS, typename R>
    __device__ __forceinline__ void add_up(int slots, const R& row, int n) const {
        if (n < 2) return;
        const int lane = threadIdx.x & 31;
        for (int h0 = threadIdx.x - lane; h0 < slots; h0 += THREADS) {
            const uint32_t own = h0 + lane < slots ? key[h0 + lane] : kFree;
            uint32_t marked = __ballot_sync(0xffffffffu, own != kFree && (own & kTwice) != 0);
            for (; marked != 0; marked &= marked - 1) {
                const int at = __ffs(marked) - 1;
                const int64_t id = __shfl_sync(0xffffffffu, own, at) & ~kTwice;
                float sum = 0.f;
                for (int i0 = 0; i0 < n; i0 += 32) {
                    const bool in = i0 + lane < n && row.bias_ids[i0 + lane] == id;
                    const float b = in ? row.bias[i0 + lane] : 0.f;
                    for (uint32_t m = __ballot_sync(0xffffffffu, in); m != 0; m &= m - 1)
                        sum += __shfl_sync(0xffffffffu, b, __ffs(m) - 1);
                }
                if (lane == at) value[h0 + lane] = sum;
            }
        }
        __syncthreads();
    }
};

// Columns and their counts by open addressing, at most half of the slots taken.
constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u;
struct Hash {
    uint32_t* key;
    uint32_t* count;
    int slots, shift;                    // slots = 2^(32 - shift)

    // the slots of COUNT columns of each lane (those past V have none), the warp's together: lanes
    // that search by themselves take turns, and 3000 tokens took 12 us instead of 2
    template <int COUNT>
    __device__ __forceinline__ void find(const uint32_t (&c)[COUNT], uint32_t V,
                                         uint32_t (&h)[COUNT]) const {
        uint32_t open = 0;
#pragma unroll
        for (int q = 0; q < COUNT; ++q) {
            h[q] = c[q] * 0x9e3779b1u >> shift;
            open |= c[q] < V ? 1u << q : 0u;
        }
        while (__any_sync(0xffffffffu, open != 0)) {
#pragma unroll
            for (int q = 0; q < COUNT; ++q) {
                uint32_t old = c[q];
                if ((open >> q) & 1u) old = atomicCAS(key + h[q], kFree, c[q]);
                if (old == kFree || old == c[q])
                    open &= ~(1u << q);
                else
                    h[q] = (h[q] + 1) & (slots - 1);
            }
        }
    }
};

// A row's settings and tokens, checked.
struct Row {
    float rep, freq, pres;
    int len, prompt;
    uint32_t bad;                        // error bits
    const int64_t* tokens;
    const int64_t* bias_ids;
    const float* bias;
    const int32_t* allowed;

    __device__ __forceinline__ Row(const ProcessArgs& a, int row) : len(0), prompt(0), bad(0) {
        rep = a.repetition_rows != nullptr ? a.repetition_rows[row] : a.repetition;
        freq = a.frequency_rows != nullptr ? a.frequency_rows[row] : a.frequency;
        pres = a.presence_rows != nullptr ? a.presence_rows[row] : a.presence;
        if (!(rep > 0.f && rep < INFINITY) || !(fabsf(freq) < INFINITY) || !(fabsf(pres) < INFINITY))
            bad = RLK_DEVERR_SAMPLE_PARAM;
        if (a.tokens != nullptr || a.lengths != nullptr || a.prompt_lengths != nullptr) {
            const int64_t n = a.lengths != nullptr ? a.lengths[row] : a.width;
            const int64_t m = a.prompt_lengths != nullptr ? a.prompt_lengths[row] : 0;
            if (m < 0 || n < m || n > a.width)
                bad |= RLK_DEVERR_SAMPLE_PARAM;
            else
                len = static_cast<int>(n), prompt = static_cast<int>(m);
        }
        const int64_t r = row;
        tokens = a.tokens + r * a.tokens_stride;
        bias_ids = a.bias_ids + r * a.bias;
        bias = a.bias_values + r * a.bias;
        allowed = a.allowed != nullptr ? a.allowed + r * a.allowed_stride : nullptr;
    }
    __device__ __forceinline__ bool open(int c) const {
        return allowed == nullptr || ((static_cast<uint32_t>(allowed[c >> 5]) >> (c & 31)) & 1u);
    }
    // a listed column's value: drawn `count` times, among the tokens at all, biased by b
    __device__ __forceinline__ float change(float f, uint32_t count, bool seen, float b) const {
        if (seen) f = f > 0.f ? __fdiv_rn(f, rep) : f * rep;
        if (count != 0) f = fmaf(-freq, static_cast<float>(count), f) - pres;
        return f + b;
    }
};

// The columns [lo, hi) of a row through the mask.  begin() has the first loads on their way.
template <typename T, int THREADS>
struct Copy {
    static constexpr int VEC = 16 / sizeof(T);
    const T* x;
    T* out;
    const int32_t* allowed;
    int V, lo, hi, pad, groups;
    bool vec, in_place;
    uint4 v[kUnroll];

    __device__ __forceinline__ Copy(const ProcessArgs& a, int row, const int32_t* mask)
        : x(static_cast<const T*>(a.x) + row * a.x_stride),
          out(static_cast<T*>(a.out) + row * a.out_stride), allowed(mask), V(a.V) {
        // columns that the first group of 16 aligned bytes of the output lacks in front of the row
        const uintptr_t to = reinterpret_cast<uintptr_t>(out), from = reinterpret_cast<uintptr_t>(x);
        pad = static_cast<int>(to & 15) / int(sizeof(T));
        vec = ((from ^ to) & 15) == 0;
        in_place = from == to;
    }
    __device__ __forceinline__ bool whole(int g) const {
        return lo - pad + g * VEC >= lo && lo - pad + (g + 1) * VEC <= hi;
    }
    // kUnroll groups from g0 on, a thread's
    __device__ __forceinline__ void load(int g0) {
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int g = g0 + q * THREADS;
            if (g >= groups) continue;
            const T* from = x + (lo - pad + g * VEC);
            if (vec && whole(g)) {
                v[q] = __ldcs(reinterpret_cast<const uint4*>(from));
            } else {
                alignas(16) T e[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int c = lo - pad + g * VEC + i;
                    e[i] = c >= lo && c < hi ? from[i] : T(0.f);
                }
                v[q] = *reinterpret_cast<const uint4*>(e);
            }
        }
    }
    // and to the output; LISTED: with what the table and the biases change
    template <bool LISTED>
    __device__ __forceinline__ void store(int g0, const Row& row, const Table& table,
                                          const Biases& biases) {
        uint32_t bits[kUnroll];                  // bit i: column i of the group is open
        uint32_t listed = 0;                     // bit q VEC + i
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int g = g0 + q * THREADS, c = lo - pad + g * VEC;
            bits[q] = ~0u;
            if (g >= groups || allowed == nullptr) continue;
            const int c1 = max(c, 0), c2 = min(c + VEC, V) - 1;
            const uint32_t w1 = static_cast<uint32_t>(allowed[c1 >> 5]);
            const uint32_t w2 = pad != 0 ? static_cast<uint32_t>(allowed[c2 >> 5]) : w1;
            bits[q] = c >= 0 ? __funnelshift_r(w1, w2, c & 31) : w1 << -c;
        }
        constexpr uint32_t kAll = (1u << VEC) - 1;
        if constexpr (LISTED) {
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int g = g0 + q * THREADS;
                if (g < groups)
                    listed |= (table.template listed<VEC>(g * VEC) & bits[q] & kAll) << q * VEC;
            }
        }
        // in place a group that is open in part is read here; others are not needed
        const auto loaded = [&](int q) {
            const int g = g0 + q * THREADS;
            return g < groups && (bits[q] & kAll) != 0 && (bits[q] & kAll) != kAll && whole(g);
        };
        if (in_place && allowed != nullptr) {
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
                if (loaded(q))
                    v[q] = *reinterpret_cast<const uint4*>(x + (lo - pad + (g0 + q * THREADS) * VEC));
        }
#pragma unroll
        for (int q = 0; q < kUnroll; ++q) {
            const int g = g0 + q * THREADS;
            if (g >= groups) continue;
            T* to = out + (lo - pad + g * VEC);
            T* e = reinterpret_cast<T*>(&v[q]);
            if (allowed != nullptr) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (!((bits[q] >> i) & 1u)) put(e[i], -INFINITY);
            }
            const bool all = !in_place || (bits[q] & kAll) == 0 || loaded(q);
            if (all && whole(g)) {
                *reinterpret_cast<uint4*>(to) = v[q];
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int c = lo - pad + g * VEC + i;
                    if (c >= lo && c < hi && (all || !((bits[q] >> i) & 1u))) to[i] = e[i];
                }
            }
        }
        if constexpr (LISTED) {
            for (; listed != 0; listed &= listed - 1) {
                const int b = __ffs(listed) - 1;
                const int at = (g0 + b / VEC * THREADS) * VEC + b % VEC;
                change(at, in_place ? to_f32(out[lo - pad + at]) : value(b), row, table, biases);
            }
        }
    }
    // the column at `at` of the table, whose logit is f
    __device__ __forceinline__ void change(int at, float f, const Row& row, const Table& table,
                                           const Biases& biases) {
        const uint32_t biased = 1u << (table.width() - 2), w = table.get(at);
        const int c = lo - pad + at;
        put(out[c], row.change(f, w & (biased - 1), (w & ~biased) != 0,
                               (w & biased) ? biases.find(c) : 0.f));
    }
    // the loaded value of column b % VEC of group b / VEC, by selection
    __device__ __forceinline__ float value(int b) const {
        const int i = b * int(sizeof(T)) / 4;
        uint32_t w[4 * kUnroll];
#pragma unroll
        for (int q = 0; q < kUnroll; ++q)
            w[4 * q] = v[q].x, w[4 * q + 1] = v[q].y, w[4 * q + 2] = v[q].z, w[4 * q + 3] = v[q].w;
#pragma unroll
        for (int half = 2 * kUnroll; half > 0; half >>= 1)
#pragma unroll
            for (int j = 0; j < half; ++j) w[j] = (i & half) ? w[j + half] : w[j];
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[0]);
        return __uint_as_float((b & 1) ? w[0] & 0xffff0000u : w[0] << 16);
    }
    // begin() has the first loads on their way
    __device__ __forceinline__ void begin(int from, int to) {
        lo = from, hi = to;
        groups = lo < hi ? (hi - lo + pad + VEC - 1) / VEC : 0;
        if (!in_place) load(threadIdx.x);
    }
    template <bool LISTED>
    __device__ __forceinline__ void finish(const Row& row, const Table& table,
                                           const Biases& biases) {
        if (!LISTED && in_place && allowed == nullptr) return;
        for (int g0 = threadIdx.x; g0 < groups; g0 += kUnroll * THREADS) {
            store<LISTED>(g0, row, table, biases);
            if (!in_place && g0 + kUnroll * THREADS < groups) load(g0 + kUnroll * THREADS);
        }
    }
    __device__ __forceinline__ void fill_nan() {
        for (int c = lo + threadIdx.x; c < hi; c += THREADS) put(out[c], __int_as_float(0x7fc00000));
    }
};

// The listed columns of [lo, hi), by a table that has room for them, column lo at `pad`.
template <typename T, int THREADS>
struct Listed {
    const Row& row;
    Table table;
    Biases biases;
    int slots, V, num_biases, pad, lo, hi;
    uint32_t* list;                      // which columns have been named, by their places in the
    uint32_t* listed;                    // table, and how many

    // and for what a group reads past the last column
    __device__ __forceinline__ void clear() {
        const int room = hi - lo + pad + 7, words = table.wide ? room : (room + 1) / 2;
        for (int i = threadIdx.x; i < (words + 3) / 4; i += THREADS)
            reinterpret_cast<uint4*>(table.words)[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < slots; i += THREADS) biases.key[i] = kFree;
        if (listed != nullptr && threadIdx.x == 0) *listed = 0;
    }
    // counts the tokens and enters the biases; the thread's error bits.  LIST: with a list
    template <bool LIST>
    __device__ __forceinline__ uint32_t count() {
        uint32_t bad = 0;
        for (int i0 = threadIdx.x; i0 < row.len; i0 += 2 * kTokens * THREADS) {
            int64_t id[2 * kTokens];
#pragma unroll
            for (int q = 0; q < 2 * kTokens; ++q)
                id[q] = i0 + q * THREADS < row.len ? __ldg(row.tokens + i0 + q * THREADS) : -1;
#pragma unroll
            for (int q = 0; q < 2 * kTokens; ++q) {
                if (id[q] >= V) bad |= RLK_DEVERR_TARGET_RANGE;
                if (id[q] >= lo && id[q] < hi) {
                    const int at = static_cast<int>(id[q]) - lo + pad;
                    const bool first = table.add(at, i0 + q * THREADS >= row.prompt);
                    if (LIST && first) list[atomicAdd(listed, 1u)] = at;
                }
            }
        }
        for (int i = threadIdx.x; i < num_biases; i += THREADS) {
            const int64_t id = row.bias_ids[i];
            if (id >= V) bad |= RLK_DEVERR_TARGET_RANGE;
            if (id < lo || id >= hi) continue;
            const bool first = table.mark_biased(static_cast<int>(id) - lo + pad);
            if (LIST && first)
                list[atomicAdd(listed, 1u)] = static_cast<int>(id) - lo + pad;
            biases.insert(static_cast<uint32_t>(id), row.bias[i]);
        }
        return bad;
    }
    // after a barrier; pad = 0
    __device__ __forceinline__ void change(T* out) {
        biases.template add_up<THREADS>(slots, row, num_biases);
        visit(out, row.tokens, row.len);
        visit(out, row.bias_ids, num_biases);
    }
    __device__ __forceinline__ void visit(T* out, const int64_t* list, int n) {
        const uint32_t biased = 1u << (table.width() - 2), counted = biased - 1;
        for (int i0 = threadIdx.x; i0 < n; i0 += kTokens * THREADS) {
            int at[kTokens];
            uint32_t word[kTokens];
            float f[kTokens];
#pragma unroll
            for (int q = 0; q < kTokens; ++q) {
                const int i = i0 + q * THREADS;
                const int64_t id = i < n ? __ldg(list + i) : -1;
                at[q] = id >= lo && id < hi ? static_cast<int>(id) - lo : -1;
            }
#pragma unroll
            for (int q = 0; q < kTokens; ++q) {
                word[q] = at[q] >= 0 ? table.take(at[q]) : 0;
                if (word[q] != 0 && !row.open(lo + at[q])) word[q] = 0;
                if (word[q] != 0) f[q] = to_f32(out[lo + at[q]]);
            }
#pragma unroll
            for (int q = 0; q < kTokens; ++q) {
                if (word[q] == 0) continue;
                const int c = lo + at[q];
                put(out[c], row.change(f[q], word[q] & counted, (word[q] & ~biased) != 0,
                                       (word[q] & biased) ? biases.find(c) : 0.f));
            }
        }
    }
};

// A block copies a range of a row, LISTED: with its listed columns changed.  share: columns of a
// block, a multiple of 32; words: of its table; few_most: tokens and biases with which it lists them.
template <typename T, int THREADS, bool LISTED>
__global__ void __launch_bounds__(THREADS, THREADS == 1024 ? 1 : LISTED ? 4 : 6)
    process_kernel(const ProcessArgs args, int ranges, int share, int bias_slots, int words,
                   int few_most) {
    extern __shared__ uint4 smem[];              // the table, the biases, the list
    __shared__ uint32_t s_listed;
    ProcessArgs a = args;
    const int r = blockIdx.x / ranges, range = blockIdx.x % ranges;
    wait_previous(a.x, a.mask, a.tokens, a.lengths, a.prompt_lengths, a.repetition_rows,
                  a.frequency_rows, a.presence_rows, a.bias_ids, a.bias_values, a.allowed);
    // the launch that changes the listed columns may start: what it reads before it waits itself,
    // the call's inputs, is there
    if (!LISTED) asm volatile("griddepcontrol.launch_dependents;");
    if (a.mask != nullptr && a.mask[r] == 0) return;
    const Row row(a, r);
    Copy<T, THREADS> copy(a, r, row.allowed);
    const int first = range * share, end = min(a.V, first + share);
    uint32_t* own = reinterpret_cast<uint32_t*>(smem);
    const Table table{own, row.len - row.prompt > kMaxNarrow};
    const Biases biases(own + words, bias_slots);
    if constexpr (!LISTED) {
        copy.begin(first, end);
        if (row.bad == 0) {
            copy.template finish<false>(row, table, biases);
        } else {
            if (range == 0 && threadIdx.x == 0 && a.err != nullptr) atomicOr(a.err, row.bad);
            copy.fill_nan();
        }
    } else {
        uint32_t* list = own + words + 2 * bias_slots;
        Listed<T, THREADS> listed{row, table, biases, bias_slots, a.V, a.bias, copy.pad, 0, 0,
                                  list, &s_listed};
        const bool few = row.len + a.bias <= few_most;
        const int part = ((table.wide ? words : 2 * words) - kRoom) / 32 * 32;
        for (int lo = first; lo < end; lo += part) {
            listed.lo = lo, listed.hi = min(end, lo + part);
            copy.begin(lo, listed.hi);
            listed.clear();
            __syncthreads();
            const uint32_t bad = row.bad | (few ? listed.template count<true>()
                                                : listed.template count<false>());
            if (__syncthreads_or(bad != 0)) {
                if (bad != 0 && range == 0 && a.err != nullptr) atomicOr(a.err, bad);
                copy.fill_nan();
            } else {
                biases.template add_up<THREADS>(bias_slots, row, a.bias);
                if (few) {
                    const int n = static_cast<int>(s_listed);
                    // a thread's first kHeld are read while the row is copied
                    int at[kHeld];
                    float f[kHeld];
#pragma unroll
                    for (int q = 0; q < kHeld; ++q) {
                        const int i = threadIdx.x + q * THREADS;
                        at[q] = i < n ? list[i] : -1;
                        if (at[q] >= 0 && !row.open(lo - copy.pad + at[q])) at[q] = -1;
                        if (at[q] >= 0) f[q] = to_f32(copy.x[lo - copy.pad + at[q]]);
                    }
                    copy.template finish<false>(row, table, biases);
                    __syncthreads();
#pragma unroll
                    for (int q = 0; q < kHeld; ++q)
                        if (at[q] >= 0) copy.change(at[q], f[q], row, table, biases);
                    for (int i = threadIdx.x + kHeld * THREADS; i < n; i += THREADS) {
                        const int at = list[i], c = lo - copy.pad + at;
                        if (row.open(c)) copy.change(at, to_f32(copy.x[c]), row, table, biases);
                    }
                } else {
                    copy.template finish<true>(row, table, biases);
                }
            }
            __syncthreads();
        }
    }
}

// The listed columns of a row in the output, by a block for each range of them.  Rows of up to kFew
// tokens and biases: by the first block alone.  WORDS: of shared memory for the table.  copied: a
// copy runs before.
template <typename T, int THREADS, int WORDS>
__global__ void __launch_bounds__(THREADS, THREADS == 1024 ? 1 : 2)
    process_listed_kernel(const ProcessArgs args, int ranges, int share, int bias_slots,
                          bool copied) {
    extern __shared__ uint4 smem[];
    const int r = blockIdx.x / ranges, range = blockIdx.x % ranges, tid = threadIdx.x;
    ProcessArgs a = args;
    const auto wait = [] { asm volatile("griddepcontrol.wait;" ::: "memory"); };
    if (!copied)
        wait_previous(a.mask, a.tokens, a.lengths, a.prompt_lengths, a.repetition_rows,
                      a.frequency_rows, a.presence_rows, a.bias_ids, a.bias_values, a.allowed);
    const Row row(a, r);
    const bool few = WORDS == kFewWords || row.len + a.bias <= kFew;
    if ((a.mask != nullptr && a.mask[r] == 0) || (few && range > 0)) {
        if (copied) wait();              // a launch that waits for this one waits for the copy too
        return;
    }
    T* out = static_cast<T*>(a.out) + r * a.out_stride;
    uint32_t* words = reinterpret_cast<uint32_t*>(smem);
    const Biases biases(words + WORDS, bias_slots);
    uint32_t bad = row.bad;
    bool broken;
    int lo = range * share;
    const int end = min(a.V, lo + share);
    if (few) {
        Hash hash{words, nullptr, 1024, 22};
        while (hash.slots < 2 * (row.len + a.bias)) hash.slots *= 2, --hash.shift;
        hash.count = hash.key + hash.slots;
        for (int i = tid; i < hash.slots; i += THREADS) hash.key[i] = kFree, hash.count[i] = 0;
        for (int i = tid; i < bias_slots; i += THREADS) biases.key[i] = kFree;
        __syncthreads();
        constexpr uint32_t kNone = 0xfffffffeu;
        const uint32_t V = static_cast<uint32_t>(a.V);
        const int lane = tid & 31;
        for (int i0 = tid; i0 - lane < row.len; i0 += kTokens * THREADS) {
            uint32_t c[kTokens], h[kTokens];
#pragma unroll
            for (int q = 0; q < kTokens; ++q) {
                const int i = i0 + q * THREADS;
                const int64_t id = i < row.len ? __ldg(row.tokens + i) : -1;
                if (id >= a.V) bad |= RLK_DEVERR_TARGET_RANGE;
                c[q] = id >= 0 && id < a.V ? static_cast<uint32_t>(id) : kNone;
            }
            hash.find(c, V, h);
#pragma unroll
            for (int q = 0; q < kTokens; ++q) {
                if (c[q] == kNone) continue;
                if (i0 + q * THREADS >= row.prompt)
                    atomicAdd(hash.count + h[q], 1u);
                else
                    atomicOr(hash.count + h[q], kPrompt);
            }
        }
        for (int i = tid; i - lane < a.bias; i += THREADS) {
            const int64_t id = i < a.bias ? row.bias_ids[i] : -1;
            if (id >= a.V) bad |= RLK_DEVERR_TARGET_RANGE;
            const uint32_t c[1] = {id >= 0 && id < a.V ? static_cast<uint32_t>(id) : kNone};
            uint32_t h[1];
            hash.find(c, V, h);
            if (c[0] == kNone) continue;
            atomicOr(hash.count + h[0], kBiased);
            biases.insert(c[0], row.bias[i]);
        }
        broken = __syncthreads_or(bad != 0) != 0;
        if (!broken) biases.add_up<THREADS>(bias_slots, row, a.bias);
        if (copied) wait();
        constexpr int kEach = 2 * kTokens;
        for (int i0 = tid; i0 < hash.slots && !broken; i0 += kEach * THREADS) {
            uint32_t key[kEach];
            float f[kEach];
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                const int i = i0 + q * THREADS;
                key[q] = i < hash.slots ? hash.key[i] : kFree;
                if (key[q] != kFree && !row.open(static_cast<int>(key[q]))) key[q] = kFree;
                if (key[q] != kFree) f[q] = to_f32(out[key[q]]);
            }
#pragma unroll
            for (int q = 0; q < kEach; ++q) {
                if (key[q] == kFree) continue;
                const uint32_t w = hash.count[i0 + q * THREADS];
                put(out[key[q]], row.change(f[q], w & (kBiased - 1), (w & ~kBiased) != 0,
                                            (w & kBiased) ? biases.find(key[q]) : 0.f));
            }
        }
    } else {
        Listed<T, THREADS> listed{row, Table{words, row.len - row.prompt > kMaxNarrow}, biases,
                                  bias_slots, a.V, a.bias, 0, 0, 0, nullptr, nullptr};
        const int part = ((listed.table.wide ? WORDS : 2 * WORDS) - kRoom) / 32 * 32;
        bool waited = !copied;
        for (; lo < end; lo += part) {
            listed.lo = lo, listed.hi = min(end, lo + part);
            listed.clear();
            __syncthreads();
            bad |= listed.template count<false>();
            broken = __syncthreads_or(bad != 0) != 0;
            if (!waited) wait();
            waited = true;
            if (broken) break;
            listed.change(out);
            __syncthreads();
        }
        if (!waited) wait();
        broken = __syncthreads_or(bad != 0) != 0;
    }
    if (broken) {
        if (bad != 0 && range == 0 && a.err != nullptr) atomicOr(a.err, bad);
        for (int c = range * share + tid; c < (few ? a.V : end); c += THREADS)
            put(out[c], __int_as_float(0x7fc00000));
    }
}

// Ranges of about `columns` each, and the columns of one.
struct Ranges {
    int count, share;
    Ranges(int V, int columns) {
        count = (V + columns - 1) / columns;
        share = ((V + count - 1) / count + 31) / 32 * 32;
    }
};

constexpr int kStaticShared = 256;               // more than what is static in any kernel
constexpr int kMostShared = 227 * 1024 - kStaticShared;
static_assert(kWords * 4 + 2 * kMaxBias * 8 <= kMostShared, "a block's shared memory");
int bias_slots(const ProcessArgs& a) {
    if (a.bias == 0) return 0;
    int slots = 2;
    while (slots < 2 * a.bias) slots *= 2;
    return slots;
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(const ProcessArgs, int, int, int, Params...), int threads,
                   const ProcessArgs& a, const Ranges& r, size_t words, size_t list, cudaStream_t stream,
                   Args... args) {
    const int64_t blocks = static_cast<int64_t>(a.N) * r.count;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const size_t smem =
        words * 4 + static_cast<size_t>(words > 0 ? bias_slots(a) : 0) * 8 + list * 4;
    // without the attribute a block has 48 KB, of which what is static takes its part
    if (smem > 48 * 1024 - kStaticShared) {
        const cudaError_t e = cudaFuncSetAttribute(
            reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
            kMostShared);
        if (e != cudaSuccess) return e;
    }
    return launch_early(kernel, dim3(static_cast<unsigned>(blocks)), threads, smem, stream, nullptr,
                        a, r.count, r.share, bias_slots(a), args...);
}

// Columns that a table of kWords has room for.
constexpr int kMostColumns = (2 * kWords - kRoom) / 32 * 32;

// few_most: tokens and biases with which a row's listed columns are listed; the list has room for
// them, or for all of the range's columns.
template <typename T, int THREADS>
cudaError_t launch_listed(const ProcessArgs& a, const Ranges& r, cudaStream_t stream) {
    // a table of 32 bits takes 32 columns at least, all of them where a block has the SM to itself
    const int narrow = std::max(48, (r.share + kRoom + 31) / 32 * 16);
    const int words = THREADS == 1024 && a.width > kMaxNarrow
                          ? std::max(narrow, std::min(kWords, r.share + kRoom)) : narrow;
    const int room = std::min(THREADS == 1024 ? 4096 : 1024,
                              (kMostShared - words * 4 - bias_slots(a) * 8) / 4);
    const int list = std::min(std::min(a.V / kSparse, r.share), room);
    const int few_most = list == room ? room : a.V / kSparse;
    return launch(process_kernel<T, THREADS, true>, THREADS, a, r, words, list, stream, words, few_most);
}

template <typename T>
cudaError_t launch_rows(const ProcessArgs& a, cudaStream_t stream) {
    const bool listed = a.tokens != nullptr || a.bias > 0;
    if (listed) {
        // as many ranges as give each of 152 SMs one, of 4096 columns at least and the table's size
        // at most
        const int ranges = std::max((a.V + kMostColumns - 1) / kMostColumns,
                                    std::min(152 / a.N, (a.V + 4095) / 4096));
        const Ranges r(a.V, (a.V + ranges - 1) / ranges);
        if (static_cast<int64_t>(a.N) * r.count <= 152)
            return launch_listed<T, 1024>(a, r, stream);
    }
    // ranges, and blocks for all of 152 SMs four times
    if (listed && a.x != a.out &&
        (a.V <= 2 * kRange || kSparse * (int64_t(a.width) + a.bias) >= a.V)) {
        const int ranges = std::max((a.V + kRange - 1) / kRange,
                                    std::min(608 / a.N, (a.V + 4095) / 4096));
        const Ranges r(a.V, (a.V + ranges - 1) / ranges);
        return launch_listed<T, 256>(a, r, stream);
    }
    // a row that cannot be is found out even where nothing is changed
    const bool checked = a.repetition_rows != nullptr || a.frequency_rows != nullptr ||
                         a.presence_rows != nullptr || a.lengths != nullptr ||
                         a.prompt_lengths != nullptr;
    const bool copied = a.x != a.out || a.allowed != nullptr;
    if (copied || (!listed && checked)) {
        const cudaError_t e =
            launch(process_kernel<T, 256, false>, 256, a, Ranges(a.V, 8192), 0, 0, stream, 0, 0);
        if (e != cudaSuccess) return e;
    }
    if (!listed) return cudaSuccess;
    if (a.width + a.bias <= kFew)
        return launch(process_listed_kernel<T, 512, kFewWords>, 512, a, Ranges(a.V, a.V), kFewWords, 0,
                      stream, copied);
    // a block a row where that is enough of them
    const Ranges r(a.V, a.N > 152 ? a.V : kMostColumns);
    return launch(process_listed_kernel<T, 1024, kWords>, 1024, a, r, kWords, 0, stream, copied);
}

}  // namespace

cudaError_t launch_process(const ProcessArgs& a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_rows<__nv_bfloat16>(a, stream) : launch_rows<float>(a, stream);
}

}  // namespace rlk
