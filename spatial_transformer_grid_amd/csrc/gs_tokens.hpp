// gs_tokens.hpp -- shared parts of the token operators (layer norm, dropout,
// attention): launch parameters, the counter-based generator, 8-element
// fragments of the matrix cores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gs {

constexpr int kMaxBuckets = 512;     // buckets of a bias table
constexpr int kMaxBorder = 1024;     // largest first distance of a last bucket
constexpr float kMaxFold = 32768.0f; // largest factor of a probability (fp16 ends at 65504)

struct NormParams {
    const void *X, *dY, *scale, *bias;
    void *Y, *dX;
    float *mean, *inv_std;
    int64_t rows;
    int cols;
    int64_t x_stride, y_stride, dy_stride, dx_stride;
    float epsilon;
    int param_f32;            // scale and bias are fp32 (else the data type)
    int vec;                  // rows allow 16-byte accesses
    void *dscale, *dbias;
    float *partial;           // backward: (parts, 2, cols) sums
    int parts;
};

struct DropoutParams {
    const void *X, *residual;
    void *Y;
    int64_t count;
    uint32_t threshold, seed_lo, seed_hi, call;
    float keep_scale;
    int vec;
};

struct AttnParams {
    const void *q, *k, *v, *o_in, *d_o, *table;
    void *o, *dq, *dk, *dv, *dtable;
    float *lse;
    const int32_t *lengths;
    float *rows;              // backward: what the dK / dV kernel takes of the queries (row_stats)
    float *part;              // backward: (H, B, key tiles, parts, buckets) sums of dS
    float *split;             // sums of the parts of a split axis (see each kernel)
    int64_t qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];
    int B, H, Hkv, G, Lq, Lk, D;
    int causal, from_end, first;
    float scale, scale2;      // scale2 = scale * log2(e)
    int buckets, side, border, bidirectional, table_f32;
    int lut;                  // entries of the distance table (0: no bias)
    uint32_t threshold, seed_lo, seed_hi, call;
    float keep_scale;
    float fold, fold_log2;    // backward: the factor of keep_scale that P carries
    float rest;               // keep_scale / fold
    int vec;                  // rows of every tensor allow 16-byte accesses
    int async;                // and their tiles asynchronous loads
    int tiles;                // row tiles of a unit (a head of a sequence)
    int units;
    int pack;                 // forward, few queries: rows are the queries of all heads of a key head
    int splits, chunk;        // parts of the split axis; keys of a part
    int nblocks;
    uint16_t starts[kMaxBuckets];  // first distance of each bucket of one side
};

// How an attention call is laid out on the chip.
struct AttnPlan {
    int ways;                 // parts of the other axis that a block's waves take: 128 / ways rows a block
    int pack, splits, chunk, tiles, units;
    int64_t split_floats;     // of workspace
};
AttnPlan plan_forward(const AttnParams &p, int dtype, bool workspace);
AttnPlan plan_backward_q(const AttnParams &p, int dtype);
AttnPlan plan_backward_kv(const AttnParams &p, int dtype);

// Launchers; 0 or the hipError_t of the launch.  `dtype` 0 f32, 1 f16, 2 bf16.
int launch_layer_norm(const NormParams &p, int dtype, hipStream_t stream);
int launch_layer_norm_backward(const NormParams &p, int dtype, hipStream_t stream);
int layer_norm_parts(int64_t rows, int64_t cols);
int launch_dropout(const DropoutParams &p, int dtype, hipStream_t stream);
int launch_attention(const AttnParams &p, int dtype, hipStream_t stream);
int launch_attention_backward(const AttnParams &p, int dtype, hipStream_t stream);

constexpr int kAttnRows = 128;       // rows of a block: four waves of 32
constexpr int kMaxLds = 163840;      // bytes of LDS of a compute unit

// Entries of the distance table: the relative positions between the changes of
// bucket, and kLutPad past either end.
constexpr int kLutPad = 96;

__host__ __device__ inline int lut_entries(int border, int bidirectional) {
    return (bidirectional ? 2 * border : border) + 1 + 2 * kLutPad;
}

inline int padded_dim(int D) { return (D + 31) / 32 * 32; }
__host__ __device__ inline int split_row(int D) { return (D + 3) / 4 * 4; }   // floats of a row of partial sums

}  // namespace gs

#if defined(__HIPCC__)
#include "gs_device.hpp"

namespace gs {

typedef __attribute__((ext_vector_type(4))) float tokens_f32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16v8 __attribute__((ext_vector_type(8)));
typedef short s16v4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMaxFloat = 3.402823466e38f;
// Largest bias (base 2) that fp32 scores carry as it is: there a product beside it
// is still held to 2^-12.
constexpr float kBiasKept = 4096.0f;

// fp32 -> the raw bits of T, to nearest even
template <typename T>
__device__ __forceinline__ typename T::raw_t to_bits(float v) {
    if constexpr (T::bytes == 4) return __builtin_bit_cast(uint32_t, v);
    else if constexpr (__is_same(T, BF16)) return __builtin_bit_cast(uint16_t, (__bf16)settle(v));
    else return __builtin_bit_cast(uint16_t, (_Float16)settle(v));
}

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011): ten rounds of two 32 x 32
// -> 64-bit products, whose key words are the same for every lane, each
// followed by one three-way exclusive or.  One call serves eight elements.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                        uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = __builtin_amdgcn_bitop3_b32((uint32_t)(b >> 32), c1, k0, 0x96);
        c2 = __builtin_amdgcn_bitop3_b32((uint32_t)(a >> 32), c3, k1, 0x96);
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// 1 in each 16-bit half of a generator word that keeps its element, else 0;
// `below` holds threshold - 1 (threshold > 0) in both halves.
__device__ __forceinline__ uint32_t kept_pair(uint32_t w, uint32_t below) {
    uint32_t d;
    __asm__("v_pk_sub_u16 %0, %1, %2 clamp\n\tv_pk_min_u16 %0, %0, 1 op_sel_hi:[1,0]" : "=v"(d) : "v"(w), "s"(below));
    return d;
}

// One bit for each of a call's eight elements, 1 where it is kept.
__device__ __forceinline__ uint32_t kept_byte(const u32x4 &r, uint32_t below) {
    const uint32_t x = kept_pair(r[0], below) | kept_pair(r[1], below) << 2 | kept_pair(r[2], below) << 4 |
                       kept_pair(r[3], below) << 6;
    return x | x >> 15;
}

// Number e (0..7) of a call: low half of the first word first.
__device__ __forceinline__ bool kept(const u32x4 &r, int e, uint32_t threshold) {
    const uint32_t w = r[e >> 1];
    return ((e & 1) ? w >> 16 : w & 0xffffu) >= threshold;
}

// Eight consecutive elements of T along the contracted axis: what a lane
// feeds the 32 x 32 matrix instructions for 16 steps of that axis (lanes 0-31
// the first eight, lanes 32-63 the last eight).
template <typename T>
struct Frag {
    u32x4 w[T::bytes / 2];
};

template <typename T>
__device__ __forceinline__ float frag_get(const Frag<T> &f, int j) {
    if constexpr (T::bytes == 4) return __builtin_bit_cast(float, (uint32_t)f.w[j >> 2][j & 3]);
    else return T::from_raw((uint16_t)(f.w[0][j >> 1] >> (16 * (j & 1))));
}

template <typename T>
__device__ __forceinline__ Frag<T> frag_pack(const float *v) {
    Frag<T> f;
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f.w[j >> 2][j & 3] = __builtin_bit_cast(uint32_t, v[j]);
    } else if constexpr (__is_same(T, BF16)) {
        bf16v8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (__bf16)v[j];
        f.w[0] = __builtin_bit_cast(u32x4, x);
    } else {
        f16v8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (_Float16)v[j];
        f.w[0] = __builtin_bit_cast(u32x4, x);
    }
    return f;
}

template <typename T>
__device__ __forceinline__ void frag_negate(Frag<T> &f) {
#pragma unroll
    for (int n = 0; n < T::bytes / 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) f.w[n][i] ^= T::bytes == 4 ? 0x80000000u : 0x80008000u;
}

// Zeros where the generator drops an element (16-bit types): each half of a
// word times 1 or 0, as integers.  (As asm: the compiler would take the words
// apart into selected halves and put them together again.)
template <typename T>
__device__ __forceinline__ void frag_keep(Frag<T> &f, const u32x4 &kept) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w = f.w[0][i];
        __asm__("v_pk_mul_lo_u16 %0, %0, %1" : "+v"(w) : "v"(kept[i]));
        f.w[0][i] = w;
    }
}

// Byte n of a word as a float.
template <int N>
__device__ __forceinline__ float byte_float(uint32_t w) {
    float f;
    if constexpr (N == 0) __asm__("v_cvt_f32_ubyte0_e32 %0, %1" : "=v"(f) : "v"(w));
    else if constexpr (N == 1) __asm__("v_cvt_f32_ubyte1_e32 %0, %1" : "=v"(f) : "v"(w));
    else if constexpr (N == 2) __asm__("v_cvt_f32_ubyte2_e32 %0, %1" : "=v"(f) : "v"(w));
    else __asm__("v_cvt_f32_ubyte3_e32 %0, %1" : "=v"(f) : "v"(w));
    return f;
}

// The value of lane ^ 32.
__device__ __forceinline__ float other_half(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                    false, false);
    return __builtin_bit_cast(float, (uint32_t)((threadIdx.x & 32) ? r[0] : r[1]));
}

// Keeps a branch that few tiles take a branch: what it does to the N values is
// not computed beforehand and selected.
template <int N>
__device__ __forceinline__ void rare(float *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) __asm__ volatile("" : "+v"(v[i]));
}

// acc (32 x 32) += A (32 x 16) B (16 x 32).  Lane l holds row l % 32 of A and
// column l % 32 of B, steps 8 (l / 32) .. + 7; it holds column l % 32 of acc
// and its rows 8 (r / 4) + 4 (l / 32) + r % 4.  fp32 runs eight products of
// two steps each: both operands name the steps in the same order.
template <typename T>
__device__ __forceinline__ void mma(f32x16 &acc, const Frag<T> &a, const Frag<T> &b) {
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(frag_get<T>(a, j), frag_get<T>(b, j), acc, 0,
                                                       0, 0);
    } else if constexpr (__is_same(T, BF16)) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16v8, a.w[0]),
                                                      __builtin_bit_cast(bf16v8, b.w[0]), acc, 0, 0, 0);
    } else {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16v8, a.w[0]),
                                                     __builtin_bit_cast(f16v8, b.w[0]), acc, 0, 0, 0);
    }
}

// Row of a 32-row tile that row m of the A operand carries, chosen so that a
// lane's results r = 8 t + j are rows 16 t + 8 (lane / 32) + j of the tile:
// eight consecutive ones, which is the order in which the next product's B
// operand wants them.  The results feed it without leaving the registers, and
// one generator call covers them.
__device__ __forceinline__ int a_row(int m) {
    return 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
}

// An LDS tile: rows of DP elements without gaps (an asynchronous load writes a
// wave's 16-byte chunks one after another), whose chunks change places by row
// so that neither of two reads meets a bank twice.  The 64 banks of four bytes
// serve sixteen lanes of a 16-byte read at once, which lie in one chunk column
// of sixteen rows (a_row), and 32 lanes of a transposing read, which cover
// four chunks, an aligned group, of rows r .. r + 3, r a multiple of four.
template <typename T, int DP>
struct Tile {
    static constexpr int EPC = 16 / T::bytes;       // elements of a chunk
    static constexpr int CPR = DP / EPC;            // chunks of a row
    __device__ __forceinline__ static int turn(int row) {
        if constexpr (T::bytes == 4) return CPR % 16 == 0 ? row & 15 : row >> 1 & 7;
        const int low = row >> 2 & 3;
        if constexpr (DP == 128) return (row & 3) << 2 | low;
        if constexpr (DP == 64) return (row & 2) << 1 | low;
        return low;
    }
    // element offset of the chunk that holds column col
    __device__ __forceinline__ static int chunk(int row, int col) {
        return row * DP + ((col / EPC) ^ turn(row)) * EPC;
    }
};

__device__ __forceinline__ void async_wait() { __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Rows row0 .. row0 + ROWS - 1 of a strided tensor into an LDS tile, in 16-byte
// chunks over the NT threads that share it, zeros outside rows < limit (FROM:
// and from <= row) and columns < D.  `async`: by loads that write LDS by themselves (async_wait,
// then tile_sync, before the tile is read), which leaves the registers to the
// products.  A lane's chunk lands at its own place of the tile, so it is the
// source column that changes place; reads outside the range of the descriptor
// give zeros, and ROWS rows span less than 2 GiB.  Otherwise through registers.
template <typename T, int DP, int ROWS, int NT, bool FROM = false>
__device__ __forceinline__ void copy_tile(typename T::raw_t *lds, const typename T::raw_t *base, int64_t stride,
                                          int row0, int limit, int D, bool async, bool vec, int t, int from = 0) {
    typedef typename T::raw_t raw_t;
    typedef Tile<T, DP> L;
    constexpr int EPC = L::EPC, CPR = L::CPR, N = (ROWS * CPR + NT - 1) / NT;
    static_assert(ROWS * CPR % 64 == 0, "a wave has a whole step or none");
    if (async) {
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            (void *)(base + (int64_t)row0 * stride), 0, 0x7fffffff, 0x00027000);
        const uint32_t rows = max(limit - from, 0);  // in one comparison, by wrapping
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = t + n * NT, r = c / CPR, col = ((c - r * CPR) ^ L::turn(r)) * EPC;
            const bool in = FROM ? (uint32_t)(r + (row0 - from)) < rows : row0 + r < limit;
            const uint32_t at = in && col < D ? (uint32_t)(r * (int)stride + col) * T::bytes : 0x80000000u;
            if (ROWS * CPR % NT == 0 || c < ROWS * CPR)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rsrc, (__attribute__((address_space(3))) void *)(lds + ((t & ~63) + n * NT) * EPC), 16, (int)at, 0,
                    0, 0);
        }
        return;
    }
#pragma unroll 1
    for (int c = t; c < ROWS * CPR; c += NT) {
        const int r = c / CPR, col = (c - r * CPR) * EPC;
        u32x4 v = {0, 0, 0, 0};
        if ((!FROM || row0 + r >= from) && row0 + r < limit && col < D) {
            const raw_t *src = base + (int64_t)(row0 + r) * stride + col;
            if (vec) {
                v = *(const u32x4 *)src;
            } else {
                raw_t e[EPC];
#pragma unroll
                for (int j = 0; j < EPC; ++j) e[j] = col + j < D ? src[j] : raw_t(0);
                __builtin_memcpy(&v, e, 16);
            }
        }
        *(u32x4 *)(lds + L::chunk(r, col)) = v;
    }
}

// Eight elements from column col of a global row (zeros at and past D).
template <typename T>
__device__ __forceinline__ Frag<T> frag_global(const typename T::raw_t *row, int col, int D, bool ok,
                                               bool vec) {
    typedef typename T::raw_t raw_t;
    constexpr int EPC = 16 / T::bytes;
    Frag<T> f;
#pragma unroll
    for (int n = 0; n < T::bytes / 2; ++n) {
        u32x4 v = {0, 0, 0, 0};
        const int c = col + n * EPC;
        if (ok && c < D) {
            if (vec) {
                v = *(const u32x4 *)(row + c);
            } else {
                raw_t e[EPC];
#pragma unroll
                for (int j = 0; j < EPC; ++j) e[j] = c + j < D ? row[c + j] : raw_t(0);
                __builtin_memcpy(&v, e, 16);
            }
        }
        f.w[n] = v;
    }
    return f;
}

// Eight elements of an LDS tile from column col (a multiple of 8) of a row.
template <typename T, int DP>
__device__ __forceinline__ Frag<T> frag_lds(const typename T::raw_t *lds, int row, int col) {
    Frag<T> f;
#pragma unroll
    for (int n = 0; n < T::bytes / 2; ++n)
        f.w[n] = *(const u32x4 *)(lds + Tile<T, DP>::chunk(row, col + n * Tile<T, DP>::EPC));
    return f;
}

// A operand of a transposed tile: lane l gets column col0 + l % 32 of LDS
// rows row0 + 8 (l / 32) .. + 7.  16-bit elements go through the transposing
// LDS read: sixteen lanes name four rows of sixteen columns, four elements
// each, and each gets one column of the four rows.  A lane reads four-byte
// elements on their own.
template <typename T, int DP>
__device__ __forceinline__ Frag<T> frag_lds_transposed(const typename T::raw_t *lds, int row0, int col0,
                                                       int lane) {
    Frag<T> f;
    if constexpr (T::bytes == 4) {
        const int col = col0 + (lane & 31);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f.w[j >> 2][j & 3] = lds[Tile<T, DP>::chunk(row0 + 8 * (lane >> 5) + j, col) + (col & 3)];
    } else {
        typedef __attribute__((address_space(3))) s16v4 *lds_s16v4;
        const int row = row0 + 8 * (lane >> 5) + (lane >> 2 & 3), col = col0 + (lane & 16) + 4 * (lane & 3);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const typename T::raw_t *p = lds + Tile<T, DP>::chunk(row + 4 * n, col) + (col & 4);
            const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16v4)p));
            f.w[0][2 * n] = v[0];
            f.w[0][2 * n + 1] = v[1];
        }
    }
    return f;
}

// N products whose A operands are read from LDS, GROUP at a time: a group is
// read while the one before is multiplied.  Left alone the compiler reads each
// operand right before its product and waits for it, and a wave stands still
// for the latency of LDS each time.  Nothing moves across the fences: arithmetic
// that follows in the source runs while the last products are under way, not
// before the first.  GROUP 0 leaves the order to the compiler.
template <typename T, int N, int GROUP, typename Read, typename Multiply>
__device__ __forceinline__ void pipelined(const Read &read, const Multiply &multiply) {
    if constexpr (GROUP == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) multiply(i, read(i));
    } else {
    static_assert(N % GROUP == 0, "whole groups");
    Frag<T> a[2][GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) a[0][i] = read(i);
#pragma unroll
    for (int g = 0; g < N / GROUP; ++g) {
        if (g + 1 < N / GROUP) {
#pragma unroll
            for (int i = 0; i < GROUP; ++i) a[(g + 1) & 1][i] = read((g + 1) * GROUP + i);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) multiply(g * GROUP + i, a[g & 1][i]);
        __builtin_amdgcn_sched_barrier(0);
    }
    }
}

// Whether 16 columns of the contracted axis hold any: a step past head_dim is
// left out where it is long (fp32: eight products of 64 clocks).
template <typename T>
__device__ __forceinline__ bool step_counts(const AttnParams &p, int step) {
    return T::bytes == 2 || 16 * step < p.D;
}

// Four consecutive elements of an output row.
template <typename T>
__device__ __forceinline__ void store4(typename T::raw_t *row, int col, int D, bool vec, float a, float b,
                                       float c, float d) {
    if (col >= D) return;
    const float v[4] = {a, b, c, d};
    if (vec) {
        if constexpr (T::bytes == 4) {
            *(tokens_f32x4 *)(row + col) = tokens_f32x4{a, b, c, d};
        } else {
            u32x2 w;
            w[0] = (uint32_t)to_bits<T>(a) | (uint32_t)to_bits<T>(b) << 16;
            w[1] = (uint32_t)to_bits<T>(c) | (uint32_t)to_bits<T>(d) << 16;
            *(u32x2 *)(row + col) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j < D) row[col + j] = to_bits<T>(v[j]);
    }
}

// ----------------------------------------------------- relative positions

// Bucket of one side that distance d >= 0 falls into: the last one whose
// first distance is at most d.
__device__ __forceinline__ int bucket_of(const uint16_t *starts, int side, int d) {
    int lo = 0, hi = side - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= d) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The distance table of a head in LDS: entry rel + border + kLutPad is the
// bias of relative position rel, times log2(e) (the scores are kept in base
// 2), from kLutPad positions before the first distance of the last bucket to
// as many past the last change.  A tile that touches a change of bucket reads
// it without limits on the index; any other tile has one bias, that of its end
// of the table.  A finite bias stays finite (the lowest value of fp32 and bf16,
// a usual mask, would pass the range in base 2).  Returns whether the thread's
// entries hold one that row_shift is for.
template <typename T>
__device__ __forceinline__ bool fill_lut(const AttnParams &p, int h, float *lut, const uint16_t *starts, int t,
                                         int nt) {
    bool large = false;
    for (int i = t; i < p.lut; i += nt) {
        const int rel = i - p.border - kLutPad;
        int b = bucket_of(starts, p.side, rel < 0 ? -rel : (p.bidirectional ? rel : 0));
        if (p.bidirectional && rel > 0) b += p.side;
        const size_t at = (size_t)b * p.H + h;
        float v;
        if (p.table_f32) v = ((const float *)p.table)[at];
        else v = T::from_raw(((const typename T::raw_t *)p.table)[at]);
        const float w = v * kLog2e, held = __builtin_amdgcn_fmed3f(w, -kMaxFloat, kMaxFloat);
        const bool finite = fabsf(v) <= kMaxFloat;
        lut[i] = finite ? held : w;
        large |= finite & (fabsf(w) > kBiasKept);
    }
    return large;
}

// What the biases of a query's scores are taken relative to: the largest one
// among the keys that it sees (0 .. seen - 1), where that passes kBiasKept, else
// 0.  A query whose every key has a mask's bias of, say, -1e9 would otherwise
// lose the products beside it, and the sum of the exponentials in its lse: the
// softmax does not change when a constant leaves every score.  Few queries are
// such, so it costs the others nothing but a test where a tile reads the table.
__device__ __forceinline__ float row_shift(const AttnParams &p, const float *lut, int pos, int seen) {
    if (seen <= 0) return 0.0f;
    const int zero = p.border + kLutPad - pos;       // entry of key 0
    const int lo = min(max(zero, 0), p.lut - 1), hi = min(max(zero + seen - 1, 0), p.lut - 1);
    float top = -INFINITY;
    for (int i = lo; i <= hi; ++i) top = fmaxf(top, lut[i]);
    return fabsf(top) > kBiasKept && fabsf(top) <= kMaxFloat ? top : 0.0f;
}

// A shift in the base of the scores as they are given (a mask's lowest value,
// held to the range in base 2, as that).
__device__ __forceinline__ float natural(float shift) {
    return fabsf(shift) < kMaxFloat ? shift * kLn2 : shift;
}

// N entries of an LDS table, all on their way before the first is used.
template <int N, typename Index>
__device__ __forceinline__ void read_all(const float *at, float *v, const Index &index) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = at[index(i)];
    __builtin_amdgcn_sched_barrier(0);
}

// Which bias the relative positions lo .. hi have: 0 the table's, entry by
// entry; 1 that of its first entry; 2 that of its last; 3 none.
__device__ __forceinline__ int bias_class(const AttnParams &p, int lo, int hi) {
    if (!p.lut) return 3;
    if (hi <= -p.border) return 1;
    return lo >= (p.bidirectional ? p.border : 0) ? 2 : 0;
}

// Writes of a tile by the threads that share it, before its reads by them (and
// the reverse): a block's, or one wave's own.
template <bool WAVE>
__device__ __forceinline__ void tile_sync() {
    if constexpr (WAVE) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        __syncthreads();
    }
}

// Row tile, unit and part of a block.  The eighth of the launch that an XCD runs
// takes whole groups of `group` units (the heads that read one key head) where
// eight divides the groups: their tiles read the same keys from one L2.  An XCD
// gets every eighth group, so that sequences of different lengths spread over
// all of them.  With a causal mask the longest tiles come first, then, from the
// middle on, the shortest, so that the tiles that a compute unit holds at once
// add up to about the same work; `longest_last` tells which end is long.  (1 x 4 x
// 4096 x 64 bf16 in 32-row blocks: 34.2 us, the shortest first 37.5.)
__device__ __forceinline__ bool block_place(const AttnParams &p, bool longest_last, int group, int &unit, int &tile,
                                            int &part) {
    const int x = blockIdx.x & 7, i = (int)(blockIdx.x >> 3);
    const bool whole = p.units % (8 * group) == 0;
    if (whole) {
        const int u = p.units >> 3;
        int local;
        if (p.causal && p.splits == 1) {
            const int step = i / u;
            local = i - step * u;
            const int half = (p.tiles + 1) >> 1;
            tile = step < half ? step : p.tiles - 1 - (step - half);
            part = 0;
        } else {
            int n = i;                               // (unit, tile, part), part fastest
            part = n % p.splits;
            n /= p.splits;
            tile = n % p.tiles;
            local = n / p.tiles;
        }
        unit = (local / group * 8 + x) * group + local % group;
    } else {
        int n = x * ((p.nblocks + 7) >> 3) + i;
        if (n >= p.nblocks) return false;
        part = n % p.splits;
        n /= p.splits;
        tile = n % p.tiles;
        unit = n / p.tiles;
    }
    if (p.causal && longest_last) tile = p.tiles - 1 - tile;
    return true;
}

__device__ __forceinline__ int sequence_length(const AttnParams &p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.Lk) : p.Lk;
}

}  // namespace gs
#endif
