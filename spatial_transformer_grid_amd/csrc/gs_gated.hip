// gs_gated.hip -- gated feed-forward projections, forward and backward:
// Y = act(X Wg^T) * (X Wu^T).
//
// Every product is one kernel on 32 x 32 matrix instructions, out[m][n] = sum
// over k of M(m, k) N(n, k), whose operands lie in memory along k (kAlongK) or
// across it (kAcross; read from LDS transposed):
//   forward   M = X rows        N = Wg and Wu rows, half a tile of each, so that
//             a lane holds a and b of the same element and Y needs no second pass
//   dX        M = da, then db   N = Wg, then Wu across: one sum over both
//   dWg, dWu  M = da, db across N = X across
// N is the A operand of the instructions with its rows permuted (a_row), so that
// a lane has eight neighbouring columns of an output row.  Tiles come by
// asynchronous loads into LDS, the next one while this one is multiplied.  A
// long sum of few tiles is cut into parts over blocks, whose fp32 sums a second
// kernel adds in order.
//
// Up to kSkinnyRows rows the weights are read once, straight into registers:
// sixteen hidden units a block, whose waves share the width.
#include "gs_tokens.hpp"

namespace gs {

namespace {

enum { kForward = 0, kInput = 1, kWeights = 2 };

// ------------------------------------------------------------ activations

// act(a) and its slope.  The exponentials' arguments are at most 0, so that
// nothing overflows.
__device__ __forceinline__ float logistic(float v, float &rest) {
    const float e = expf(-fabsf(v)), r = 1.0f / (1.0f + e), er = e * r;
    rest = v < 0.0f ? r : er;
    return v < 0.0f ? er : r;
}

__device__ __forceinline__ float activation(int kind, float a, float &slope) {
    float rest;
    if (kind == 0) {
        const float s = logistic(a, rest);
        slope = fmaf(a * s, rest, s);
        return a * s;
    }
    if (kind == 1) {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * a);
        slope = fmaf(a * 0.39894228040143268f, expf(-0.5f * a * a), phi);
        return a * phi;
    }
    if (kind == 2) {
        // (1 + tanh z) / 2 is the logistic function of 2 z
        const float z2 = 1.5957691216057308f * fmaf(0.044715f * a * a, a, a), s = logistic(z2, rest);
        slope = fmaf(a * s * rest, 1.5957691216057308f * fmaf(0.134145f * a, a, 1.0f), s);
        return a * s;
    }
    slope = a > 0.0f ? 1.0f : 0.0f;
    return a < 0.0f ? 0.0f : a;                      // (a NaN stays one)
}

// ---------------------------------------------------------------- operands

// How a tile's rows are brought into LDS: 16 bytes a lane, four bytes a lane
// (rows that are only so aligned), or element by element through registers.
enum { kWide = 0, kNarrow = 1, kElements = 2 };

template <typename T>
struct K {
    static constexpr int BK = 128 / T::bytes;        // of the contracted axis a tile
    static constexpr int EPC = 16 / T::bytes;
};

// One operand's tile of ROWS rows of the output by BK of the contracted axis.
// ALONG: LDS rows are the output's, BK columns each.  Else LDS rows are the
// contracted axis', 128 columns each, in ROWS / 128 such blocks one after another.
template <typename T, int ROWS, bool ALONG, int NT>
struct Operand {
    typedef typename T::raw_t raw_t;
    static constexpr int BK = K<T>::BK, EPC = K<T>::EPC, DP = ALONG ? BK : 128;
    static constexpr int CHUNKS = ROWS * BK / EPC, CPR = DP / EPC;
    typedef Tile<T, DP> L;
    static_assert(CHUNKS % NT == 0 && NT % 64 == 0, "whole waves, whole steps");

    // row and column of LDS chunk c's source, relative to the tile
    __device__ __forceinline__ static void source(int c, int &row, int &k, int part) {
        if constexpr (ALONG) {
            const int r = c / CPR;
            row = r;
            k = ((c - r * CPR) ^ L::turn(r)) * EPC + part;
        } else {
            const int block = c / (BK * CPR), q = c - block * (BK * CPR), r = q / CPR;
            k = r;
            row = block * 128 + ((q - r * CPR) ^ L::turn(r)) * EPC + part;
        }
    }

    // The tile at output row row0 and contracted index k0.  `base` is the operand's
    // first element; a row of its storage is `stride` elements.  HALVES: the upper
    // half of the tile's rows is the same rows of `base2`.
    template <bool HALVES>
    __device__ __forceinline__ static void load(raw_t *lds, const raw_t *base, const raw_t *base2, int64_t stride,
                                                int row0, int rows, int k0, int ks, int mode, int t) {
        constexpr int H = HALVES ? ROWS / 2 : ROWS;
        const int64_t first = ALONG ? row0 * stride + k0 : k0 * stride + row0;
        if (mode != kElements) {
            const __amdgpu_buffer_rsrc_t r1 =
                __builtin_amdgcn_make_buffer_rsrc((void *)(base + first), 0, 0x7fffffff, 0x00027000);
            const __amdgpu_buffer_rsrc_t r2 = HALVES
                ? __builtin_amdgcn_make_buffer_rsrc((void *)(base2 + first), 0, 0x7fffffff, 0x00027000) : r1;
            if (mode == kWide) {
#pragma unroll
                for (int n = 0; n < CHUNKS / NT; ++n) {
                    int row, k;
                    source(t + n * NT, row, k, 0);
                    const bool upper = HALVES && n >= CHUNKS / NT / 2;
                    if (upper) row -= H;
                    const bool in = row0 + row < rows && k0 + k < ks;
                    const uint32_t at = in ? (uint32_t)(ALONG ? row * (int)stride + k : k * (int)stride + row) * T::bytes
                                           : 0x80000000u;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        upper ? r2 : r1, (__attribute__((address_space(3))) void *)(lds + ((t & ~63) + n * NT) * EPC), 16,
                        (int)at, 0, 0, 0);
                }
            } else {
                constexpr int PER = 4 / T::bytes;
#pragma unroll 4
                for (int n = 0; n < 4 * CHUNKS / NT; ++n) {
                    int row, k;
                    const int word = t + n * NT;
                    source(word >> 2, row, k, (word & 3) * PER);
                    const bool upper = HALVES && n >= 4 * CHUNKS / NT / 2;
                    if (upper) row -= H;
                    const bool in = row0 + row < rows && k0 + k < ks;
                    const uint32_t at = in ? (uint32_t)(ALONG ? row * (int)stride + k : k * (int)stride + row) * T::bytes
                                           : 0x80000000u;
                    __builtin_amdgcn_raw_ptr_buffer_load_lds(
                        upper ? r2 : r1, (__attribute__((address_space(3))) void *)(lds + ((t & ~63) + n * NT) * PER), 4,
                        (int)at, 0, 0, 0);
                }
            }
            return;
        }
#pragma unroll 1
        for (int n = 0; n < CHUNKS / NT; ++n) {
            raw_t e[EPC];
#pragma unroll
            for (int j = 0; j < EPC; ++j) {
                int row, k;
                source(t + n * NT, row, k, j);
                const raw_t *from = base + first;
                if (HALVES && row >= H) {
                    row -= H;
                    from = base2 + first;
                }
                const bool in = row0 + row < rows && k0 + k < ks;
                e[j] = in ? from[ALONG ? row * stride + k : k * stride + row] : raw_t(0);
            }
            u32x4 v;
            __builtin_memcpy(&v, e, 16);
            *(u32x4 *)(lds + (t + n * NT) * EPC) = v;
        }
    }

    // The instruction's operand for 32 rows from `row` and the 16 steps from k:
    // PERMUTED rows as a_row says, else in order.
    template <bool PERMUTED>
    __device__ __forceinline__ static Frag<T> read(const raw_t *lds, int row, int k, int lane) {
        if constexpr (ALONG) {
            return frag_lds<T, DP>(lds, row + (PERMUTED ? a_row(lane & 31) : lane & 31), k + 8 * (lane >> 5));
        } else {
            const raw_t *block = lds + row / 128 * (128 * BK);
            row &= 127;
            if constexpr (!PERMUTED) {
                return frag_lds_transposed<T, DP>(block, k, row, lane);
            } else if constexpr (T::bytes == 4) {
                Frag<T> f;
                const int col = row + a_row(lane & 31);
#pragma unroll
                for (int j = 0; j < 8; ++j) f.w[j >> 2][j & 3] = block[L::chunk(k + 8 * (lane >> 5) + j, col) + (col & 3)];
                return f;
            } else {
                // of the four groups of four columns a transposing read names, the middle two change places
                const int group = lane & 3, named = (group & 1) << 1 | group >> 1;
                return frag_lds_transposed<T, DP>(block, k, row, (lane & ~3) | named);
            }
        }
    }
};

// ---------------------------------------------------------------- products

// Eight neighbouring columns of a row, from column col of cols.
template <typename T>
__device__ __forceinline__ void store8(typename T::raw_t *row, int col, int cols, bool vec, const float *v) {
    if (vec && col + 8 <= cols) {
        const Frag<T> f = frag_pack<T>(v);
#pragma unroll
        for (int i = 0; i < T::bytes / 2; ++i) *(u32x4 *)(row + col + i * (16 / T::bytes)) = f.w[i];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < cols) row[col + j] = to_bits<T>(v[j]);
    }
}

// Y of eight elements, and a and b beside it.
template <typename T>
__device__ __forceinline__ void store_gated(const GatedParams &p, int m, int n, const float *a, const float *b) {
    typedef typename T::raw_t raw_t;
    if (p.saved) {
        const int64_t plane = (int64_t)p.m * p.n, at = (int64_t)m * p.n;
        store8<F32>((uint32_t *)p.saved + at, n, p.n, p.saved_vec, a);
        store8<F32>((uint32_t *)p.saved + plane + at, n, p.n, p.saved_vec, b);
    }
    float y[8], slope;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = activation(p.activation, a[j], slope) * b[j];
    store8<T>((raw_t *)p.out0 + m * p.out_stride, n, p.n, p.out_vec, y);
}

template <typename T, int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void gated_product(GatedParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int NT = 64 * WM * WN, TM = BM / WM / 32, TN = BN / WN / 32, BK = K<T>::BK;
    typedef Operand<T, BM, MODE != kWeights, NT> OM;
    typedef Operand<T, BN, MODE == kForward, NT> ON;
    constexpr int STAGE = (BM + BN) * BK;
    constexpr int COLS = MODE == kForward ? BN / 2 : BN;    // of the output
    extern __shared__ __align__(16) unsigned char smem[];
    raw_t *const lds = (raw_t *)smem;
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = wave / WN, wn = wave % WN;

    // Tiles of an XCD are neighbours: eight tiles of rows by as many of columns as it
    // runs at once, so that they share operands in its L2.
    const int per = (p.blocks + 7) >> 3;
    int id = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (id >= p.blocks) return;
    const int part = id % p.parts;
    id /= p.parts;
    const int which = MODE == kWeights ? id / (p.tiles_m * p.tiles_n) : 0;
    if (MODE == kWeights) id -= which * (p.tiles_m * p.tiles_n);
    const int group = id / (8 * p.tiles_n), first = group * 8, high = min(p.tiles_m - first, 8);
    id -= group * 8 * p.tiles_n;
    const int m0 = (first + id % high) * BM, n0 = id / high * COLS;

    // the contracted axis in tiles: all of da and Wg, then all of db and Wu
    const int per_half = (p.k + BK - 1) / BK, all = MODE == kInput ? 2 * per_half : per_half;
    const int s0 = (int)((int64_t)all * part / p.parts), s1 = (int)((int64_t)all * (part + 1) / p.parts);
    const auto load = [&](int s, raw_t *to) {
        const int half = MODE == kInput && s >= per_half ? 1 : 0, k0 = (s - half * per_half) * BK;
        const raw_t *const mb = (const raw_t *)(MODE == kWeights ? (which ? p.m1 : p.m0) : half ? p.m1 : p.m0);
        OM::template load<false>(to, mb, mb, p.m_stride, m0, p.m, k0, p.k, p.m_mode, t);
        const raw_t *const nb = (const raw_t *)(half ? p.n1 : p.n0);
        ON::template load<MODE == kForward>(to + BM * BK, nb, (const raw_t *)p.n1, p.n_stride, n0, p.n, k0, p.k, p.n_mode, t);
    };
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    // of a forward tile a wave has the same columns of Wg and of Wu
    const auto n_row = [&](int j) {
        if (MODE == kForward) return (j < TN / 2 ? 0 : BN / 2) + (wn * (TN / 2) + j % (TN / 2)) * 32;
        return (wn * TN + j) * 32;
    };
    if (s0 < s1) load(s0, lds);
    for (int s = s0; s < s1; ++s) {
        const raw_t *const tile = lds + ((s - s0) & 1) * STAGE;
        async_wait();
        __syncthreads();
        if (s + 1 < s1) load(s + 1, lds + ((s + 1 - s0) & 1) * STAGE);
#pragma unroll
        for (int k = 0; k < BK; k += 16) {
            Frag<T> a[TN], b[TM];
#pragma unroll
            for (int j = 0; j < TN; ++j) a[j] = ON::template read<true>(tile + BM * BK, n_row(j), k, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i) b[i] = OM::template read<false>(tile, (wm * TM + i) * 32, k, lane);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) mma<T>(acc[i][j], a[j], b[i]);
        }
    }

    constexpr int HALF = MODE == kForward ? TN / 2 : TN;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int m = m0 + (wm * TM + i) * 32 + (lane & 31);
        if (m >= p.m) continue;
#pragma unroll
        for (int j = 0; j < HALF; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int n = n0 + (wn * HALF + j) * 32 + 16 * u + 8 * (lane >> 5);
                float v[8], w[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[r] = acc[i][j][8 * u + r];
                    w[r] = MODE == kForward ? acc[i][j + HALF][8 * u + r] : 0.0f;
                }
                if (n >= p.n) continue;
                if (p.parts > 1) {
                    // rows of partial sums are padded to eight columns
                    const int64_t width = (p.n + 7) / 8 * 8, plane = (int64_t)p.m * width, planes = MODE == kInput ? 1 : 2;
                    float *to = p.partial + (part * planes + which) * plane + m * width;
                    store8<F32>((uint32_t *)to, n, (int)width, true, v);
                    if (MODE == kForward) store8<F32>((uint32_t *)to + plane, n, (int)width, true, w);
                } else if (MODE == kForward) {
                    store_gated<T>(p, m, n, v, w);
                } else {
                    store8<T>((raw_t *)(which ? p.out1 : p.out0) + m * p.out_stride, n, p.n, p.out_vec, v);
                }
            }
    }
}

// The parts' sums, in order, and what follows them.
template <typename T, int MODE>
__global__ __launch_bounds__(256) void gated_join(GatedParams p) {
    typedef typename T::raw_t raw_t;
    const int64_t width = (p.n + 7) / 8 * 8, chunks = width / 8, plane = (int64_t)p.m * width;
    const int planes = MODE == kInput ? 1 : 2;
    const int64_t items = (MODE == kWeights ? 2 : 1) * (int64_t)p.m * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t line = i / chunks;
        const int n = (int)(i - line * chunks) * 8, which = (int)(line / p.m), m = (int)(line - (int64_t)which * p.m);
        const float *from = p.partial + which * plane + m * width + n;
        float v[8] = {}, w[8] = {};
        for (int part = 0; part < p.parts; ++part) {
            const Frag<F32> a = frag_global<F32>((const uint32_t *)from, 0, 8, true, true);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += frag_get<F32>(a, j);
            if (MODE == kForward) {
                const Frag<F32> b = frag_global<F32>((const uint32_t *)from + plane, 0, 8, true, true);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] += frag_get<F32>(b, j);
            }
            from += planes * plane;
        }
        if (MODE == kForward) store_gated<T>(p, m, n, v, w);
        else store8<T>((raw_t *)(which ? p.out1 : p.out0) + m * p.out_stride, n, p.n, p.out_vec, v);
    }
}

// ------------------------------------------------------- gradients of a, b

// da = dY b act'(a) and db = dY act(a), rounded to T, in rows of whole chunks of
// eight whose rest is zero.
template <typename T>
__global__ __launch_bounds__(256) void gated_gradients(GatedParams p) {
    typedef typename T::raw_t raw_t;
    const int64_t width = (p.n + 7) / 8 * 8, chunks = width / 8, items = (int64_t)p.m * chunks;
    const int64_t plane = (int64_t)p.m * p.n;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / chunks;
        const int n = (int)(i - m * chunks) * 8;
        const uint32_t *const a = (const uint32_t *)p.saved + m * p.n;
        const Frag<T> g = frag_global<T>((const raw_t *)p.dy + m * p.dy_stride, n, p.n, true, p.out_vec);
        const Frag<F32> fa = frag_global<F32>(a, n, p.n, true, p.saved_vec);
        const Frag<F32> fb = frag_global<F32>(a + plane, n, p.n, true, p.saved_vec);
        float da[8], db[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float slope;
            const float d = frag_get<T>(g, j), f = activation(p.activation, frag_get<F32>(fa, j), slope);
            da[j] = n + j < p.n ? d * frag_get<F32>(fb, j) * slope : 0.0f;
            db[j] = n + j < p.n ? d * f : 0.0f;
        }
        store8<T>((raw_t *)p.out0 + m * width, n, (int)width, true, da);
        store8<T>((raw_t *)p.out1 + m * width, n, (int)width, true, db);
    }
}

// ---------------------------------------------------------------- few rows

typedef __attribute__((ext_vector_type(4))) float f32x4_t;

// 16 x 16 products of what a lane's eight elements along k name: row lane % 16,
// four lanes a row.  It gets column lane % 16 and rows 4 (lane / 16) .. + 3.
template <typename T>
__device__ __forceinline__ f32x4_t mma16(f32x4_t acc, const Frag<T> &a, const Frag<T> &b) {
    if constexpr (T::bytes == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(frag_get<T>(a, j), frag_get<T>(b, j), acc, 0, 0, 0);
        return acc;
    } else if constexpr (__is_same(T, BF16)) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8, a.w[0]), __builtin_bit_cast(bf16v8, b.w[0]),
                                                       acc, 0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16v8, a.w[0]), __builtin_bit_cast(f16v8, b.w[0]),
                                                      acc, 0, 0, 0);
    }
}

constexpr int kSkinnyWaves = 8, kSkinnyAhead = 4;

// RG groups of sixteen rows.  Wave w takes steps w, w + 8, .. of 32 of the width,
// kSkinnyAhead of them in flight.
template <typename T, int RG>
__global__ __launch_bounds__(64 * kSkinnyWaves) void gated_skinny(GatedParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ f32x4_t part[kSkinnyWaves][2 * RG][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (int)blockIdx.x * 16, row = lane & 15, steps = (p.k + 31) / 32;
    const bool on = n0 + row < p.n;
    const raw_t *const wg = (const raw_t *)p.n0 + (int64_t)(n0 + row) * p.k;
    const raw_t *const wu = (const raw_t *)p.n1 + (int64_t)(n0 + row) * p.k;
    f32x4_t acc[2 * RG];
#pragma unroll
    for (int i = 0; i < 2 * RG; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const bool nvec = p.n_mode == kWide, mvec = p.m_mode == kWide;
    for (int s0 = wave; s0 < steps; s0 += kSkinnyWaves * kSkinnyAhead) {
        Frag<T> g[kSkinnyAhead], u[kSkinnyAhead];
#pragma unroll
        for (int j = 0; j < kSkinnyAhead; ++j) {
            const int k = (s0 + j * kSkinnyWaves) * 32 + 8 * (lane >> 4);
            g[j] = frag_global<T>(wg, k, p.k, on, nvec);
            u[j] = frag_global<T>(wu, k, p.k, on, nvec);
        }
#pragma unroll
        for (int j = 0; j < kSkinnyAhead; ++j) {
            const int k = (s0 + j * kSkinnyWaves) * 32 + 8 * (lane >> 4);
#pragma unroll
            for (int i = 0; i < RG; ++i) {
                const int m = 16 * i + row;
                const Frag<T> x = frag_global<T>((const raw_t *)p.m0 + m * p.m_stride, k, p.k, m < p.m, mvec);
                acc[2 * i] = mma16<T>(acc[2 * i], g[j], x);
                acc[2 * i + 1] = mma16<T>(acc[2 * i + 1], u[j], x);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2 * RG; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    // one element of Y a thread: row m of X, hidden unit n
    for (int i = threadIdx.x; i < 256 * RG; i += 64 * kSkinnyWaves) {
        const int m = i >> 4, n = i & 15, from = (n >> 2) * 16 + (m & 15);
        float a = 0.0f, b = 0.0f, slope;
#pragma unroll
        for (int w = 0; w < kSkinnyWaves; ++w) {
            a += part[w][2 * (m >> 4)][from][n & 3];
            b += part[w][2 * (m >> 4) + 1][from][n & 3];
        }
        if (m >= p.m || n0 + n >= p.n) continue;
        const int64_t at = (int64_t)m * p.n + n0 + n;
        if (p.saved) {
            p.saved[at] = a;
            p.saved[(int64_t)p.m * p.n + at] = b;
        }
        ((raw_t *)p.out0)[m * p.out_stride + n0 + n] = to_bits<T>(activation(p.activation, a, slope) * b);
    }
}

// --------------------------------------------------------------- launches

constexpr int kSkinnyRows = 64;

int tiles_of(int64_t n, int size) { return (int)((n + size - 1) / size); }

// Tiles of the output of a product, 256 or 128 rows and columns each, and the
// parts of its sum.
struct Shape {
    int big, tiles_m, tiles_n, parts;
    int64_t blocks;
};

Shape shape_of(int mode, int dtype, int64_t m, int64_t n, int64_t k) {
    Shape s = {};
    const int planes = mode == kWeights ? 2 : 1;
    for (s.big = 1; s.big >= 0; --s.big) {
        const int size = s.big ? 256 : 128;
        s.tiles_m = tiles_of(m, size);
        s.tiles_n = tiles_of(n, mode == kForward ? size / 2 : size);
        s.blocks = (int64_t)planes * s.tiles_m * s.tiles_n;
        if (s.big == 0 || s.blocks >= 200) break;
    }
    const int64_t steps = (int64_t)tiles_of(k, dtype == 0 ? 32 : 64) * (mode == kInput ? 2 : 1);
    s.parts = 1;
    if (s.blocks < 192) {
        int64_t parts = 512 / s.blocks;
        if (parts > steps / 4) parts = steps / 4;
        if (parts > 64) parts = 64;
        if (parts > 1) s.parts = (int)parts;
    }
    s.blocks *= s.parts;
    return s;
}

template <typename T, int MODE, int SIZE, int WM, int WN>
int launch_tiles(const GatedParams &p, hipStream_t stream) {
    const auto fn = gated_product<T, MODE, SIZE, SIZE, WM, WN>;
    const int smem = 2 * 2 * SIZE * 128;
    const hipError_t e = hipFuncSetAttribute((const void *)fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != hipSuccess) return (int)e;
    hipLaunchKernelGGL(fn, dim3((unsigned)((p.blocks + 7) / 8 * 8)), dim3(64 * WM * WN), smem, stream, p);
    return (int)hipGetLastError();
}

template <typename T, int MODE>
int product(GatedParams p, int dtype, hipStream_t stream) {
    const Shape s = shape_of(MODE, dtype, p.m, p.n, p.k);
    p.tiles_m = s.tiles_m;
    p.tiles_n = s.tiles_n;
    p.parts = p.partial ? s.parts : 1;
    p.blocks = (int)(s.blocks / s.parts * p.parts);
    const int e = s.big ? launch_tiles<T, MODE, 256, 2, 4>(p, stream) : launch_tiles<T, MODE, 128, 2, 2>(p, stream);
    if (e || p.parts == 1) return e;
    const int64_t items = (MODE == kWeights ? 2 : 1) * (int64_t)p.m * ((p.n + 7) / 8), blocks = (items + 255) / 256;
    hipLaunchKernelGGL((gated_join<T, MODE>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int run(const GatedParams &p, int mode, int dtype, hipStream_t stream) {
    if (mode == kGatedForward) {
        if (p.m <= kSkinnyRows) {
            const dim3 grid((unsigned)tiles_of(p.n, 16)), block(64 * kSkinnyWaves);
            if (p.m <= 16) hipLaunchKernelGGL((gated_skinny<T, 1>), grid, block, 0, stream, p);
            else if (p.m <= 32) hipLaunchKernelGGL((gated_skinny<T, 2>), grid, block, 0, stream, p);
            else hipLaunchKernelGGL((gated_skinny<T, 4>), grid, block, 0, stream, p);
            return (int)hipGetLastError();
        }
        return product<T, kForward>(p, dtype, stream);
    }
    if (mode == kGatedInput) return product<T, kInput>(p, dtype, stream);
    if (mode == kGatedWeights) return product<T, kWeights>(p, dtype, stream);
    const int64_t items = (int64_t)p.m * ((p.n + 7) / 8), blocks = (items + 255) / 256;
    hipLaunchKernelGGL(gated_gradients<T>, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

}  // namespace

// Floats of the parts' sums of a product (0: its sum is not cut).
int64_t gated_partial_floats(int mode, int dtype, int64_t m, int64_t n, int64_t k) {
    if (m == 0 || n == 0 || (mode == kGatedForward && m <= kSkinnyRows)) return 0;
    const Shape s = shape_of(mode, dtype, m, n, k);
    if (s.parts == 1) return 0;
    return (int64_t)s.parts * (mode == kGatedInput ? 1 : 2) * m * ((n + 7) / 8 * 8);
}

int64_t gated_blocks(int mode, int dtype, int64_t m, int64_t n, int64_t k) {
    return m == 0 || n == 0 ? 0 : shape_of(mode, dtype, m, n, k).blocks;
}

int launch_gated(const GatedParams &p, int mode, int dtype, hipStream_t stream) {
    if (dtype == 0) return run<F32>(p, mode, dtype, stream);
    if (dtype == 1) return run<F16>(p, mode, dtype, stream);
    return run<BF16>(p, mode, dtype, stream);
}

}  // namespace gs
