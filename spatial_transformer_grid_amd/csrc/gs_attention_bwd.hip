// gs_attention_bwd.hip -- gradients of attention with a relative position bias.
//
// With P the probabilities, M the dropout's factors (0 or keep_scale) and
// delta_i = sum_j P_ij M_ij (dO_i . V_j) = dO_i . O_i:
//   dS_ij = P_ij (M_ij (dO_i . V_j) - delta_i),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = (P M)^T dO,
//   dtable[n] = sum of dS_ij over the pairs whose distance is in bucket n.
// P is computed again from the scores and lse.  Two kernels: one per query
// tile (dQ, delta), one per key tile (dK, dV, the table's sums, over all query
// heads that share the key head).  Each output element has one writer
// and a fixed order of summation; the price is the scores and dO V^T twice,
// seven products in place of the five of a single pass that would add dQ with
// atomics, in an order that varies.
//
// O has been rounded, so that dO . O is delta only to that rounding, and what is
// wrong in it does not cancel where many dS of a query are added up (a bucket
// that holds most keys: its sum is that of the few others, negated).  But the
// exact dS of a query add up to 0, so the sum of those computed with dO . O
// tells delta exactly: the dQ kernel corrects it for the dK / dV kernel, which
// therefore makes the table's sums, and where a block sees at most kExactKeys
// keys it goes over them once more with the corrected delta for its own dQ.
//
// M's factor is 0 or 1 beside dO . V, delta is divided by keep_scale, and P carries
// keep_scale in its exponent: dS and P M are then rounded to the element type as
// they are (an fp16 dS without the factor of 10 of a ratio of 0.9 loses three bits
// below the smallest normal value).
//
// Measured: 16 heads of 4096 x 4096 x 128 fp16 on four key heads, with a bias:
// dQ 230 us (900 TFLOP/s over its three products), dK and dV 445 to 460 us (600
// over four; K, V and both sums fill the registers of a SIMD's one wave, whose
// products and exponentials follow one another); 2 x 16 x 2048 x 64 causal
// bf16 with bias and dropout: 74 to 80 and 108 to 116 us, of which the generator
// takes 13 and 20, the bias 7 and 18.
#include "gs_tokens.hpp"

namespace gs {

namespace {

// Queries of a block that sees at most this many keys get the corrected delta in dQ
// too.  Without it the error of dQ is 1.6 times the rounding's own at 2 keys and
// 1.05 times at 32 where V has no mean, 1.5 times at any number where V's mean is
// its deviation, 10 times where it is eight of them (bf16 and fp16, against 64
// bits).  The second pass takes a sixth of the backward pass (64 x 16 x 256 x 64
// bf16: 247 us, without it 213; 8 x 8 x 256 x 64 fp32: 97 and 87; 4 x 8 x 144 x 16
// fp32: 36 and 33): taken where a call is short, left out where it would cost 100
// us and more.
constexpr int kExactKeys = 256;

// Sums of dS by distance.  A wave writes a 32 x 32 part of dS to LDS, a key a
// row of kDiagonalRow floats of which the last 36 stay zero; lane d then adds
// up the diagonal query - key = d - 31, an element a row (what lies left or
// right of a row's 32 are the zeros of the row before or its own), and adds the
// sum to the wave's entry for that distance.  The row length spreads the rows
// over the banks.  LDS adds by atomics in the place of the
// 32 reads cost about 180 cycles an instruction.
constexpr int kDiagonalRow = 68;
constexpr int kDiagonal = 32 + 32 * kDiagonalRow;    // floats of a wave

// What the dK / dV kernel takes of 64 queries from the dQ kernel: log2(fold) - lse
// (base 2, relative to the row's shift) without and with the biases of the two ends of the
// table, and delta / keep_scale; 64 of each, so that one asynchronous load of a wave
// brings them.  Queries past the last have -inf: their probabilities are 0.  The
// shifts themselves, read where a table has any, follow the stats of all rows.
constexpr int kRowStats = 4 * 64;

__device__ __forceinline__ float *row_stats(const AttnParams &p, int64_t bh, int tile) {
    return p.rows + (bh * ((p.Lq + 63) >> 6) + tile) * kRowStats;
}

__device__ __forceinline__ float *row_shifts(const AttnParams &p, int64_t bh) {
    const int64_t tiles = (p.Lq + 63) >> 6;
    return p.rows + (int64_t)p.B * p.H * tiles * kRowStats + bh * tiles * 64;
}

__device__ __forceinline__ void put_row(const AttnParams &p, int64_t bh, int q, float minus_lse, float lo, float hi,
                                        float delta, float shift) {
    float *s = row_stats(p, bh, q >> 6) + (q & 63);
    s[0] = minus_lse;
    s[64] = lo;
    s[128] = hi;
    s[192] = delta;
    if (p.lut) row_shifts(p, bh)[q] = shift;
}

// The stats of 64 rows into LDS, by one wave.
__device__ __forceinline__ void copy_rows(float *lds, const float *from, int lane) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void *)from, 0, kRowStats * 4, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)lds, 16, lane * 16, 0, 0, 0);
}

// Geometry of both kernels.  WS: into how many parts (1 or 4) the waves of a block
// split the axis that is walked; a block has BLOCK = 128 / WS rows of the other.  ROWS
// rows of the walked axis in an LDS tile, two buffers of two tensors, a block's
// or each wave's own (FEW; one where two would take more than half of the LDS).
template <typename T, int DP, int WS, bool KV>
struct BwdGeo {
    static constexpr bool FEW = WS == 4;
    static constexpr int BLOCK = kAttnRows / WS;
    // (64 rows of 128 columns leave a compute unit one block: no loss to the
    // dK / dV kernel, whose registers allow no more, and fewer barriers)
    static constexpr int ROWS = FEW || T::bytes == 4 || (!KV && DP > 64) ? 32 : 64;
    static constexpr int tile_elems = ROWS * DP;
    static constexpr int bufs = FEW && DP * T::bytes > 128 ? 1 : 2;       // of a block, or of a wave
    static constexpr int copies = (FEW ? 4 : 1) * bufs;
    static constexpr int SUM = DP + 4;
    static constexpr int own_bytes = copies * 2 * tile_elems * T::bytes;
    // (WS > 1: the parts' sums take the tiles' place)
    static constexpr int tile_bytes = WS > 1 && 128 * SUM * 4 > own_bytes ? 128 * SUM * 4 : own_bytes;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// A wave's 32-row result (transposed: the lane's column is its row) into LDS,
// from row `row` of its part on.
template <int DP, int SUM>
__device__ __forceinline__ void put_sums(float *sums, const f32x16 *acc, int row, int lane) {
    float *mine = sums + (row + (lane & 31)) * SUM + 4 * (lane >> 5);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            *(tokens_f32x4 *)(mine + 32 * d + 2 * r) =
                tokens_f32x4{acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]};
}

template <int SUM, int WS>
__device__ __forceinline__ tokens_f32x4 add_sums(const float *sums, int r, int at) {
    tokens_f32x4 v = *(const tokens_f32x4 *)(sums + r * SUM + at);
#pragma unroll
    for (int w = 1; w < WS; ++w) v += *(const tokens_f32x4 *)(sums + (w * (128 / WS) + r) * SUM + at);
    return v;
}

template <typename T, int DP, bool DROP, int WS>
__global__ __launch_bounds__(256, (WS == 4 || T::bytes == 4) && DP > 64 ? 1 : 2) void attention_backward_q(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef BwdGeo<T, DP, WS, false> Geo;
    constexpr bool FEW = Geo::FEW;
    constexpr int KEYS = Geo::ROWS, BLOCK = Geo::BLOCK, NT = FEW ? 64 : 256;
    extern __shared__ __align__(16) unsigned char smem[];
    float *lut = (float *)(smem + Geo::tile_bytes);
    uint16_t *starts = (uint16_t *)(lut + (p.lut + 3) / 4 * 4);
    __shared__ float row_sums[WS][BLOCK], row_tops[WS][BLOCK];
    __shared__ float shifts[BLOCK];                  // row_shift of each row, where `shifted`
    __shared__ int large;                            // the table holds a bias that row_shift is for

    int unit, tile, part;
    if (!block_place(p, true, p.G, unit, tile, part)) return;
    const int b = unit / p.H, h = unit - b * p.H, hk = h / p.G;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int len = sequence_length(p, b);
    const int first = p.from_end ? len - p.Lq : p.first;
    const int rg = wave % (4 / WS), wp = wave / (4 / WS);   // the wave's 32 rows, its part of the keys
    const int q0 = tile * BLOCK + rg * 32;
    const int qi = q0 + (lane & 31);
    const int pos = first + qi;
    const int block_last = first + min((tile + 1) * BLOCK, p.Lq) - 1;
    const int end = p.causal ? min(len, block_last + 1) : len;
    const int wave_first = first + q0, wave_last = wave_first + 31;
    const int begin = FEW ? wave * KEYS : 0;
    constexpr int STEP = FEW ? 4 * KEYS : KEYS;
    const bool vec = p.vec, live = qi < p.Lq;

    const raw_t *kb = (const raw_t *)p.k + (int64_t)b * p.ks[0] + (int64_t)hk * p.ks[1];
    const raw_t *vb = (const raw_t *)p.v + (int64_t)b * p.vs[0] + (int64_t)hk * p.vs[1];
    const int tt = FEW ? lane : t;
    raw_t *Kt = (raw_t *)smem + (FEW ? wave * Geo::bufs * 2 * Geo::tile_elems : 0);
    const auto load = [&](raw_t *to, int k0) {
        copy_tile<T, DP, KEYS, NT>(to, kb, p.ks[2], k0, end, p.D, p.async, vec, tt);
        copy_tile<T, DP, KEYS, NT>(to + Geo::tile_elems, vb, p.vs[2], k0, end, p.D, p.async, vec, tt);
    };
    if (begin < end) load(Kt, begin);
    Frag<T> qf[DP / 16], gf[DP / 16];
    float delta = 0.0f;
    {
        const raw_t *qrow =
            (const raw_t *)p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)qi * p.qs[2];
        const raw_t *grow =
            (const raw_t *)p.d_o + (int64_t)b * p.dos[0] + (int64_t)h * p.dos[1] + (int64_t)qi * p.dos[2];
        const raw_t *orow =
            (const raw_t *)p.o_in + (int64_t)b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)qi * p.os[2];
#pragma unroll
        for (int s = 0; s < DP / 16; ++s) {
            const int col = 16 * s + 8 * half;
            qf[s] = frag_global<T>(qrow, col, p.D, live, vec);
            gf[s] = frag_global<T>(grow, col, p.D, live, vec);
            const Frag<T> of = frag_global<T>(orow, col, p.D, live, vec);
#pragma unroll
            for (int j = 0; j < 8; ++j) delta = fmaf(frag_get<T>(gf[s], j), frag_get<T>(of, j), delta);
        }
    }
    delta += __shfl_xor(delta, 32);
    float minus_lse = -INFINITY;                     // 2^(s - inf) = 0: no key seen
    if (live) {
        const int64_t at = (int64_t)unit * p.Lq + qi;
        const float v = p.lse[at];
        if (v != -INFINITY) minus_lse = p.fold_log2 - v * kLog2e;
    }
    delta = delta / p.keep_scale;
    float bias_lo = 0.0f, bias_hi = 0.0f;
    bool shifted = false;
    const int col = rg * 32 + (lane & 31);           // the lane's row in the block
    if (p.lut) {
        if (t == 0) large = 0;
        for (int i = t; i < p.side; i += 256) starts[i] = p.starts[i];
        __syncthreads();
        if (fill_lut<T>(p, h, lut, starts, t, 256)) large = 1;
        __syncthreads();
        bias_lo = lut[0];
        bias_hi = lut[p.lut - 1];
        shifted = __builtin_amdgcn_readfirstlane(large);
    }
    if (__builtin_expect(shifted, 0)) {
        const float shift = row_shift(p, lut, pos, p.causal ? min(len, pos + 1) : len);
        bias_lo -= shift;
        bias_hi -= shift;
        shifts[col] = shift;                         // (kept there: no register of the loop's)
        if (__syncthreads_or(shift != 0.0f)) {
            // the lse of a row with a shift has lost the sum beside it: maximum and
            // sum of the exponentials once more, relative to the shift
            float top = -INFINITY, sum = 0.0f;
            for (int k0 = begin, n = 0; k0 < end; k0 += STEP, ++n) {
                const raw_t *Ks = Kt + (Geo::bufs == 2 ? (n & 1) * 2 * Geo::tile_elems : 0);
                async_wait();
                tile_sync<FEW>();
                const bool more = k0 + STEP < end;
                if (Geo::bufs == 2 && more) load(Kt + ((n + 1) & 1) * 2 * Geo::tile_elems, k0 + STEP);
#pragma unroll 1
                for (int u = 0; u < KEYS / 32; ++u) {
                    const int ku = k0 + 32 * u, key0 = ku + 8 * half;
                    if (q0 >= p.Lq || ku >= end || (p.causal && ku > wave_last)) continue;
                    f32x16 st;
#pragma unroll
                    for (int r = 0; r < 16; ++r) st[r] = 0.0f;
                    const int row = 32 * u + a_row(lane & 31);
                    pipelined<T, DP / 16, 1>([&](int i) { return frag_lds<T, DP>(Ks, row, 16 * i + 8 * half); },
                                             [&](int i, const Frag<T> &a) {
                                                 if (step_counts<T>(p, i)) mma<T>(st, a, qf[i]);
                                             });
                    const int cls = bias_class(p, ku - wave_last, ku + 31 - wave_first);
                    const int seen = (p.causal ? min(end, pos + 1) : end) - key0;
                    float high = top;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = 16 * (i >> 3) + (i & 7);
                        const float c = cls == 0 ? lut[key0 - pos + p.border + kLutPad + j] - shift
                                                 : cls == 1 ? bias_lo : bias_hi;
                        st[i] = j < seen ? fmaf(st[i], p.scale2, c) : -INFINITY;
                        high = fmaxf(high, st[i]);
                    }
                    const float from = high == -INFINITY ? 0.0f : high;
                    sum *= __builtin_amdgcn_exp2f(top - from);
#pragma unroll
                    for (int i = 0; i < 16; ++i) sum += __builtin_amdgcn_exp2f(st[i] - from);
                    top = high;
                }
                if (Geo::bufs == 1 && more) {
                    tile_sync<true>();
                    load(Kt, k0 + STEP);
                }
            }
            float all = fmaxf(top, other_half(top));
            if constexpr (WS > 1) {
                if (half == 0) row_tops[wp][col] = all;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < WS; ++w) all = fmaxf(all, row_tops[w][col]);
            }
            sum *= __builtin_amdgcn_exp2f(top - (all == -INFINITY ? 0.0f : all));
            sum += other_half(sum);
            if constexpr (WS > 1) {
                if (half == 0) row_sums[wp][col] = sum;
                __syncthreads();
                sum = 0.0f;
#pragma unroll
                for (int w = 0; w < WS; ++w) sum += row_sums[w][col];
            }
            if (shift != 0.0f) minus_lse = p.fold_log2 - (all + __builtin_amdgcn_logf(sum));
            __syncthreads();
            if (begin < end) load(Kt, begin);
        }
    }
    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

    const int passes = end <= kExactKeys ? 2 : 1;
    for (int pass = 0; pass < passes; ++pass) {
        const bool last = pass == passes - 1;
        float sum = 0.0f;                            // of the query's dS
        if (pass > 0) {
            __syncthreads();
            if (begin < end) load(Kt, begin);
        }
        for (int k0 = begin, n = 0; k0 < end; k0 += STEP, ++n) {
            const raw_t *Ks = Kt + (Geo::bufs == 2 ? (n & 1) * 2 * Geo::tile_elems : 0);
            const raw_t *Vs = Ks + Geo::tile_elems;
            async_wait();
            tile_sync<FEW>();
            const bool more = k0 + STEP < end;
            if (Geo::bufs == 2 && more) load(Kt + ((n + 1) & 1) * 2 * Geo::tile_elems, k0 + STEP);
#pragma unroll
            for (int u = 0; u < KEYS / 32; ++u) {
                const int ku = k0 + 32 * u;              // this 32-key part
                if (q0 >= p.Lq || ku >= end || (p.causal && ku > wave_last)) continue;
                f32x16 st, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) st[r] = dp[r] = 0.0f;
                const int row = 32 * u + a_row(lane & 31);
                pipelined<T, 2 * (DP / 16), T::bytes == 4 ? 1 : 4>(
                    [&](int i) { return frag_lds<T, DP>(i & 1 ? Vs : Ks, row, 8 * (i & ~1) + 8 * half); },
                    [&](int i, const Frag<T> &a) {
                        if (step_counts<T>(p, i >> 1)) mma<T>(i & 1 ? dp : st, a, i & 1 ? gf[i >> 1] : qf[i >> 1]);
                    });
                const int key0 = ku + 8 * half;
                u32x4 rnd[2];                            // the generator runs while the products do
                if constexpr (DROP)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        rnd[x] = philox((uint32_t)(key0 + 16 * x) >> 3, (uint32_t)qi, (uint32_t)unit, p.call, p.seed_lo,
                                        p.seed_hi);
                const int cls = bias_class(p, ku - wave_last, ku + 31 - wave_first);
                float e[16];
                if (cls == 0) {
                    float bias[16];
                    read_all<16>(lut + (key0 - pos + p.border + kLutPad), bias,
                                 [](int i) { return 16 * (i >> 3) + (i & 7); });
                    if (__builtin_expect(shifted, 0)) {
                        rare<16>(bias);
                        const float shift = *(volatile float *)(shifts + col);
#pragma unroll
                        for (int i = 0; i < 16; ++i) bias[i] -= shift;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        e[i] = __builtin_amdgcn_exp2f(fmaf(st[i], p.scale2, bias[i]) + minus_lse);
                } else {
                    const float c = minus_lse + (cls == 1 ? bias_lo : cls == 2 ? bias_hi : 0.0f);
#pragma unroll
                    for (int i = 0; i < 16; ++i) e[i] = __builtin_amdgcn_exp2f(fmaf(st[i], p.scale2, c));
                }
                float ds[16];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int i = 8 * x + j;
                        float g = dp[i];
                        if constexpr (DROP) g = kept(rnd[x], j, p.threshold) ? g : 0.0f;
                        ds[i] = e[i] * (g - delta);
                    }
                }
                if (ku + 32 > end || (p.causal && ku + 31 > wave_first)) {
                    rare<16>(ds);
                    int seen = p.causal ? min(end, pos + 1) : end;
                    seen = (seen == 1 ? 0 : seen) - key0;    // the softmax of one key does not change
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * (i >> 3) + (i & 7) >= seen) ds[i] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 16; i += 4) sum += (ds[i] + ds[i + 1]) + (ds[i + 2] + ds[i + 3]);
                if (!last) continue;
                // dS in K's type, as P in the forward pass (with V's)
                const Frag<T> df[2] = {frag_pack<T>(ds), frag_pack<T>(ds + 8)};
                pipelined<T, 2 * (DP / 32), T::bytes == 4 ? 1 : DP / 32>(
                    [&](int i) {
                        return frag_lds_transposed<T, DP>(Ks, 32 * u + 16 * (i / (DP / 32)), 32 * (i % (DP / 32)), lane);
                    },
                    [&](int i, const Frag<T> &a) { mma<T>(acc[i % (DP / 32)], a, df[i / (DP / 32)]); });
            }
            if (Geo::bufs == 1 && more) {
                tile_sync<true>();
                load(Kt, k0 + STEP);
            }
        }
        sum += other_half(sum);
        if constexpr (WS > 1) {
            if (half == 0) row_sums[wp][col] = sum;
            __syncthreads();
            sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WS; ++w) sum += row_sums[w][col];
        }
        delta += sum / p.fold;
    }
    if (live && half == 0 && wp == 0)
        put_row(p, unit, qi, minus_lse, minus_lse + bias_lo, minus_lse + bias_hi, delta, shifted ? shifts[col] : 0.0f);
    if (tile == p.tiles - 1)
        for (int q = p.Lq + t; q < (p.Lq + 63) / 64 * 64; q += 256)
            put_row(p, unit, q, -INFINITY, -INFINITY, -INFINITY, 0.0f, 0.0f);
    const float scale = p.scale * p.rest;
    if constexpr (WS == 1) {
        if (live) {
            raw_t *drow = (raw_t *)p.dq + (int64_t)b * p.dqs[0] + (int64_t)h * p.dqs[1] + (int64_t)qi * p.dqs[2];
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4)
                    store4<T>(drow, 32 * d + 2 * r + 4 * half, p.D, vec, acc[d][r] * scale, acc[d][r + 1] * scale,
                              acc[d][r + 2] * scale, acc[d][r + 3] * scale);
        }
    } else {
        float *sums = (float *)smem;
        __syncthreads();
        put_sums<DP, Geo::SUM>(sums, acc, wp * BLOCK + rg * 32, lane);
        __syncthreads();
        for (int i = t; i < BLOCK * (DP / 4); i += 256) {
            const int r = i / (DP / 4), at = (i - r * (DP / 4)) * 4, q = tile * BLOCK + r;
            if (q >= p.Lq) continue;
            const tokens_f32x4 v = add_sums<Geo::SUM, WS>(sums, r, at);
            raw_t *drow = (raw_t *)p.dq + (int64_t)b * p.dqs[0] + (int64_t)h * p.dqs[1] + (int64_t)q * p.dqs[2];
            store4<T>(drow, at, p.D, vec, v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
        }
    }
}

template <typename T, int DP, bool DROP, int WS>
__global__ __launch_bounds__(256, DP > (T::bytes == 4 ? 32 : 64) ? 1 : 2) void attention_backward_kv(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef BwdGeo<T, DP, WS, true> Geo;
    constexpr bool FEW = Geo::FEW;
    constexpr int ROWS = Geo::ROWS, BLOCK = Geo::BLOCK, NT = FEW ? 64 : 256;
    extern __shared__ __align__(16) unsigned char smem[];
    float *stats = (float *)(smem + Geo::tile_bytes);          // row_stats of each copy of a tile
    unsigned char *masks = (unsigned char *)(stats + Geo::copies * kRowStats);   // [wave][4][32]
    float *lut = (float *)(masks + 512);
    float *diagonals = lut + (p.lut + 3) / 4 * 4;    // [wave][kDiagonal]
    float *near = diagonals + (p.part ? 4 * kDiagonal : 0);   // [wave][lut]
    float *far = near + (p.part ? 4 * p.lut : 0);    // [wave][2]
    uint16_t *starts = (uint16_t *)(far + 8);
    __shared__ int large;                            // a head's table holds a bias that row_shift is for

    int unit, tile, part;
    if (!block_place(p, false, 1, unit, tile, part)) return;
    const int b = unit / p.Hkv, hk = unit - b * p.Hkv;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int len = sequence_length(p, b);
    const int first = p.from_end ? len - p.Lq : p.first;
    const int rg = wave % (4 / WS), wp = wave / (4 / WS);   // the wave's 32 rows, its part of the queries
    const int block0 = tile * BLOCK, k0 = block0 + rg * 32;
    const int key = k0 + (lane & 31);
    const bool vec = p.vec, live = key < len;

    const raw_t *krow =
        (const raw_t *)p.k + (int64_t)b * p.ks[0] + (int64_t)hk * p.ks[1] + (int64_t)key * p.ks[2];
    const raw_t *vrow =
        (const raw_t *)p.v + (int64_t)b * p.vs[0] + (int64_t)hk * p.vs[1] + (int64_t)key * p.vs[2];
    Frag<T> kf[DP / 16], vf[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        kf[s] = frag_global<T>(krow, 16 * s + 8 * half, p.D, live, vec);
        vf[s] = frag_global<T>(vrow, 16 * s + 8 * half, p.D, live, vec);
    }
    f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) dk[d][r] = dv[d][r] = 0.0f;
    if (p.lut)
        for (int i = t; i < p.side; i += 256) starts[i] = p.starts[i];

    // queries before q_first see no key of this block, and stay out of its products
    // (they may hold NaN: queries before a sequence's first token); the block's part
    // is a range of the (head, query tile) pairs that are left
    const int q_first = p.causal ? max(0, block0 - first) : 0, q_begin = q_first / ROWS * ROWS;
    const int q_tiles = block0 < len && q_begin < p.Lq ? (p.Lq - q_begin + ROWS - 1) / ROWS : 0;
    const int64_t pairs = (int64_t)p.G * q_tiles;
    const int64_t p0 = pairs * part / p.splits, p1 = pairs * (part + 1) / p.splits;
    const int tt = FEW ? lane : t;
    raw_t *Qt = (raw_t *)smem + (FEW ? wave * Geo::bufs * 2 * Geo::tile_elems : 0);
    if (FEW) stats += wave * Geo::bufs * kRowStats;
    unsigned char *mask = masks + wave * 128;
    float *diagonal = diagonals + wave * kDiagonal + 32, *mine = near + wave * p.lut;
    if (t == 0) large = 0;
    if (p.part)
        for (int i = t; i < 4 * kDiagonal; i += 256) diagonals[i] = 0.0f;

    for (int g = 0; g < p.G; ++g) {
        const int64_t base = (int64_t)g * q_tiles;
        const int t0 = (int)max(p0 - base, (int64_t)0), t1 = (int)min(p1 - base, (int64_t)q_tiles);
        const int h = hk * p.G + g, bh = b * p.H + h;
        float *sums_out =
            p.part ? p.part + ((((int64_t)h * p.B + b) * p.tiles + tile) * p.splits + part) * p.buckets : nullptr;
        if (t0 >= t1) {
            if (p.part)
                for (int n = t; n < p.buckets; n += 256) sums_out[n] = 0.0f;
            continue;
        }
        const raw_t *qb = (const raw_t *)p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1];
        const raw_t *gb = (const raw_t *)p.d_o + (int64_t)b * p.dos[0] + (int64_t)h * p.dos[1];
        __syncthreads();
        float far_lo = 0.0f, far_hi = 0.0f;          // sums of distances past the last change
        bool shifted = false;
        if (p.lut) {
            if (fill_lut<T>(p, h, lut, starts, t, 256)) large = 1;
            if (p.part)
                for (int i = t; i < 4 * p.lut; i += 256) near[i] = 0.0f;
            __syncthreads();
            shifted = __builtin_amdgcn_readfirstlane(large);
        }
        const auto load = [&](int copy, int q0) {
            raw_t *to = Qt + copy * 2 * Geo::tile_elems;
            if (tt < 64) copy_rows(stats + copy * kRowStats, row_stats(p, bh, q0 >> 6), tt);
            copy_tile<T, DP, ROWS, NT, true>(to, qb, p.qs[2], q0, p.Lq, p.D, p.async, vec, tt, q_first);
            copy_tile<T, DP, ROWS, NT, true>(to + Geo::tile_elems, gb, p.dos[2], q0, p.Lq, p.D, p.async, vec, tt, q_first);
        };
        constexpr int STEP = FEW ? 4 : 1;
        const int begin = FEW ? t0 + wave : t0;
        if (begin < t1) load(0, q_begin + begin * ROWS);
        for (int n = begin, it = 0; n < t1; n += STEP, ++it) {
            const int q0 = q_begin + n * ROWS, copy = Geo::bufs == 2 ? it & 1 : 0;
            const raw_t *Qs = Qt + copy * 2 * Geo::tile_elems, *Gs = Qs + Geo::tile_elems;
            const float *rs = stats + copy * kRowStats + (q0 & 63);
            async_wait();
            tile_sync<FEW>();
            const bool more = n + STEP < t1;
            if (Geo::bufs == 2 && more) load((it + 1) & 1, q0 + STEP * ROWS);
#pragma unroll
            for (int u = 0; u < ROWS / 32; ++u) {
                const int qu = q0 + 32 * u;          // this 32-query part
                if (k0 >= len || qu >= p.Lq || (p.causal && first + qu + 31 < k0)) continue;
                f32x16 st, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) st[r] = dp[r] = 0.0f;
                const int row = 32 * u + a_row(lane & 31);
                pipelined<T, 2 * (DP / 16), T::bytes == 4 ? 1 : 4>(
                    [&](int i) { return frag_lds<T, DP>(i & 1 ? Gs : Qs, row, 8 * (i & ~1) + 8 * half); },
                    [&](int i, const Frag<T> &a) {
                        if (step_counts<T>(p, i >> 1)) mma<T>(i & 1 ? dp : st, a, i & 1 ? vf[i >> 1] : kf[i >> 1]);
                    });
                if constexpr (DROP) {
                    // this lane's two calls: query qu + lane % 32, keys
                    // k0 + 16 half .. + 15; one byte of kept bits each
                    tile_sync<true>();
#pragma unroll
                    for (int n2 = 0; n2 < 2; ++n2) {
                        const int oct = 2 * half + n2;
                        const u32x4 rnd = philox((uint32_t)(k0 >> 3) + oct, (uint32_t)(qu + (lane & 31)),
                                                 (uint32_t)bh, p.call, p.seed_lo, p.seed_hi);
                        mask[oct * 32 + (lane & 31)] = (unsigned char)kept_byte(rnd, (p.threshold - 1) * 0x10001u);
                    }
                    tile_sync<true>();
                }
                const int cls = bias_class(p, k0 - (first + qu + 31), k0 + 31 - (first + qu));
                const bool edge = k0 + 32 > len || (p.causal && first + qu < k0 + 31);
                Frag<T> pf[2], df[2];                // P and dS in the type of dO and Q
                float all[16];                       // dS
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r0 = 32 * u + 16 * x + 8 * half;   // this lane's eight queries
                    const float *ml = rs + (cls == 1 ? 64 : cls == 2 ? 128 : 0) + r0;
                    const float *dl = rs + 192 + r0;
                    float pd[8], *ds = all + 8 * x;
                    if (cls == 0) {
                        float bias[8];
                        read_all<8>(lut + (key - first - q0 - r0 + p.border + kLutPad), bias,
                                    [](int j) { return -j; });
                        if (__builtin_expect(shifted, 0)) {
                            rare<8>(bias);
                            const float *shift = row_shifts(p, bh) + q0 + r0;
#pragma unroll
                            for (int j = 0; j < 8; ++j) bias[j] -= shift[j];
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j) pd[j] = fmaf(st[8 * x + j], p.scale2, bias[j]) + ml[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) pd[j] = fmaf(st[8 * x + j], p.scale2, ml[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) pd[j] = __builtin_amdgcn_exp2f(pd[j]);
                    if constexpr (DROP) {
                        u32x2 bits = *(const u32x2 *)(mask + ((lane & 31) >> 3) * 32 + 16 * x + 8 * half);
                        bits = (bits >> (uint32_t)(lane & 7)) & 0x01010101u;
                        const float keep[8] = {byte_float<0>(bits[0]), byte_float<1>(bits[0]), byte_float<2>(bits[0]),
                                               byte_float<3>(bits[0]), byte_float<0>(bits[1]), byte_float<1>(bits[1]),
                                               byte_float<2>(bits[1]), byte_float<3>(bits[1])};
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            ds[j] = pd[j] * fmaf(dp[8 * x + j], keep[j], -dl[j]);
                            pd[j] *= keep[j];
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) ds[j] = pd[j] * (dp[8 * x + j] - dl[j]);
                    }
                    if (edge) {
                        rare<8>(pd);
                        rare<8>(ds);
                        const int hidden = p.causal ? key - (first + q0 + r0) : 0;   // queries before the key
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (!live || j < hidden) pd[j] = ds[j] = 0.0f;
                        if (key == 0)                // queries that see no other key: dS is 0
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                if (len == 1 || (p.causal && first + q0 + r0 + j == 0)) ds[j] = 0.0f;
                    }
                    pf[x] = frag_pack<T>(pd);
                    df[x] = frag_pack<T>(ds);
                }
                if (p.part) {
                    if (cls == 0) {
                        float *to = diagonal + (lane & 31) * kDiagonalRow + 8 * half;
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *(tokens_f32x4 *)(to + 16 * (i >> 3) + (i & 7)) =
                                tokens_f32x4{all[i], all[i + 1], all[i + 2], all[i + 3]};
                        tile_sync<true>();
                        float v[32];
                        read_all<32>(diagonal + lane - 31, v, [](int i) { return (kDiagonalRow + 1) * i; });
                        float sum[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                        for (int i = 4; i < 32; ++i) sum[i & 3] += v[i];
                        // one entry a lane; a wave's additions keep their order, and nothing waits for them
                        __hip_atomic_fetch_add(mine + (k0 - first - qu + 31 - lane + p.border + kLutPad),
                                               (sum[0] + sum[1]) + (sum[2] + sum[3]), __ATOMIC_RELAXED,
                                               __HIP_MEMORY_SCOPE_WORKGROUP);
                        tile_sync<true>();
                    } else {
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; i += 4) sum += (all[i] + all[i + 1]) + (all[i + 2] + all[i + 3]);
                        if (cls == 1) far_lo += sum;
                        else far_hi += sum;
                    }
                }
                // i: (16 queries, 32 columns, dV or dK)
                pipelined<T, 4 * (DP / 32), T::bytes == 4 ? 1 : 4>(
                    [&](int i) {
                        return frag_lds_transposed<T, DP>(i & 1 ? Qs : Gs, 32 * u + 16 * (i / (DP / 16)),
                                                          32 * (i / 2 % (DP / 32)), lane);
                    },
                    [&](int i, const Frag<T> &a) {
                        mma<T>(i & 1 ? dk[i / 2 % (DP / 32)] : dv[i / 2 % (DP / 32)], a,
                               i & 1 ? df[i / (DP / 16)] : pf[i / (DP / 16)]);
                    });
            }
            if (Geo::bufs == 1 && more) {
                tile_sync<true>();
                load(0, q0 + STEP * ROWS);
            }
        }
        if (p.part) {
            far_lo = wave_sum(far_lo);
            far_hi = wave_sum(far_hi);
            if (lane == 0) {
                far[wave * 2] = far_lo;
                far[wave * 2 + 1] = far_hi;
            }
            __syncthreads();
            for (int i = t; i < p.lut; i += 256)
                near[i] = (near[i] + near[p.lut + i]) + (near[2 * p.lut + i] + near[3 * p.lut + i]);
            __syncthreads();
            // bucket n of a side holds distances starts[n] .. starts[n + 1] - 1, the
            // last one all that follow.  Without the other side a key after the query
            // counts as distance 0.  Eight lanes a bucket: the last ones are long.
            const float *zero = near + p.border + kLutPad;   // of distance 0
            for (int n0 = 0; n0 < p.buckets; n0 += 32) {
                const int n = n0 + (t >> 3), e = t & 7;
                const bool after = n >= p.side;              // the side of keys after the query
                const int m = after ? n - p.side : n;
                const bool last = m == p.side - 1, in = n < p.buckets;
                float sum = 0.0f;
                if (in) {
                    const int lo = max((int)starts[m], after ? 1 : 0), hi = last ? p.border + kLutPad + 1 : starts[m + 1];
                    for (int d = lo + e; d < hi; d += 8) sum += zero[after ? d : -d];
                    if (!p.bidirectional && m == 0)
                        for (int d = 1 + e; d <= kLutPad; d += 8) sum += zero[d];
                }
#pragma unroll
                for (int s = 1; s < 8; s <<= 1) sum += __shfl_xor(sum, s);
                if (!in || e) continue;
                if (last)
                    for (int w = 0; w < 4; ++w) sum += far[2 * w + (after ? 1 : 0)];
                if (!p.bidirectional && m == 0)
                    for (int w = 0; w < 4; ++w) sum += far[2 * w + 1];
                sums_out[n] = sum * p.rest;
            }
        }
    }
    const float sk = p.scale * p.rest, sv = p.rest;
    if constexpr (WS > 1) {
        float *sums = (float *)smem;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
            put_sums<DP, Geo::SUM>(sums, which ? dv : dk, wp * BLOCK + rg * 32, lane);
            __syncthreads();
            const float scale = which ? sv : sk;
            const int64_t *s = which ? p.dvs : p.dks;
            raw_t *to = (raw_t *)(which ? p.dv : p.dk) + (int64_t)b * s[0] + (int64_t)hk * s[1];
            for (int i = t; i < BLOCK * (DP / 4); i += 256) {
                const int r = i / (DP / 4), at = (i - r * (DP / 4)) * 4, row = block0 + r;
                if (row >= p.Lk) continue;
                const tokens_f32x4 v = add_sums<Geo::SUM, WS>(sums, r, at);
                if (p.splits > 1) {
                    const int dr = split_row(p.D);
                    if (at < p.D)
                        *(tokens_f32x4 *)(p.split + ((((int64_t)part * p.units + unit) * p.Lk + row) * 2 + which) * dr + at) = v;
                    continue;
                }
                store4<T>(to + (int64_t)row * s[2], at, p.D, vec, v[0] * scale, v[1] * scale, v[2] * scale,
                          v[3] * scale);
            }
        }
    } else {
        if (key >= p.Lk) return;
        if (p.splits > 1) {
            // this part's sums: (part, b, hk, key), dK then dV
            const int dr = split_row(p.D);
            float *out = p.split + (((int64_t)part * p.units + unit) * p.Lk + key) * 2 * dr;
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int col = 32 * d + 2 * r + 4 * half;
                    if (col >= p.D) continue;
                    *(tokens_f32x4 *)(out + col) = tokens_f32x4{dk[d][r], dk[d][r + 1], dk[d][r + 2], dk[d][r + 3]};
                    *(tokens_f32x4 *)(out + dr + col) =
                        tokens_f32x4{dv[d][r], dv[d][r + 1], dv[d][r + 2], dv[d][r + 3]};
                }
            return;
        }
        raw_t *dkrow = (raw_t *)p.dk + (int64_t)b * p.dks[0] + (int64_t)hk * p.dks[1] + (int64_t)key * p.dks[2];
        raw_t *dvrow = (raw_t *)p.dv + (int64_t)b * p.dvs[0] + (int64_t)hk * p.dvs[1] + (int64_t)key * p.dvs[2];
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int col = 32 * d + 2 * r + 4 * half;
                store4<T>(dkrow, col, p.D, vec, dk[d][r] * sk, dk[d][r + 1] * sk, dk[d][r + 2] * sk,
                          dk[d][r + 3] * sk);
                store4<T>(dvrow, col, p.D, vec, dv[d][r] * sv, dv[d][r + 1] * sv, dv[d][r + 2] * sv,
                          dv[d][r + 3] * sv);
            }
    }
}

// What is left once the sums of all blocks are there.  The first blocks, one a
// head and bucket, make dtable[n][h]: the sums of one head over sequences, key
// tiles and parts, in double.  The others add the parts of dK and dV in their
// order, a thread four columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void attention_backward_finish(AttnParams p) {
    typedef typename T::raw_t raw_t;
    const int tables = p.dtable ? p.buckets * p.H : 0;
    if ((int)blockIdx.x < tables) {
        __shared__ double red[4];
        const int n = blockIdx.x % p.buckets, h = blockIdx.x / p.buckets, t = threadIdx.x;
        const int64_t rows = (int64_t)p.B * p.tiles * p.splits;
        const float *part = p.part + (int64_t)h * rows * p.buckets + n;
        double sum = 0.0;
        for (int64_t r = t; r < rows; r += 256) sum += (double)part[r * p.buckets];
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) sum += __shfl_xor(sum, s);
        if ((t & 63) == 0) red[t >> 6] = sum;
        __syncthreads();
        if (t != 0) return;
        const float v = (float)((red[0] + red[1]) + (red[2] + red[3]));
        const int64_t at = (int64_t)n * p.H + h;
        if (p.table_f32) ((float *)p.dtable)[at] = v;
        else ((typename T::raw_t *)p.dtable)[at] = to_bits<T>(v);
        return;
    }
    const int dr = split_row(p.D), quads = 2 * dr / 4;
    const int64_t rows = (int64_t)p.units * p.Lk, i = (int64_t)(blockIdx.x - tables) * 256 + threadIdx.x;
    const int64_t row = i / quads;
    if (row >= rows) return;
    const int at = (int)(i - row * quads) * 4;
    tokens_f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; ++s) v += *(const tokens_f32x4 *)(p.split + (s * rows + row) * 2 * dr + at);
    const bool second = at >= dr;
    const float scale = second ? p.rest : p.scale * p.rest;
    const int64_t unit = row / p.Lk, key = row - unit * p.Lk, b = unit / p.Hkv, hk = unit - b * p.Hkv;
    const int64_t *st = second ? p.dvs : p.dks;
    raw_t *to = (raw_t *)(second ? p.dv : p.dk) + b * st[0] + hk * st[1] + key * st[2];
    store4<T>(to, second ? at - dr : at, p.D, p.vec, v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
}

template <typename T, int DP, int WS>
int q_lds(const AttnParams &p) {
    return BwdGeo<T, DP, WS, false>::tile_bytes + (p.lut + 3) / 4 * 16 + p.side * 2;
}

template <typename T, int DP, int WS>
int kv_lds(const AttnParams &p, bool table) {
    typedef BwdGeo<T, DP, WS, true> Geo;
    return Geo::tile_bytes + Geo::copies * kRowStats * 4 + 512 + (p.lut + 3) / 4 * 16 +
           (table ? 4 * (kDiagonal + p.lut) * 4 : 0) + 32 + p.side * 2;
}

int launch(void (*fn)(AttnParams), const AttnParams &p, int smem, hipStream_t stream) {
    if (smem > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != hipSuccess) return (int)e;
    }
    hipLaunchKernelGGL(fn, dim3((p.nblocks + 7) / 8 * 8), dim3(256), smem, stream, p);
    return (int)hipGetLastError();
}

void take_plan(AttnParams &p, const AttnPlan &a) {
    p.splits = a.splits;
    p.tiles = a.tiles;
    p.units = a.units;
    p.nblocks = a.units * a.tiles * a.splits;
}

template <typename T, int DP, int WS>
int launch_q(const AttnParams &p, hipStream_t stream) {
    return launch(p.threshold ? attention_backward_q<T, DP, true, WS> : attention_backward_q<T, DP, false, WS>, p,
                  q_lds<T, DP, WS>(p), stream);
}

template <typename T, int DP, int WS>
int launch_kv(const AttnParams &p, hipStream_t stream) {
    return launch(p.threshold ? attention_backward_kv<T, DP, true, WS> : attention_backward_kv<T, DP, false, WS>, p,
                  kv_lds<T, DP, WS>(p, p.part != nullptr), stream);
}

template <typename T, int DP>
int launch_dp(const AttnParams &p0, int dtype, hipStream_t stream) {
    AttnParams p = p0;
    AttnPlan a = plan_backward_q(p, dtype);
    take_plan(p, a);
    if (p.nblocks > 0) {
        if (const int e = a.ways == 4 ? launch_q<T, DP, 4>(p, stream) : launch_q<T, DP, 1>(p, stream)) return e;
    }
    a = plan_backward_kv(p, dtype);
    take_plan(p, a);
    if (p.nblocks > 0) {
        if (const int e = a.ways == 4 ? launch_kv<T, DP, 4>(p, stream) : launch_kv<T, DP, 1>(p, stream)) return e;
    }
    const int64_t tables = p.dtable ? (int64_t)p.buckets * p.H : 0;
    const int64_t threads = p.nblocks > 0 && p.splits > 1 ? (int64_t)p.units * p.Lk * (split_row(p.D) / 2) : 0;
    const int64_t blocks = tables + (threads + 255) / 256;
    if (blocks == 0) return 0;
    hipLaunchKernelGGL(attention_backward_finish<T>, dim3((unsigned)blocks), dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int launch_t(const AttnParams &p, int dtype, hipStream_t stream) {
    const int dp = padded_dim(p.D);
    if (dp == 32) return launch_dp<T, 32>(p, dtype, stream);
    if (dp == 64) return launch_dp<T, 64>(p, dtype, stream);
    if (dp == 96) return launch_dp<T, 96>(p, dtype, stream);
    return launch_dp<T, 128>(p, dtype, stream);
}

// LDS of the 32-row form of the dK / dV kernel.
int few_kv_lds(const AttnParams &p, int dtype) {
    const int dp = padded_dim(p.D);
    const bool table = p.buckets > 0;
    if (dtype == 0)
        return dp == 32   ? kv_lds<F32, 32, 4>(p, table)
               : dp == 64 ? kv_lds<F32, 64, 4>(p, table)
               : dp == 96 ? kv_lds<F32, 96, 4>(p, table)
                          : kv_lds<F32, 128, 4>(p, table);
    return dp == 32   ? kv_lds<F16, 32, 4>(p, table)
           : dp == 64 ? kv_lds<F16, 64, 4>(p, table)
           : dp == 96 ? kv_lds<F16, 96, 4>(p, table)
                      : kv_lds<F16, 128, 4>(p, table);
}

}  // namespace

// 32-row blocks where 128-row blocks would leave compute units without one: 512
// blocks of 2048 x 64 causal take 78 us, as 32-row blocks 90 us.
AttnPlan plan_backward_q(const AttnParams &p, int) {
    AttnPlan a = {};
    a.splits = 1;
    a.units = p.B * p.H;
    const int64_t full = (int64_t)a.units * ((p.Lq + kAttnRows - 1) / kAttnRows);
    a.ways = full < 256 ? 4 : 1;
    a.tiles = (p.Lq + kAttnRows / a.ways - 1) / (kAttnRows / a.ways);
    return a;
}

// Where the blocks are too few, parts of the (head, query tile) pairs go to
// blocks of their own, as long as a wave keeps a tile: as many as run at once,
// one a compute unit where registers or LDS allow no two.  16 heads of 4096
// queries on four key heads of 128 columns: the backward pass takes 616 us with
// 2 parts, 660 with 6, 969 with one.
AttnPlan plan_backward_kv(const AttnParams &p, int dtype) {
    AttnPlan a = {};
    a.splits = 1;
    a.units = p.B * p.Hkv;
    const int64_t full = (int64_t)a.units * ((p.Lk + kAttnRows - 1) / kAttnRows);
    a.ways = full < 64 && few_kv_lds(p, dtype) <= kMaxLds ? 4 : 1;
    a.tiles = (p.Lk + kAttnRows / a.ways - 1) / (kAttnRows / a.ways);
    const int64_t blocks = (int64_t)a.units * a.tiles, tile = a.ways == 4 ? 32 : 64;
    const int64_t room = (padded_dim(p.D) > (dtype == 0 ? 32 : 64) ? 256 : 512);
    if (blocks == 0 || 2 * blocks > room) return a;
    const int64_t pairs = (int64_t)p.G * ((p.Lq + tile - 1) / tile);
    int64_t splits = room / blocks;
    if (splits > pairs / (a.ways == 4 ? 4 : 8)) splits = pairs / (a.ways == 4 ? 4 : 8);
    if (splits <= 1) return a;
    a.splits = (int)splits;
    a.split_floats = splits * a.units * p.Lk * 2 * split_row(p.D);
    return a;
}

int launch_attention_backward(const AttnParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return launch_t<F32>(p, dtype, stream);
    if (dtype == 1) return launch_t<F16>(p, dtype, stream);
    return launch_t<BF16>(p, dtype, stream);
}

}  // namespace gs
