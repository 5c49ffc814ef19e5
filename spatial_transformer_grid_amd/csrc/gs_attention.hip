// gs_attention.hip -- attention with a relative position bias, forward.
//
// One pass over the keys with a running maximum m and sum l per query
// (softmax is unchanged when a constant leaves every score): scores of a key
// tile, m' = max(m, scores), O and l scaled by 2^(m - m'), then O += P V.
// Scores are kept in base 2 (scale and bias times log2 e).
//
// A wave owns 32 queries.  It computes S^T = K Q^T, so a lane holds one
// query's scores: the softmax needs no exchange but one with lane + 32, and
// the probabilities are already the B operand of O^T += V^T P^T (a_row).
//
// Two forms.  Where 128-query blocks fill the chip, the four waves of a block
// share each tile of keys, two buffers deep.  Where they do not, a block has 32
// queries and its waves take every fourth key tile, each into LDS of its own
// without block barriers, and add up at the end; if that is still too few
// blocks, the key axis is also split over blocks and attention_combine joins
// them.  There the rows may be the queries of all the heads that share a key
// head, so that the cache is read once.
//
// Bound by vector arithmetic beside the products (an exponential, two products
// and two sums a score, and with dropout a twelfth of a generator call), at 128
// columns by the products themselves.  Measured: 16 x 4096 x 4096 x 128 fp16
// with a bias 172 us (800 TFLOP/s, where an 8192^3 product reaches 1093);
// 2 x 16 x 2048 x 64 causal bf16 with bias and dropout 57 to 61 us, 45 us without
// dropout, 40 us without either; 16 caches of up to 8192 keys x 8 heads x 128
// bf16, one query each: 72 us (4.8 TB/s, memory) and 5 us for the join.
#include "gs_tokens.hpp"

namespace gs {

namespace {

// WS: into how many parts (1 or 4) the waves of a block split the keys; a block
// has 128 / WS rows.
template <typename T, int DP, int WS>
struct FwdGeo {
    static constexpr bool FEW = WS == 4;
    static constexpr int ROWS = kAttnRows / WS;
    static constexpr int KEYS = FEW || T::bytes == 4 ? 32 : 64;   // keys of an LDS tile
    static constexpr int U = KEYS / 32;
    static constexpr int tile_elems = KEYS * DP;
    static constexpr int SUM = DP + 4;                            // floats of a row of a wave's O
    // two buffers of K and V, a block's or each wave's own (one, where two would
    // leave a compute unit with one block); the waves' O takes their place
    static constexpr int bufs = FEW && DP * T::bytes > 128 ? 1 : 2;
    static constexpr int tile_bytes = (FEW ? 4 : 1) * bufs * 2 * tile_elems * T::bytes;
    static constexpr int fixed_bytes = WS > 1 && 128 * SUM * 4 > tile_bytes ? 128 * SUM * 4 : tile_bytes;
};

// A new maximum is taken up only where a score passes the old one by more than
// this (base 2): the probabilities then stay below 2^kSlack, far from the
// largest fp16 value, and O is not scaled again with each small step.
constexpr float kSlack = 8.0f;

// What a part of the keys with maximum m counts under the common maximum.  Where
// no part has one, a row's scores are all -inf (sums 0) or all NaN (a maximum
// leaves NaN out, a sum does not): the sums count as they are, so that NaN stays.
__device__ __forceinline__ float part_weight(float m, float common) {
    return common == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - common);
}

template <typename T, int DP, bool DROP, int WS>
__global__ __launch_bounds__(256, T::bytes == 4 && DP > 64 ? 1 : 2) void attention_forward(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef FwdGeo<T, DP, WS> Geo;
    constexpr bool FEW = Geo::FEW;
    constexpr int KEYS = Geo::KEYS, U = Geo::U, ROWS = Geo::ROWS, NT = FEW ? 64 : 256;
    extern __shared__ __align__(16) unsigned char smem[];
    float *luts = (float *)(smem + Geo::fixed_bytes);
    __shared__ float stat[WS][2][ROWS];              // maximum and sum of each part
    __shared__ float shifts[ROWS];                   // row_shift of each row, where `shifted`
    __shared__ int large;                            // the table holds a bias that row_shift is for

    int unit, tile, part;
    if (!block_place(p, true, FEW && p.pack ? 1 : p.G, unit, tile, part)) return;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int rg = wave % (4 / WS), wp = wave / (4 / WS);   // the wave's 32 rows, its part of the keys
    // the lane's row: query qi of head h
    int b, h, hk, g = 0, qi, rows;
    const int row0 = tile * ROWS + rg * 32, row = row0 + (lane & 31);
    if (FEW && p.pack) {
        b = unit / p.Hkv;
        hk = unit - b * p.Hkv;
        rows = p.G * p.Lq;
        g = row < rows ? row / p.Lq : 0;
        qi = row < rows ? row - g * p.Lq : 0;
        h = hk * p.G + g;
    } else {
        b = unit / p.H;
        h = unit - b * p.H;
        hk = h / p.G;
        rows = p.Lq;
        qi = row;
    }
    const bool live = row < rows;
    const int len = sequence_length(p, b);
    const int first = p.from_end ? len - p.Lq : p.first;
    const int pos = first + qi;
    // positions of the wave's rows, and the last one of the block's
    const int wave_first = FEW && p.pack ? first : first + row0;
    const int wave_last = FEW && p.pack ? first + p.Lq - 1 : wave_first + 31;
    const int block_last =
        FEW && p.pack ? wave_last : first + min((tile + 1) * ROWS, p.Lq) - 1;
    const int end = min(p.causal ? min(len, block_last + 1) : len, FEW ? (part + 1) * p.chunk : len);
    const int begin = FEW ? part * p.chunk + wave * KEYS : 0;
    constexpr int STEP = FEW ? 4 * KEYS : KEYS;
    const bool vec = p.vec;

    const raw_t *kb = (const raw_t *)p.k + (int64_t)b * p.ks[0] + (int64_t)hk * p.ks[1];
    const raw_t *vb = (const raw_t *)p.v + (int64_t)b * p.vs[0] + (int64_t)hk * p.vs[1];
    const raw_t *qrow =
        (const raw_t *)p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)qi * p.qs[2];
    const int tt = FEW ? lane : t;
    raw_t *Kt = (raw_t *)smem + (FEW ? wave * Geo::bufs * 2 * Geo::tile_elems : 0);
    const auto load = [&](raw_t *to, int k0) {
        copy_tile<T, DP, KEYS, NT>(to, kb, p.ks[2], k0, end, p.D, p.async, vec, tt);
        copy_tile<T, DP, KEYS, NT>(to + Geo::tile_elems, vb, p.vs[2], k0, end, p.D, p.async, vec, tt);
    };
    if (begin < end) load(Kt, begin);
    // a negative scale moves into Q: the maximum of the scores is then that of the products
    const float scale2 = fabsf(p.scale2);
    Frag<T> qf[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
        qf[s] = frag_global<T>(qrow, 16 * s + 8 * half, p.D, live, vec);
        if (p.scale2 < 0.0f) frag_negate<T>(qf[s]);
    }
    const float *lut = luts;
    float bias_lo = 0.0f, bias_hi = 0.0f;
    bool shifted = false;
    const int col = rg * 32 + (lane & 31);           // the lane's row in the block
    if (p.lut) {
        if (t == 0) large = 0;
        const int heads = FEW && p.pack ? p.G : 1;
        uint16_t *starts = (uint16_t *)(luts + heads * p.lut);
        for (int i = t; i < p.side; i += 256) starts[i] = p.starts[i];
        __syncthreads();
        for (int i = 0; i < heads; ++i)
            if (fill_lut<T>(p, FEW && p.pack ? hk * p.G + i : h, luts + i * p.lut, starts, t, 256)) large = 1;
        __syncthreads();
        lut = luts + (FEW ? g * p.lut : 0);
        shifted = __builtin_amdgcn_readfirstlane(large);
        bias_lo = lut[0];
        bias_hi = lut[p.lut - 1];
        if (__builtin_expect(shifted, 0)) {
            const float shift = row_shift(p, lut, pos, p.causal ? min(len, pos + 1) : len);
            bias_lo -= shift;
            bias_hi -= shift;
            shifts[col] = shift;                     // (kept there: no register of the loop's)
            tile_sync<true>();
        }
    }

    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    const uint32_t below = (p.threshold - 1) * 0x10001u;

    for (int k0 = begin, n = 0; k0 < end; k0 += STEP, ++n) {
        const raw_t *Ks = Kt + (Geo::bufs == 2 ? (n & 1) * 2 * Geo::tile_elems : 0);
        const raw_t *Vs = Ks + Geo::tile_elems;
        async_wait();
        tile_sync<FEW>();
        const bool more = k0 + STEP < end;
        if (Geo::bufs == 2 && more) load(Kt + ((n + 1) & 1) * 2 * Geo::tile_elems, k0 + STEP);
        if (FEW || (row0 < p.Lq && !(p.causal && k0 > wave_last))) {
            float s[16 * U];
            f32x16 st[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) st[u][r] = 0.0f;
            pipelined<T, U * (DP / 16), T::bytes == 4 ? 1 : DP == 32 ? 2 : DP == 96 ? 3 : 4>(
                [&](int i) {
                    return frag_lds<T, DP>(Ks, 32 * (i % U) + a_row(lane & 31), 16 * (i / U) + 8 * half);
                },
                [&](int i, const Frag<T> &a) {
                    if (step_counts<T>(p, i / U)) mma<T>(st[i % U], a, qf[i / U]);
                });
            // the generator runs while the products do
            u32x4 rnd[2 * U];
            if constexpr (DROP)
#pragma unroll
                for (int x = 0; x < 2 * U; ++x) {
                    rnd[x] = philox((uint32_t)(k0 + 8 * half + 16 * x) >> 3, (uint32_t)qi, (uint32_t)(b * p.H + h),
                                    p.call, p.seed_lo, p.seed_hi);
                    if constexpr (T::bytes == 2)
#pragma unroll
                        for (int i = 0; i < 4; ++i) rnd[x][i] = kept_pair(rnd[x][i], below);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) s[16 * u + r] = st[u][r];
            // s[8 x + j]: key k0 + 16 x + 8 half + j of this lane's query, a score
            // once multiplied by mul, with c added
            const int key0 = k0 + 8 * half;
            float mul = scale2, c = 0.0f;
            const int cls = bias_class(p, k0 - wave_last, k0 + KEYS - 1 - wave_first);
            const bool edge = shifted || k0 + KEYS > end || (p.causal && k0 + KEYS - 1 > wave_first);
            if (cls == 1) c = bias_lo;
            if (cls == 2) c = bias_hi;
            // fp32 rounds every score before the maximum leaves it, so that the
            // largest one's probability is 1 exactly; elsewhere the probability's
            // own rounding hides the difference, but for a bias so large that the
            // maximum loses the products (`shifted`: keys masked by -1e9 before others)
            if (cls == 0 || edge || T::bytes == 4) {
                if (cls == 0) {
                    float bias[16 * U];
                    read_all<16 * U>(lut + (key0 - pos + p.border + kLutPad), bias,
                                     [](int i) { return 16 * (i >> 3) + (i & 7); });
                    if (__builtin_expect(shifted, 0)) {
                        rare<16 * U>(bias);
                        const float shift = *(volatile float *)(shifts + col);
#pragma unroll
                        for (int i = 0; i < 16 * U; ++i) bias[i] -= shift;
                    }
#pragma unroll
                    for (int i = 0; i < 16 * U; ++i) s[i] = fmaf(s[i], mul, bias[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16 * U; ++i) s[i] = fmaf(s[i], mul, c);
                }
                mul = 1.0f;
                c = 0.0f;
                if (edge) {
                    rare<16 * U>(s);
                    const int seen = (p.causal ? min(end, pos + 1) : end) - key0;
#pragma unroll
                    for (int i = 0; i < 16 * U; ++i)
                        if (16 * (i >> 3) + (i & 7) >= seen) s[i] = -INFINITY;
                }
            }
            float top = s[0];
#pragma unroll
            for (int i = 1; i < 16 * U; ++i) top = fmaxf(top, s[i]);
            top = fmaf(top, mul, c);
            top = fmaxf(top, other_half(top));
            if (__any(top > m + kSlack)) {
                const float next = fmaxf(m, top);
                const float alpha = next == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - next);
                m = next;
                l *= alpha;
#pragma unroll
                for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= alpha;
            }
            c -= m == -INFINITY ? 0.0f : m;
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 16 * U; ++i) {
                s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], mul, c));
                sum[i & 1] += s[i];
            }
            l += sum[0] + sum[1];
            // P in V's type: the matrix cores multiply two operands of one type.  Its sum
            // is of the unrounded P, whose roundings average out over the keys; lse keeps
            // fp32.  O's error is 1.4 times that of rounding O alone.
            Frag<T> pf[2 * U];
#pragma unroll
            for (int x = 0; x < 2 * U; ++x) {
                if constexpr (DROP && T::bytes == 4) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[8 * x + j] = kept(rnd[x], j, p.threshold) ? s[8 * x + j] : 0.0f;
                }
                pf[x] = frag_pack<T>(s + 8 * x);
                if constexpr (DROP && T::bytes == 2) frag_keep<T>(pf[x], rnd[x]);
            }
            pipelined<T, 2 * U * (DP / 32), T::bytes == 4 ? 1 : DP / 32>(
                [&](int i) { return frag_lds_transposed<T, DP>(Vs, 16 * (i / (DP / 32)), 32 * (i % (DP / 32)), lane); },
                [&](int i, const Frag<T> &a) { mma<T>(acc[i % (DP / 32)], a, pf[i / (DP / 32)]); });
        }
        if (Geo::bufs == 1 && more) {
            tile_sync<true>();
            load(Kt, k0 + STEP);
        }
    }
    l += __shfl_xor(l, 32);
    if constexpr (WS == 1) {
        if (!live) return;
        const float norm = l > 0.0f || l != l ? p.keep_scale / l : 0.0f;
        raw_t *orow = (raw_t *)p.o + (int64_t)b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)qi * p.os[2];
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                store4<T>(orow, 32 * d + 2 * r + 4 * half, p.D, vec, acc[d][r] * norm, acc[d][r + 1] * norm,
                          acc[d][r + 2] * norm, acc[d][r + 3] * norm);
        if (p.lse && half == 0)
            p.lse[(int64_t)unit * p.Lq + qi] =
                l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2 + (shifted ? natural(shifts[col]) : 0.0f);
    } else {
        // the parts' O and l under a common maximum, added in the order of the parts
        if (half == 0) {
            stat[wp][0][col] = m;
            stat[wp][1][col] = l;
        }
        __syncthreads();
        float all = stat[0][0][col];
#pragma unroll
        for (int w = 1; w < WS; ++w) all = fmaxf(all, stat[w][0][col]);
        const float alpha = all == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - all);
        float *sums = (float *)smem;
        float *mine = sums + (wp * ROWS + col) * Geo::SUM + 4 * half;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *(tokens_f32x4 *)(mine + 32 * d + 2 * r) = tokens_f32x4{acc[d][r] * alpha, acc[d][r + 1] * alpha,
                                                                       acc[d][r + 2] * alpha, acc[d][r + 3] * alpha};
        __syncthreads();
        for (int i = t; i < ROWS * (DP / 4); i += 256) {
            const int r = i / (DP / 4), at = (i - r * (DP / 4)) * 4;
            const int rr = tile * ROWS + r;
            if (rr >= rows || at >= p.D) continue;
            float big = stat[0][0][r], lr = 0.0f;
#pragma unroll
            for (int w = 1; w < WS; ++w) big = fmaxf(big, stat[w][0][r]);
#pragma unroll
            for (int w = 0; w < WS; ++w) lr = fmaf(stat[w][1][r], part_weight(stat[w][0][r], big), lr);
            tokens_f32x4 v = *(const tokens_f32x4 *)(sums + r * Geo::SUM + at);
#pragma unroll
            for (int w = 1; w < WS; ++w) v += *(const tokens_f32x4 *)(sums + (w * ROWS + r) * Geo::SUM + at);
            const int64_t flat = (int64_t)unit * rows + rr;       // (b, h, qi) in either order of the rows
            if (p.splits > 1) {
                const int64_t all_rows = (int64_t)p.B * p.H * p.Lq, dr = split_row(p.D);
                float *out = p.split + ((int64_t)part * all_rows + flat) * dr;
                *(tokens_f32x4 *)(out + at) = v;
                if (at == 0) {
                    float *st = p.split + (int64_t)p.splits * all_rows * dr + ((int64_t)part * all_rows + flat) * 2;
                    st[0] = big;
                    st[1] = lr;
                    if (p.lse && part == 0)                  // attention_combine adds the rest
                        p.lse[flat] = shifted ? natural(shifts[r]) : 0.0f;
                }
                continue;
            }
            const float norm = lr > 0.0f || lr != lr ? p.keep_scale / lr : 0.0f;
            const int64_t bh = flat / p.Lq;
            const int bb = (int)(bh / p.H), hh = (int)(bh - (int64_t)bb * p.H), q = (int)(flat - bh * p.Lq);
            raw_t *orow = (raw_t *)p.o + (int64_t)bb * p.os[0] + (int64_t)hh * p.os[1] + (int64_t)q * p.os[2];
            store4<T>(orow, at, p.D, vec, v[0] * norm, v[1] * norm, v[2] * norm, v[3] * norm);
            if (p.lse && at == 0)
                p.lse[flat] = lr == 0.0f ? -INFINITY
                                         : (big + __builtin_amdgcn_logf(lr)) * kLn2 + (shifted ? natural(shifts[r]) : 0.0f);
        }
    }
}

// O and lse from the parts of the key axis, a wave a row: the parts' O and
// sums under their common maximum, added in the order of the parts.
template <typename T>
__global__ __launch_bounds__(256) void attention_combine(AttnParams p) {
    typedef typename T::raw_t raw_t;
    const int64_t rows = (int64_t)p.B * p.H * p.Lq;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (r >= rows) return;
    const int lane = threadIdx.x & 63, dr = split_row(p.D);
    const float *st = p.split + (int64_t)p.splits * rows * dr;
    // a lane a part for the statistics
    float big = -INFINITY;
    for (int i = lane; i < p.splits; i += 64) big = fmaxf(big, st[(i * rows + r) * 2]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) big = fmaxf(big, __shfl_xor(big, x));
    float l = 0.0f, v[2] = {0.0f, 0.0f};
    const int c0 = lane < p.D ? lane : 0, c1 = lane + 64 < p.D ? lane + 64 : 0;
    for (int i0 = 0; i0 < p.splits; i0 += 64) {
        const int left = min(64, p.splits - i0);
        float w = 0.0f, mine = 0.0f;
        if (lane < left) {
            const int64_t at = ((i0 + lane) * rows + r) * 2;
            w = part_weight(st[at], big);
            mine = st[at + 1];
        }
        for (int i = 0; i < left; ++i) {
            const float wi = __shfl(w, i);
            const float *o = p.split + ((i0 + i) * rows + r) * dr;
            l = fmaf(__shfl(mine, i), wi, l);
            v[0] = fmaf(o[c0], wi, v[0]);
            v[1] = fmaf(o[c1], wi, v[1]);
        }
    }
    const float norm = l > 0.0f || l != l ? p.keep_scale / l : 0.0f;
    const int64_t bh = r / p.Lq;
    const int b = (int)(bh / p.H), h = (int)(bh - (int64_t)b * p.H), q = (int)(r - bh * p.Lq);
    raw_t *orow = (raw_t *)p.o + (int64_t)b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)q * p.os[2];
    if (lane < p.D) orow[lane] = to_bits<T>(v[0] * norm);
    if (lane + 64 < p.D) orow[lane + 64] = to_bits<T>(v[1] * norm);
    if (p.lse && lane == 0) p.lse[r] = l == 0.0f ? -INFINITY : (big + __builtin_amdgcn_logf(l)) * kLn2 + p.lse[r];
}

template <typename T, int DP, bool DROP, int WS>
int launch_form(const AttnParams &p, hipStream_t stream) {
    const int heads = p.pack ? p.G : 1;
    const int smem = FwdGeo<T, DP, WS>::fixed_bytes + heads * p.lut * 4 + (p.lut ? p.side * 2 : 0);
    const dim3 grid((p.nblocks + 7) / 8 * 8);
    void (*const fn)(AttnParams) = attention_forward<T, DP, DROP, WS>;
    if (smem > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != hipSuccess) return (int)e;
    }
    hipLaunchKernelGGL(fn, grid, dim3(256), smem, stream, p);
    return (int)hipGetLastError();
}

template <typename T, int DP, int WS>
int launch_ws(const AttnParams &p, hipStream_t stream) {
    return p.threshold ? launch_form<T, DP, true, WS>(p, stream) : launch_form<T, DP, false, WS>(p, stream);
}

template <typename T, int DP>
int launch_dp(const AttnParams &p, int ways, hipStream_t stream) {
    if (ways == 4) return launch_ws<T, DP, 4>(p, stream);
    return launch_ws<T, DP, 1>(p, stream);
}

template <typename T>
int launch_t(const AttnParams &p, int ways, hipStream_t stream) {
    const int dp = padded_dim(p.D);
    const int e = dp == 32   ? launch_dp<T, 32>(p, ways, stream)
                  : dp == 64 ? launch_dp<T, 64>(p, ways, stream)
                  : dp == 96 ? launch_dp<T, 96>(p, ways, stream)
                             : launch_dp<T, 128>(p, ways, stream);
    if (e || p.splits <= 1) return e;
    const int64_t rows = (int64_t)p.B * p.H * p.Lq;
    hipLaunchKernelGGL(attention_combine<T>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

}  // namespace

// The 32-row form where 128-row blocks would leave compute units without one,
// or would be mostly empty.  Decode of 16 ragged caches: 76 us, with 128-row
// blocks 189 us; 512 blocks of 2048 x 64 causal: 77 us, with 128-row blocks 60 us.
AttnPlan plan_forward(const AttnParams &p, int, bool workspace) {
    AttnPlan a = {};
    a.splits = 1;
    a.units = p.B * p.H;
    a.tiles = (p.Lq + kAttnRows - 1) / kAttnRows;
    a.chunk = p.Lk;
    const int64_t full = (int64_t)a.units * a.tiles;
    a.ways = p.Lq <= 32 || full < 256 ? 4 : 1;
    if (a.ways == 1) return a;
    // tables of all heads that share a key head take at most 16 KiB of LDS
    if (p.G > 1 && p.G * (int64_t)p.Lq <= 32 && (int64_t)p.G * p.lut * 4 <= 16384) {
        a.pack = 1;
        a.units = p.B * p.Hkv;
    }
    a.tiles = a.pack ? 1 : (p.Lq + 31) / 32;
    // two blocks a compute unit; more only repeat what a block does before its
    // first key (the ragged decode: 4 parts 71 us, 8 parts 80 us, 16 parts 91 us)
    const int64_t blocks = (int64_t)a.units * a.tiles;
    if (!workspace || blocks >= 256 || blocks == 0) return a;
    int64_t splits = 512 / blocks;
    if (splits > p.Lk / 256) splits = p.Lk / 256;    // two tiles a wave at least
    if (splits <= 1) return a;
    a.chunk = (int)(((p.Lk + splits - 1) / splits + 127) / 128 * 128);
    a.splits = (p.Lk + a.chunk - 1) / a.chunk;
    a.split_floats = (int64_t)a.splits * p.B * p.H * p.Lq * (split_row(p.D) + 2);
    return a;
}

int launch_attention(const AttnParams &p0, int dtype, hipStream_t stream) {
    AttnParams p = p0;
    const AttnPlan a = plan_forward(p, dtype, p.split != nullptr);
    p.pack = a.pack;
    p.splits = a.splits;
    p.chunk = a.chunk;
    p.tiles = a.tiles;
    p.units = a.units;
    p.nblocks = a.units * a.tiles * a.splits;
    if (dtype == 0) return launch_t<F32>(p, a.ways, stream);
    if (dtype == 1) return launch_t<F16>(p, a.ways, stream);
    return launch_t<BF16>(p, a.ways, stream);
}

}  // namespace gs
