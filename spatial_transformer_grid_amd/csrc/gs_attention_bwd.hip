// gs_attention_bwd.hip -- gradients of attention with a relative position bias.
//
// With P the probabilities, M the dropout's factors (0 or keep_scale) and
// delta_i = sum_j P_ij M_ij (dO_i . V_j) = dO_i . O_i:
//   dS_ij = P_ij (M_ij (dO_i . V_j) - delta_i),
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = (P M)^T dO,
//   dtable[n] = sum of dS_ij over the pairs whose distance is in bucket n.
// P is computed again from the scores and lse.  Two kernels: one per query
// tile (dQ, delta, the table's sums), one per key tile (dK, dV, over all
// query heads that share the key head).  Each output element has one writer
// and a fixed order of summation; the price is the scores and dO V^T twice,
// seven products in place of the five of a single pass that would add dQ with
// atomics, in an order that varies.
#include "gs_tokens.hpp"

namespace gs {

namespace {

constexpr int kKeys = 64;      // keys of an LDS tile (dQ)
constexpr int kRows = 64;      // queries of an LDS tile (dK, dV)

// Sums of dS by distance, per wave: one copy for each half of the wave, so
// that no two lanes of an instruction add to one address (the lanes of a half
// hold different queries and the same key, hence different distances).  An
// LDS add without return keeps the order of a wave's instructions, so the sums
// do not depend on timing.
__host__ __device__ constexpr int near_pitch(int lut) { return (lut + 31) / 64 * 64 + 32; }

template <typename T, int DP>
struct BwdGeo {
    static constexpr int PITCH = DP + 16 / T::bytes;
    static constexpr int tile_bytes = 2 * kKeys * PITCH * T::bytes;
};

__device__ __forceinline__ void lds_add(float *p, float v) {
    __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

template <typename T, int DP, bool DROP>
__global__ __launch_bounds__(256) void attention_backward_q(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef BwdGeo<T, DP> Geo;
    constexpr int PITCH = Geo::PITCH;
    extern __shared__ __align__(16) unsigned char smem[];
    raw_t *Ks = (raw_t *)smem;
    raw_t *Vs = Ks + kKeys * PITCH;
    float *lut = (float *)(smem + Geo::tile_bytes);
    const int pitch = near_pitch(p.lut);
    float *near = lut + (p.lut + 3) / 4 * 4;         // [wave][half][pitch]
    float *far = near + (p.lut ? 8 * pitch : 0);     // [wave][2]
    uint16_t *starts = (uint16_t *)(far + 8);

    const int lb = xcd_contiguous_block(p.nblocks);
    if (lb >= p.nblocks) return;
    int tile = lb % p.tiles;
    const int bh = lb / p.tiles;
    if (p.causal) tile = p.tiles - 1 - tile;
    const int b = bh / p.H, h = bh - b * p.H, hk = h / p.G;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int len = sequence_length(p, b);
    const int first = p.from_end ? len - p.Lq : p.first;
    const int q0 = tile * kAttnQueries + wave * 32;
    const int qi = q0 + (lane & 31);
    const int pos = first + qi;
    const int block_last = first + min((tile + 1) * kAttnQueries, p.Lq) - 1;
    const int end = p.causal ? min(len, block_last + 1) : len;
    const bool vec = p.vec, live = qi < p.Lq;

    const raw_t *kb = (const raw_t *)p.k + (int64_t)b * p.ks[0] + (int64_t)hk * p.ks[1];
    const raw_t *vb = (const raw_t *)p.v + (int64_t)b * p.vs[0] + (int64_t)hk * p.vs[1];
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
    float lse2 = INFINITY;                           // 2^(s - inf) = 0: no key seen
    if (live) {
        const int64_t at = (int64_t)bh * p.Lq + qi;
        const float v = p.lse[at];
        if (v != -INFINITY) lse2 = v * kLog2e;
        if (half == 0) p.delta[at] = delta;
    }
    if (p.lut) {
        fill_lut<T>(p, h, lut, starts, t, 256);
        for (int i = t; i < 8 * pitch; i += 256) near[i] = 0.0f;
    }
    float far_lo = 0.0f, far_hi = 0.0f;              // distances at or past the borders
    float *mine = near + (wave * 2 + half) * pitch;

    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

    TileCopy<T, DP, kKeys, 256, PITCH> copy;
    for (int k0 = 0; k0 < end; k0 += kKeys) {
        __syncthreads();
        copy.fetch(kb, p.ks[2], k0, end, p.D, vec, t);
        copy.put(Ks, t);
        copy.fetch(vb, p.vs[2], k0, end, p.D, vec, t);
        copy.put(Vs, t);
        __syncthreads();
        const int wave_first = first + q0, wave_last = wave_first + 31;
        if (q0 >= p.Lq) continue;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int ku = k0 + 32 * u;              // this 32-key part
            if (ku >= end || (p.causal && ku > wave_last)) continue;
            f32x16 st, dp;
#pragma unroll
            for (int r = 0; r < 16; ++r) st[r] = dp[r] = 0.0f;
            const int row = (32 * u + a_row(lane & 31)) * PITCH + 8 * half;
#pragma unroll
            for (int x = 0; x < DP / 16; ++x) {
                mma<T>(st, frag_lds<T>(Ks + row + 16 * x), qf[x]);
                mma<T>(dp, frag_lds<T>(Vs + row + 16 * x), gf[x]);
            }
            const int key0 = ku + 8 * half;
            float ds[16];
            const bool edge = ku + 32 > end || (p.causal && ku + 31 > wave_first);
            const int seen = p.causal ? min(end, pos + 1) : end;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                u32x4 rnd;
                if constexpr (DROP)
                    rnd = philox((uint32_t)(key0 + 16 * x) >> 3, (uint32_t)qi, (uint32_t)bh, p.call, p.seed_lo,
                                 p.seed_hi);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 8 * x + j, key = key0 + 16 * x + j;
                    float s = st[i] * p.scale2;
                    if (p.lut) s = fmaf(st[i], p.scale2, lut[lut_index(p, key - pos)]);
                    float e = __builtin_amdgcn_exp2f(s - lse2);
                    if (edge && key >= seen) e = 0.0f;
                    float g = dp[i];
                    if constexpr (DROP) g = kept(rnd, j, p.threshold) ? g * p.keep_scale : 0.0f;
                    ds[i] = e * (g - delta);
                }
            }
            if (p.lut) {
                const int rel_lo = ku - wave_last, rel_hi = ku + 31 - wave_first;
                float sum = 0.0f;
                if (rel_lo >= p.lut - p.border || rel_hi <= -p.border) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) sum += (ds[i] + ds[i + 1]) + (ds[i + 2] + ds[i + 3]);
                    if (rel_hi <= -p.border) far_lo += sum;
                    else far_hi += sum;
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int at = key0 + 16 * (i >> 3) + (i & 7) - pos + p.border;
                        if (at <= 0) far_lo += ds[i];
                        else if (at >= p.lut - (p.bidirectional ? 1 : 0)) far_hi += ds[i];
                        else lds_add(mine + at, ds[i]);
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Frag<T> df = frag_pack<T>(ds + 8 * x);
#pragma unroll
                for (int d = 0; d < DP / 32; ++d)
                    mma<T>(acc[d], frag_lds_transposed<T, PITCH>(Ks, 32 * u + 16 * x, 32 * d, lane), df);
            }
        }
    }
    if (live) {
        raw_t *drow = (raw_t *)p.dq + (int64_t)b * p.dqs[0] + (int64_t)h * p.dqs[1] + (int64_t)qi * p.dqs[2];
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                store4<T>(drow, 32 * d + 2 * r + 4 * half, p.D, vec, acc[d][r] * p.scale, acc[d][r + 1] * p.scale,
                          acc[d][r + 2] * p.scale, acc[d][r + 3] * p.scale);
    }
    if (!p.lut || !p.part) return;
    far_lo = wave_sum(far_lo);
    far_hi = wave_sum(far_hi);
    if (lane == 0) {
        far[wave * 2] = far_lo;
        far[wave * 2 + 1] = far_hi;
    }
    __syncthreads();
    // bucket n of a side holds distances starts[n] .. starts[n + 1] - 1; the
    // last one lies wholly in the far sums.  Without the other side a key
    // after the query counts as distance 0 (the far sum of that direction).
    float *out = p.part + (((int64_t)h * p.B + b) * p.tiles + tile) * p.buckets;
    for (int n = t; n < p.buckets; n += 256) {
        const bool after = n >= p.side;              // the side of keys after the query
        const int m = after ? n - p.side : n;
        float sum = 0.0f;
        if (m == p.side - 1) {
            for (int w = 0; w < 4; ++w) sum += far[2 * w + (after ? 1 : 0)];
        } else {
            for (int d = max((int)starts[m], after ? 1 : 0); d < (int)starts[m + 1]; ++d) {
                const int at = p.border + (after ? d : -d);
                for (int w = 0; w < 8; ++w) sum += near[w * pitch + at];
            }
        }
        if (!p.bidirectional && m == 0)
            for (int w = 0; w < 4; ++w) sum += far[2 * w + 1];
        out[n] = sum;
    }
}

template <typename T, int DP, bool DROP>
__global__ __launch_bounds__(256) void attention_backward_kv(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef BwdGeo<T, DP> Geo;
    constexpr int PITCH = Geo::PITCH;
    extern __shared__ __align__(16) unsigned char smem[];
    raw_t *Qs = (raw_t *)smem;
    raw_t *Gs = Qs + kRows * PITCH;
    float *lse2s = (float *)(smem + Geo::tile_bytes);
    float *deltas = lse2s + kRows;
    unsigned char *masks = (unsigned char *)(deltas + kRows);   // [wave][4][32]
    float *lut = (float *)(masks + 512);
    uint16_t *starts = (uint16_t *)(lut + (p.lut + 3) / 4 * 4);

    const int lb = xcd_contiguous_block(p.nblocks);
    if (lb >= p.nblocks) return;
    const int tile = lb % p.tiles;
    const int bk = lb / p.tiles;
    const int b = bk / p.Hkv, hk = bk - b * p.Hkv;
    const int t = threadIdx.x, lane = t & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int len = sequence_length(p, b);
    const int first = p.from_end ? len - p.Lq : p.first;
    const int k0 = tile * kAttnQueries + wave * 32;
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

    // queries before q_begin see no key of this block
    const int q_begin =
        p.causal ? max(0, tile * kAttnQueries - first) / kRows * kRows : 0;
    const int q_end = tile * kAttnQueries < len ? p.Lq : 0;
    TileCopy<T, DP, kRows, 256, PITCH> copy;
    for (int g = 0; g < p.G; ++g) {
        const int h = hk * p.G + g, bh = b * p.H + h;
        const raw_t *qb = (const raw_t *)p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1];
        const raw_t *gb = (const raw_t *)p.d_o + (int64_t)b * p.dos[0] + (int64_t)h * p.dos[1];
        if (p.lut) {
            __syncthreads();
            fill_lut<T>(p, h, lut, starts, t, 256);
        }
        for (int q0 = q_begin; q0 < q_end; q0 += kRows) {
            __syncthreads();
            copy.fetch(qb, p.qs[2], q0, p.Lq, p.D, vec, t);
            copy.put(Qs, t);
            copy.fetch(gb, p.dos[2], q0, p.Lq, p.D, vec, t);
            copy.put(Gs, t);
            if (t < kRows) {
                const int64_t at = (int64_t)bh * p.Lq + q0 + t;
                float e = INFINITY, d = 0.0f;
                if (q0 + t < p.Lq) {
                    const float v = p.lse[at];
                    if (v != -INFINITY) e = v * kLog2e;
                    d = p.delta[at];
                }
                lse2s[t] = e;
                deltas[t] = d;
            }
            __syncthreads();
            if (k0 >= len) continue;
#pragma unroll
            for (int u = 0; u < kRows / 32; ++u) {
                const int qu = q0 + 32 * u;          // this 32-query part
                if (qu >= p.Lq || (p.causal && first + qu + 31 < k0)) continue;
                f32x16 st, dp;
#pragma unroll
                for (int r = 0; r < 16; ++r) st[r] = dp[r] = 0.0f;
                const int row = (32 * u + a_row(lane & 31)) * PITCH + 8 * half;
#pragma unroll
                for (int x = 0; x < DP / 16; ++x) {
                    mma<T>(st, frag_lds<T>(Qs + row + 16 * x), kf[x]);
                    mma<T>(dp, frag_lds<T>(Gs + row + 16 * x), vf[x]);
                }
                unsigned char *mask = masks + wave * 128;
                if constexpr (DROP) {
                    // this lane's two calls: query qu + lane % 32, keys
                    // k0 + 16 half .. + 15; one byte of kept bits each
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int oct = 2 * half + n;
                        const u32x4 rnd = philox((uint32_t)(k0 >> 3) + oct, (uint32_t)(qu + (lane & 31)),
                                                 (uint32_t)bh, p.call, p.seed_lo, p.seed_hi);
                        uint32_t bits = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) bits |= kept(rnd, j, p.threshold) ? 1u << j : 0u;
                        mask[oct * 32 + (lane & 31)] = (unsigned char)bits;
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
                const bool edge = k0 + 32 > len || (p.causal && first + qu < k0 + 31);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r0 = 32 * u + 16 * x + 8 * half;   // this lane's eight queries
                    const int pos0 = first + q0 + r0;
                    u32x2 bits = {0, 0};
                    if constexpr (DROP)
                        bits = *(const u32x2 *)(mask + ((lane & 31) >> 3) * 32 + 16 * x + 8 * half);
                    float pd[8], ds[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int i = 8 * x + j;
                        float s = st[i] * p.scale2;
                        if (p.lut) s = fmaf(st[i], p.scale2, lut[lut_index(p, key - (pos0 + j))]);
                        float e = __builtin_amdgcn_exp2f(s - lse2s[r0 + j]);
                        if (edge && (key >= len || (p.causal && key > pos0 + j))) e = 0.0f;
                        float g = dp[i], f = e;
                        if constexpr (DROP) {
                            const bool keep = bits[j >> 2] >> (8 * (j & 3) + (lane & 7)) & 1u;
                            g = keep ? g * p.keep_scale : 0.0f;
                            f = keep ? e : 0.0f;
                        }
                        pd[j] = f;
                        ds[j] = e * (g - deltas[r0 + j]);
                    }
                    const Frag<T> pf = frag_pack<T>(pd), df = frag_pack<T>(ds);
#pragma unroll
                    for (int d = 0; d < DP / 32; ++d) {
                        mma<T>(dv[d], frag_lds_transposed<T, PITCH>(Gs, 32 * u + 16 * x, 32 * d, lane), pf);
                        mma<T>(dk[d], frag_lds_transposed<T, PITCH>(Qs, 32 * u + 16 * x, 32 * d, lane), df);
                    }
                }
            }
        }
    }
    if (key >= p.Lk) return;
    raw_t *dkrow = (raw_t *)p.dk + (int64_t)b * p.dks[0] + (int64_t)hk * p.dks[1] + (int64_t)key * p.dks[2];
    raw_t *dvrow = (raw_t *)p.dv + (int64_t)b * p.dvs[0] + (int64_t)hk * p.dvs[1] + (int64_t)key * p.dvs[2];
    const float sk = p.scale, sv = p.keep_scale;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            const int col = 32 * d + 2 * r + 4 * half;
            store4<T>(dkrow, col, p.D, vec, dk[d][r] * sk, dk[d][r + 1] * sk, dk[d][r + 2] * sk, dk[d][r + 3] * sk);
            store4<T>(dvrow, col, p.D, vec, dv[d][r] * sv, dv[d][r + 1] * sv, dv[d][r + 2] * sv, dv[d][r + 3] * sv);
        }
}

// dtable[n][h]: the sums of one head over sequences and query tiles, in
// double, one block per head and bucket.
template <typename T>
__global__ __launch_bounds__(256) void attention_backward_table(AttnParams p) {
    __shared__ double red[4];
    const int n = blockIdx.x % p.buckets, h = blockIdx.x / p.buckets, t = threadIdx.x;
    const int64_t rows = (int64_t)p.B * p.tiles;
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
}

int big_lds(void (*fn)(AttnParams), int smem) {
    return smem > 65536
               ? (int)hipFuncSetAttribute((const void *)fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem)
               : 0;
}

template <typename T, int DP>
int launch_dp(const AttnParams &p0, hipStream_t stream) {
    AttnParams p = p0;
    const int lut = p.lut ? (p.lut + 3) / 4 * 16 : 0;
    if (p.Lq > 0) {
        p.tiles = (p.Lq + kAttnQueries - 1) / kAttnQueries;
        p.nblocks = p.B * p.H * p.tiles;
        const int smem = BwdGeo<T, DP>::tile_bytes + lut + (p.lut ? 8 * near_pitch(p.lut) * 4 : 0) + 32 + p.side * 2;
        void (*const fn)(AttnParams) =
            p.threshold ? attention_backward_q<T, DP, true> : attention_backward_q<T, DP, false>;
        if (const int e = big_lds(fn, smem)) return e;
        hipLaunchKernelGGL(fn, dim3((p.nblocks + 7) / 8 * 8), dim3(256), smem, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    if (p.dtable && p.buckets) {
        p.tiles = (p.Lq + kAttnQueries - 1) / kAttnQueries;
        hipLaunchKernelGGL(attention_backward_table<T>, dim3(p.buckets * p.H), dim3(256), 0, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    if (p.Lk > 0) {
        p.tiles = (p.Lk + kAttnQueries - 1) / kAttnQueries;
        p.nblocks = p.B * p.Hkv * p.tiles;
        const int smem = BwdGeo<T, DP>::tile_bytes + 2 * kRows * 4 + 512 + lut + p.side * 2;
        void (*const fn)(AttnParams) =
            p.threshold ? attention_backward_kv<T, DP, true> : attention_backward_kv<T, DP, false>;
        if (const int e = big_lds(fn, smem)) return e;
        hipLaunchKernelGGL(fn, dim3((p.nblocks + 7) / 8 * 8), dim3(256), smem, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    return 0;
}

template <typename T>
int launch_t(const AttnParams &p, hipStream_t stream) {
    if (p.D <= 32) return launch_dp<T, 32>(p, stream);
    if (p.D <= 64) return launch_dp<T, 64>(p, stream);
    if (p.D <= 96) return launch_dp<T, 96>(p, stream);
    return launch_dp<T, 128>(p, stream);
}

}  // namespace

int launch_attention_backward(const AttnParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return launch_t<F32>(p, stream);
    if (dtype == 1) return launch_t<F16>(p, stream);
    return launch_t<BF16>(p, stream);
}

}  // namespace gs
