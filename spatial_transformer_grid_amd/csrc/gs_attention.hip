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
#include "gs_tokens.hpp"

namespace gs {

namespace {

constexpr int kKeys = 64;   // keys of an LDS tile

template <typename T, int DP>
struct FwdGeo {
    static constexpr int PITCH = DP + 16 / T::bytes;
    static constexpr int tile_elems = kKeys * PITCH;
    static constexpr int fixed_bytes = 2 * tile_elems * T::bytes;
};

template <typename T, int DP, bool DROP>
__global__ __launch_bounds__(256) void attention_forward(AttnParams p) {
    typedef typename T::raw_t raw_t;
    typedef FwdGeo<T, DP> Geo;
    constexpr int PITCH = Geo::PITCH;
    extern __shared__ __align__(16) unsigned char smem[];
    raw_t *Ks = (raw_t *)smem;
    raw_t *Vs = Ks + Geo::tile_elems;
    float *lut = (float *)(smem + Geo::fixed_bytes);

    const int lb = xcd_contiguous_block(p.nblocks);
    if (lb >= p.nblocks) return;
    int tile = lb % p.tiles;
    const int bh = lb / p.tiles;
    if (p.causal) tile = p.tiles - 1 - tile;        // the longest rows first
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
    const bool vec = p.vec;

    const raw_t *kb = (const raw_t *)p.k + (int64_t)b * p.ks[0] + (int64_t)hk * p.ks[1];
    const raw_t *vb = (const raw_t *)p.v + (int64_t)b * p.vs[0] + (int64_t)hk * p.vs[1];
    const raw_t *qrow =
        (const raw_t *)p.q + (int64_t)b * p.qs[0] + (int64_t)h * p.qs[1] + (int64_t)qi * p.qs[2];
    Frag<T> qf[DP / 16];
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) qf[s] = frag_global<T>(qrow, 16 * s + 8 * half, p.D, qi < p.Lq, vec);
    if (p.lut) fill_lut<T>(p, h, lut, (uint16_t *)(lut + p.lut), t, 256);

    f32x16 acc[DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    TileCopy<T, DP, kKeys, 256, PITCH> copy;
    for (int k0 = 0; k0 < end; k0 += kKeys) {
        __syncthreads();
        copy.fetch(kb, p.ks[2], k0, end, p.D, vec, t);
        copy.put(Ks, t);
        copy.fetch(vb, p.vs[2], k0, end, p.D, vec, t);
        copy.put(Vs, t);
        __syncthreads();
        const int wave_first = first + q0, wave_last = wave_first + 31;
        if (q0 >= p.Lq || (p.causal && k0 > wave_last)) continue;

        float s[32];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x16 st;
#pragma unroll
            for (int r = 0; r < 16; ++r) st[r] = 0.0f;
            const raw_t *row = Ks + (32 * u + a_row(lane & 31)) * PITCH + 8 * half;
#pragma unroll
            for (int x = 0; x < DP / 16; ++x) mma<T>(st, frag_lds<T>(row + 16 * x), qf[x]);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[16 * u + r] = st[r];
        }
        // s[16 u + 8 x + j]: key k0 + 32 u + 16 x + 8 half + j of this lane's query
        const int key0 = k0 + 8 * half;
        if (p.lut) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                s[i] = fmaf(s[i], p.scale2, lut[lut_index(p, key0 + 16 * (i >> 3) + (i & 7) - pos)]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] *= p.scale2;
        }
        if (k0 + kKeys > end || (p.causal && k0 + kKeys - 1 > wave_first)) {
            const int seen = p.causal ? min(end, pos + 1) : end;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (key0 + 16 * (i >> 3) + (i & 7) >= seen) s[i] = -INFINITY;
        }
        float top = m;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, s[i]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float base = top == -INFINITY ? 0.0f : top;
        const float alpha = __builtin_amdgcn_exp2f(m - base);
        m = top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            s[i] = __builtin_amdgcn_exp2f(s[i] - base);
            sum += s[i];
        }
        l = fmaf(l, alpha, sum);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[d][r] *= alpha;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if constexpr (DROP) {
                const u32x4 rnd = philox((uint32_t)(key0 + 16 * x) >> 3, (uint32_t)qi, (uint32_t)bh, p.call,
                                         p.seed_lo, p.seed_hi);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[8 * x + j] = kept(rnd, j, p.threshold) ? s[8 * x + j] : 0.0f;
            }
            const Frag<T> pf = frag_pack<T>(s + 8 * x);
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
                mma<T>(acc[d], frag_lds_transposed<T, PITCH>(Vs, 16 * x, 32 * d, lane), pf);
        }
    }
    l += __shfl_xor(l, 32);
    if (qi >= p.Lq) return;
    const float norm = l > 0.0f || l != l ? p.keep_scale / l : 0.0f;
    raw_t *orow = (raw_t *)p.o + (int64_t)b * p.os[0] + (int64_t)h * p.os[1] + (int64_t)qi * p.os[2];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            store4<T>(orow, 32 * d + 2 * r + 4 * half, p.D, vec, acc[d][r] * norm, acc[d][r + 1] * norm,
                      acc[d][r + 2] * norm, acc[d][r + 3] * norm);
    if (p.lse && half == 0)
        p.lse[(int64_t)bh * p.Lq + qi] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

template <typename T, int DP>
int launch_dp(const AttnParams &p, hipStream_t stream) {
    const int smem = FwdGeo<T, DP>::fixed_bytes + p.lut * 4 + (p.lut ? p.side * 2 : 0);
    const dim3 grid((p.nblocks + 7) / 8 * 8);
    void (*const fn)(AttnParams) = p.threshold ? attention_forward<T, DP, true> : attention_forward<T, DP, false>;
    if (smem > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)fn, hipFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != hipSuccess) return (int)e;
    }
    hipLaunchKernelGGL(fn, grid, dim3(256), smem, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int launch_t(const AttnParams &p, hipStream_t stream) {
    if (p.D <= 32) return launch_dp<T, 32>(p, stream);
    if (p.D <= 64) return launch_dp<T, 64>(p, stream);
    if (p.D <= 96) return launch_dp<T, 96>(p, stream);
    return launch_dp<T, 128>(p, stream);
}

}  // namespace

int launch_attention(const AttnParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return launch_t<F32>(p, stream);
    if (dtype == 1) return launch_t<F16>(p, stream);
    return launch_t<BF16>(p, stream);
}

}  // namespace gs
