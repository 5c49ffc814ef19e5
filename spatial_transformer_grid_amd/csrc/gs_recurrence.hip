// gs_recurrence.hip -- a gated linear recurrence along the tokens, forward and
// backward:  h_t = a_t h_(t-1) + (1 - a_t) x_t,  a_t = 1 / (1 + exp(-g_t)).
//
// n steps are one step with the product of their a and the state that they
// reach from zero.  A block has 64 lanes of channels and W waves of S steps
// each: every wave makes its steps' pair from the registers that hold them, the
// pairs go through LDS, each wave folds those before its own onto the state that
// the tile began at, and walks its steps again from there: everything is read
// once.  The order of the folds is fixed, so the same call gives the same bits.
//
// Backward: U_t = a_t D_t, the gradient that leaves step t towards h_(t-1), is
// the same recurrence the other way, U_t = a_t (dY_t + U_(t+1)).  The states are
// made again, a tile at a time, from those that the forward pass saved before
// every tile (a state a channel for kTile steps), in fp32: the rounded Y would
// carry its rounding into dG where h and x are close.
//
// Where there are too few channels for the chip, the tokens are split in parts
// over blocks: a first kernel makes each part's pair, and the blocks of the
// second one fold the pairs of the parts before theirs.
#include "gs_tokens.hpp"

namespace gs {

namespace {

constexpr int kTile = 128;             // steps of a tile: of a saved state
constexpr int kMaxParts = 256;

// a and 1 - a of a gate, neither from the other: both keep their relative
// precision.  e = exp(-|g|) is made in base 2, where fp32's product g log2(e)
// is rounded; with CORRECT (fp32 data) its remainder is put back.  The reciprocal
// takes one Newton step, since the error of a product of many a adds up.
template <bool CORRECT>
__device__ __forceinline__ void gate_of(float g, float &a, float &rest) {
    const float n = -fabsf(g), z = n * kLog2e;
    float e = __builtin_amdgcn_exp2f(z);
    if constexpr (CORRECT) {
        const float low = fmaf(n, 1.925963033500801e-8f, fmaf(n, kLog2e, -z));
        e = z > -120.0f ? fmaf(e * kLn2, low, e) : e;
    }
    const float d = 1.0f + e, r0 = __builtin_amdgcn_rcpf(d), r = fmaf(fmaf(-d, r0, 1.0f), r0, r0), er = e * r;
    a = g < 0.0f ? er : r;
    rest = g < 0.0f ? r : er;
}

// V neighbouring channels of a step, as they lie in memory.
template <typename T, int V>
struct Raw {
    typename T::raw_t v[V];
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const typename T::raw_t *src) {
    Raw<T, V> r;
    if constexpr (V * T::bytes == 2) r.v[0] = src[0];
    else if constexpr (V * T::bytes == 4) __builtin_memcpy(&r, (const uint32_t *)src, 4);
    else {
        const u32x2 w = *(const u32x2 *)src;
        __builtin_memcpy(&r, &w, 8);
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store_raw(typename T::raw_t *dst, const float *v) {
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = to_bits<T>(v[i]);
    if constexpr (V * T::bytes == 2) dst[0] = r.v[0];
    else if constexpr (V * T::bytes == 4) {
        uint32_t w;
        __builtin_memcpy(&w, &r, 4);
        *(uint32_t *)dst = w;
    } else {
        u32x2 w;
        __builtin_memcpy(&w, &r, 8);
        *(u32x2 *)dst = w;
    }
}

template <int V>
struct Floats {
    float v[V];
};

// The sequence, channels and part of a block, and a lane's first channel.
struct Place {
    int b, part, c, len;
    bool on;                                         // the lane has channels
    int t0, t1;                                      // steps of the part
};

template <int V>
__device__ __forceinline__ Place place(const ScanParams &p) {
    Place s;
    const int groups = (p.channels + 64 * V - 1) / (64 * V);
    int n = (int)blockIdx.x;
    s.part = n % p.parts;
    n /= p.parts;
    s.c = (n % groups * 64 + (int)(threadIdx.x & 63)) * V;
    s.b = n / groups;
    s.on = s.c < p.channels;
    s.len = p.lengths ? min(max(p.lengths[s.b], 0), p.length) : p.length;
    const int tiles = (p.length + kTile - 1) / kTile;
    s.t0 = (int)((int64_t)tiles * s.part / p.parts) * kTile;
    s.t1 = min((int)((int64_t)tiles * (s.part + 1) / p.parts) * kTile, p.length);
    return s;
}

// The state (or gradient) that a part begins at: `first` through the pairs of
// the parts before it, in the order that `from` and `step` say, a range of them
// a wave.  All of a block's threads take part.
template <int V, int W>
__device__ __forceinline__ void fold_parts(const ScanParams &p, const Place &s, int count, int from, int step, float *u,
                                           Floats<V> (*lds)[2][64]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t width = (int64_t)p.batch * p.channels, at = (int64_t)s.b * p.channels + s.c;
    float P[V], H[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        P[i] = 1.0f;
        H[i] = 0.0f;
    }
    if (s.on) {
        const int i1 = count * (wave + 1) / W;
#pragma unroll 8
        for (int i = count * wave / W; i < i1; ++i) {
            const float *pair = p.pairs + ((int64_t)(from + step * i) * 2) * width + at;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                P[j] *= pair[j];
                H[j] = fmaf(pair[j], H[j], pair[width + j]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        lds[wave][0][lane].v[i] = P[i];
        lds[wave][1][lane].v[i] = H[i];
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = fmaf(lds[w][0][lane].v[i], u[i], lds[w][1][lane].v[i]);
    __syncthreads();
}

template <int V>
__device__ __forceinline__ void load_state(const float *src, const Place &s, int channels, float *u) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = src && s.on ? src[(int64_t)s.b * channels + s.c + i] : 0.0f;
}

template <int V>
__device__ __forceinline__ void store_state(float *dst, int64_t at, const float *u) {
#pragma unroll
    for (int i = 0; i < V; ++i) dst[at + i] = u[i];
}

// Forward.  PAIRS: only the part's pair (the product of its gates, the state that
// it reaches) goes to the workspace; part 0 begins at the given state, which is
// copied, since the other kernel may write the last state over it.
template <typename T, int V, int W, bool PAIRS>
__global__ __launch_bounds__(64 * W) void recurrence_forward(ScanParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int S = kTile / W;
    __shared__ Floats<V> lds[2][W][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place s = place<V>(p);
    if (PAIRS && s.part == p.parts - 1) return;      // nothing follows it
    const int64_t width = (int64_t)p.batch * p.channels, at = (int64_t)s.b * p.channels + s.c;
    float u[V], product[V];
    const bool split = p.parts > 1;
    load_state<V>(!PAIRS && split ? p.copy : (s.part == 0 ? p.state : nullptr), s, p.channels, u);
    if (PAIRS && s.part == 0 && wave == 0 && s.on) store_state<V>(p.copy, at, u);
    if (!PAIRS && split) {
        // part 0's pair holds the first state already
        float first[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            first[i] = u[i];
            u[i] = 0.0f;
        }
        fold_parts<V, W>(p, s, s.part, 0, 1, u, lds[0]);
        if (s.part == 0)
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = first[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) product[i] = 1.0f;
    const raw_t *const x = (const raw_t *)p.x + (int64_t)s.b * p.xs[0] + s.c;
    const raw_t *const g = (const raw_t *)p.g + (int64_t)s.b * p.gs[0] + s.c;
    raw_t *const y = (raw_t *)p.y + (int64_t)s.b * p.ys[0] + s.c;
    const int chunks = (p.length + kTile - 1) / kTile;
    int turn = 0;
    Raw<T, V> xr[S], gr[S];
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int t = t0 + wave * S + i;
            xr[i] = gr[i] = Raw<T, V>{};
            if (t < s.len && t < s.t1 && s.on) {
                xr[i] = load_raw<T, V>(x + t * p.xs[1]);
                gr[i] = load_raw<T, V>(g + t * p.gs[1]);
            }
        }
    };
    fetch(s.t0);
    for (int t0 = s.t0; t0 < s.t1; t0 += kTile) {
        float a[S][V], b[S][V], P[V], H[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            P[i] = 1.0f;
            H[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const bool held = t0 + wave * S + i < s.len;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float rest;
                gate_of<T::bytes == 4>(T::from_raw(gr[i].v[j]), a[i][j], rest);
                b[i][j] = rest * T::from_raw(xr[i].v[j]);
                a[i][j] = held ? a[i][j] : 1.0f;     // past its length a sequence keeps its state
                b[i][j] = held ? b[i][j] : 0.0f;
                P[j] *= a[i][j];
                H[j] = fmaf(a[i][j], H[j], b[i][j]);
            }
        }
        fetch(t0 + kTile);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            lds[turn][wave][0][lane].v[j] = P[j];
            lds[turn][wave][1][lane].v[j] = H[j];
        }
        __syncthreads();
        if (!PAIRS && p.saved && wave == 0 && s.on && t0 < s.len)
            store_state<V>(p.saved, ((int64_t)s.b * chunks + t0 / kTile) * p.channels + s.c, u);
        float h[V];
#pragma unroll
        for (int w = 0; w < W; ++w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (w == wave) h[j] = u[j];
                const float q = lds[turn][w][0][lane].v[j];
                u[j] = fmaf(q, u[j], lds[turn][w][1][lane].v[j]);
                if (PAIRS) product[j] *= q;
            }
        turn ^= 1;                                   // the next tile's pairs do not wait for this one's readers
        if constexpr (!PAIRS) {
#pragma unroll
            for (int i = 0; i < S; ++i) {
                const int t = t0 + wave * S + i;
                float out[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    h[j] = fmaf(a[i][j], h[j], b[i][j]);
                    out[j] = t < s.len ? h[j] : 0.0f;
                }
                if (t < s.t1 && s.on) store_raw<T, V>(y + t * p.ys[1], out);
            }
        }
    }
    if (wave || !s.on) return;
    if (PAIRS) {
        float *pair = p.pairs + (int64_t)s.part * 2 * width;
        store_state<V>(pair, at, product);
        store_state<V>(pair + width, at, u);
    } else if (p.last && s.part == p.parts - 1) {
        store_state<V>(p.last, at, u);
    }
}

// Backward.  PAIRS: only the part's pair, in the other direction; the last part
// begins at dlast, which is copied for the same reason.
template <typename T, int V, int W, bool PAIRS>
__global__ __launch_bounds__(64 * W) void recurrence_backward(ScanParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int S = kTile / W, N = PAIRS ? 2 : 3;
    __shared__ Floats<V> lds[2][W][N][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place s = place<V>(p);
    if (PAIRS && s.part == 0) return;                // nothing follows it
    const int64_t width = (int64_t)p.batch * p.channels, at = (int64_t)s.b * p.channels + s.c;
    const int final_part = p.parts - 1;
    const bool split = p.parts > 1;
    float u[V], product[V];
    load_state<V>(!PAIRS && split ? p.copy : (s.part == final_part ? p.dlast : nullptr), s, p.channels, u);
    if (PAIRS && s.part == final_part && wave == 0 && s.on) store_state<V>(p.copy, at, u);
    if (!PAIRS && split) {
        float first[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            first[i] = u[i];
            u[i] = 0.0f;
        }
        fold_parts<V, W>(p, s, final_part - s.part, final_part, -1, u, (Floats<V>(*)[2][64])lds);
        if (s.part == final_part)
#pragma unroll
            for (int i = 0; i < V; ++i) u[i] = first[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) product[i] = 1.0f;
    const raw_t *const x = (const raw_t *)p.x + (int64_t)s.b * p.xs[0] + s.c;
    const raw_t *const g = (const raw_t *)p.g + (int64_t)s.b * p.gs[0] + s.c;
    const raw_t *const dy = (const raw_t *)p.dy + (int64_t)s.b * p.dys[0] + s.c;
    raw_t *const dx = (raw_t *)p.dx + (int64_t)s.b * p.dxs[0] + s.c;
    raw_t *const dg = (raw_t *)p.dg + (int64_t)s.b * p.dgs[0] + s.c;
    const int chunks = (p.length + kTile - 1) / kTile;
    int turn = 0;
    Raw<T, V> xn[S], gn[S], dn[S];
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const int t = t0 + wave * S + i;
            xn[i] = gn[i] = dn[i] = Raw<T, V>{};
            if (t < s.len && t >= s.t0 && t < s.t1 && s.on) {
                if (!PAIRS) xn[i] = load_raw<T, V>(x + t * p.xs[1]);
                gn[i] = load_raw<T, V>(g + t * p.gs[1]);
                dn[i] = load_raw<T, V>(dy + t * p.dys[1]);
            }
        }
    };
    const int last_tile = s.t1 > s.t0 ? s.t0 + (s.t1 - 1 - s.t0) / kTile * kTile : s.t0 - kTile;
    fetch(last_tile);
    for (int t0 = last_tile; t0 >= s.t0; t0 -= kTile) {
        Raw<T, V> xr[S], dr[S];
        float a[S][V], rest[S][V], P[V], H[V], U[V], h[V];
        if (!PAIRS) load_state<V>(p.saved ? p.saved + (int64_t)(t0 / kTile + s.b * (chunks - 1)) * p.channels : nullptr, s,
                                  p.channels, h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            P[j] = 1.0f;
            H[j] = U[j] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < S; ++i) {
            const bool held = t0 + wave * S + i < s.len;
            xr[i] = xn[i];
            dr[i] = dn[i];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                gate_of<T::bytes == 4>(T::from_raw(gn[i].v[j]), a[i][j], rest[i][j]);
                a[i][j] = held ? a[i][j] : 1.0f;
                rest[i][j] = held ? rest[i][j] : 0.0f;
                P[j] *= a[i][j];
                if (!PAIRS) H[j] = fmaf(a[i][j], H[j], rest[i][j] * T::from_raw(xr[i].v[j]));
            }
        }
#pragma unroll
        for (int i = S - 1; i >= 0; --i)
#pragma unroll
            for (int j = 0; j < V; ++j) U[j] = a[i][j] * (T::from_raw(dr[i].v[j]) + U[j]);
        fetch(t0 - kTile);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            lds[turn][wave][0][lane].v[j] = P[j];
            lds[turn][wave][1][lane].v[j] = U[j];
            if (!PAIRS) lds[turn][wave][N - 1][lane].v[j] = H[j];
        }
        __syncthreads();
        float mine[V];
#pragma unroll
        for (int w = W - 1; w >= 0; --w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (w == wave) mine[j] = u[j];
                const float q = lds[turn][w][0][lane].v[j];
                u[j] = fmaf(q, u[j], lds[turn][w][1][lane].v[j]);
                if (PAIRS) product[j] *= q;
            }
        if constexpr (!PAIRS) {
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (w < wave) h[j] = fmaf(lds[turn][w][0][lane].v[j], h[j], lds[turn][w][N - 1][lane].v[j]);
            float before[S][V];
#pragma unroll
            for (int i = 0; i < S; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    before[i][j] = h[j];
                    h[j] = fmaf(a[i][j], h[j], rest[i][j] * T::from_raw(xr[i].v[j]));
                }
#pragma unroll
            for (int i = S - 1; i >= 0; --i) {
                const int t = t0 + wave * S + i;
                float ox[V], og[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float D = T::from_raw(dr[i].v[j]) + mine[j];
                    const bool held = t < s.len;
                    ox[j] = held ? rest[i][j] * D : 0.0f;
                    og[j] = held ? D * (before[i][j] - T::from_raw(xr[i].v[j])) * (a[i][j] * rest[i][j]) : 0.0f;
                    mine[j] = a[i][j] * D;
                }
                if (t < s.t1 && s.on) {
                    store_raw<T, V>(dx + t * p.dxs[1], ox);
                    store_raw<T, V>(dg + t * p.dgs[1], og);
                }
            }
        }
        turn ^= 1;
    }
    if (wave || !s.on) return;
    if (PAIRS) {
        float *pair = p.pairs + (int64_t)s.part * 2 * width;
        store_state<V>(pair, at, product);
        store_state<V>(pair + width, at, u);
    } else if (p.dstate && s.part == 0) {
        store_state<V>(p.dstate, at, u);
    }
}

// --------------------------------------------------------------- launches

constexpr int kWaves = 8, kBackwardWaves = 16;

template <typename T, int V>
int launch(const ScanParams &p, bool backward, hipStream_t stream) {
    const int64_t units = (int64_t)p.batch * ((p.channels + 64 * V - 1) / (64 * V));
    const dim3 grid((unsigned)(units * p.parts)), fwd(64 * kWaves), bwd(64 * kBackwardWaves);
    if (p.parts > 1) {
        if (backward) hipLaunchKernelGGL((recurrence_backward<T, V, kBackwardWaves, true>), grid, bwd, 0, stream, p);
        else hipLaunchKernelGGL((recurrence_forward<T, V, kWaves, true>), grid, fwd, 0, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    if (backward) hipLaunchKernelGGL((recurrence_backward<T, V, kBackwardWaves, false>), grid, bwd, 0, stream, p);
    else hipLaunchKernelGGL((recurrence_forward<T, V, kWaves, false>), grid, fwd, 0, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int pick(const ScanParams &p, bool backward, hipStream_t stream) {
    return p.pairwise ? launch<T, 2>(p, backward, stream) : launch<T, 1>(p, backward, stream);
}

}  // namespace

// Parts of the tokens: as many as give every compute unit two blocks, of four
// tiles at least.
int recurrence_parts(int64_t batch, int64_t length, int64_t channels, bool pairwise) {
    const int64_t lanes = pairwise ? 128 : 64, units = batch * ((channels + lanes - 1) / lanes);
    if (units == 0 || units >= 256) return 1;
    const int64_t tiles = (length + kTile - 1) / kTile;
    int64_t parts = 512 / units;
    if (parts > tiles / 4) parts = tiles / 4;
    if (parts > kMaxParts) parts = kMaxParts;
    return parts < 2 ? 1 : (int)parts;
}

int launch_recurrence(const ScanParams &p, int dtype, bool backward, hipStream_t stream) {
    if (dtype == 0) return pick<F32>(p, backward, stream);
    if (dtype == 1) return pick<F16>(p, backward, stream);
    return pick<BF16>(p, backward, stream);
}

}  // namespace gs
