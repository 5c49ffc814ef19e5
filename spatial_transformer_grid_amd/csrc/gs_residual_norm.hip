// gs_residual_norm.hip -- the norms before and after a block, joined with its
// gate and the residual, forward and backward.
//
// Forward: p = norm(branch), H = alpha X + gate p, Y = norm(H): one pass, a
// row stays in the registers of the NT threads that share it, eight or sixteen
// elements each.  As in gs_norm.hip a layer norm's mean is a division and the
// variance a second sum over the registers.
//
// Backward, with fh and hh the normalised branch and H, made again from X and
// branch (as many bytes as H and branch, and H is not rounded):
//   dh = dH + inv_h (g - mean(g) - hh mean(g hh)),  g = dY pre_scale,
//   dX = alpha dh,  dgate = dh p,  dp = dh gate,
//   dbranch = inv_f (k - mean(k) - fh mean(k fh)),  k = dp post_scale,
//   dpre = sum of dY hh,  dpost = sum of dp fh, and the biases' sums.
// (mean(g) and mean(k) are there with `layer` only.)  The sums over rows are
// made in parts, one a block, its rows in order, and added up by a second
// kernel, so that the order is fixed.
#include "gs_rows.hpp"

namespace gs {

namespace {

constexpr int kThreads = 512;         // of a block whose rows take fewer

constexpr int join_threads(int nt) { return nt < kThreads ? kThreads : nt; }

// Two sums over the NT threads of a row; `red` has room for the waves of a
// block, twice, and `turn` says which half is used: one barrier a sum, since
// the other half's readers have passed it.
template <int NT>
__device__ __forceinline__ void join_totals(float &a, float &b, float *red, int &turn) {
    a = lanes_total<(NT < 64 ? NT : 64)>(a);
    b = lanes_total<(NT < 64 ? NT : 64)>(b);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64, ALL = join_threads(NT) / 64;
        float *at = red + turn * 2 * ALL;
        turn ^= 1;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            at[wave] = a;
            at[ALL + wave] = b;
        }
        __syncthreads();
        const int first = wave / W * W;
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += at[first + w];
            b += at[ALL + first + w];
        }
    }
}

// Mean and factor of a row's values v (zeros past its end), which come out as
// v - mean where `layer`.
template <int NT, int E, bool VEC>
__device__ __forceinline__ void row_stats(float *v, int layer, int cols, int t, float epsilon, float *red, int &turn,
                                          float &mean, float &inv) {
    float s = 0.0f, none = 0.0f;
    mean = 0.0f;
    if (layer) {
#pragma unroll
        for (int e = 0; e < E; ++e) s += v[e];
        join_totals<NT>(s, none, red, turn);
        mean = s / (float)cols;
        s = none = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = column<NT, VEC>(t, e) < cols ? v[e] - mean : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(v[e], v[e], s);
    join_totals<NT>(s, none, red, turn);
    inv = 1.0f / sqrtf(s / (float)cols + epsilon);
}

// A row of the gate: ones where there is none.
template <typename T, int NT, int E, bool VEC>
__device__ __forceinline__ void load_gate(const JoinParams &p, int64_t row, int t, float *m) {
    if (!p.gate) {
#pragma unroll
        for (int e = 0; e < E; ++e) m[e] = 1.0f;
    } else if (p.gate_f32) {
        load_row<F32, NT, E, VEC>((const uint32_t *)p.gate + row * p.cols, p.cols, t, m);
    } else {
        load_row<T, NT, E, VEC>((const typename T::raw_t *)p.gate + row * p.cols, p.cols, t, m);
    }
}

template <typename T, int NT, int E, bool VEC>
__global__ __launch_bounds__(join_threads(NT)) void residual_norm_rows(JoinParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int ROWS = join_threads(NT) / NT;
    __shared__ float red[NT > 64 ? 4 * join_threads(NT) / 64 : 1];
    int turn = 0;
    const int t = threadIdx.x % NT, cols = p.cols;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < p.rows; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + threadIdx.x / NT;
        const bool live = r < p.rows;                // (a block's rows meet the same barriers)
        const int64_t at = live ? r : p.rows - 1;
        float f[E], x[E], m[E];
        load_row<T, NT, E, VEC>((const raw_t *)p.branch + at * p.branch_stride, cols, t, f);
        load_row<T, NT, E, VEC>((const raw_t *)p.x + at * p.x_stride, cols, t, x);
        load_gate<T, NT, E, VEC>(p, p.gate ? at / p.group : 0, t, m);
        float mean_f = 0.0f, inv_f = 1.0f, mean_h = 0.0f, inv_h = 1.0f;
        if (p.post) {
            float w[E], b[E];
            load_params<T, NT, E, VEC>(p.post, p.param_f32, cols, t, w);
            load_params<T, NT, E, VEC>(p.post_bias, p.param_f32, cols, t, b);
            row_stats<NT, E, VEC>(f, p.layer, cols, t, p.epsilon, red, turn, mean_f, inv_f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = fmaf(f[e] * inv_f, w[e], b[e]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(p.alpha, x[e], m[e] * f[e]);
        if (live) store_row<T, NT, E, VEC>((raw_t *)p.h + r * p.h_stride, cols, t, x);
        if (p.pre) {
            float w[E], b[E];
            load_params<T, NT, E, VEC>(p.pre, p.param_f32, cols, t, w);
            load_params<T, NT, E, VEC>(p.pre_bias, p.param_f32, cols, t, b);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = column<NT, VEC>(t, e) < cols ? x[e] : 0.0f;
            row_stats<NT, E, VEC>(x, p.layer, cols, t, p.epsilon, red, turn, mean_h, inv_h);
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = fmaf(x[e] * inv_h, w[e], b[e]);
            if (live) store_row<T, NT, E, VEC>((raw_t *)p.y + r * p.y_stride, cols, t, x);
        }
        if (live && t == 0 && p.stats) *(tokens_f32x4 *)(p.stats + 4 * r) = tokens_f32x4{mean_f, inv_f, mean_h, inv_h};
    }
}

// Adds up v over a block's rows (row slots in order) and hands each column's
// sum to `write`, from the threads of the first slot.
template <int NT, int E, bool VEC, typename Write>
__device__ __forceinline__ void slot_sums(const float *v, float *sums, int t, int slot, int cols, const Write &write) {
    constexpr int ROWS = join_threads(NT) / NT;
    if constexpr (ROWS > 1) {
#pragma unroll
        for (int e = 0; e < E; e += 8) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[(slot * 8 + j) * NT + t] = v[e + j];
            __syncthreads();
            if (slot == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float s = v[e + j];
                    for (int i = 1; i < ROWS; ++i) s += sums[(i * 8 + j) * NT + t];
                    const int c = column<NT, VEC>(t, e + j);
                    if (c < cols) write(c, s);
                }
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = column<NT, VEC>(t, e);
            if (c < cols) write(c, v[e]);
        }
    }
}

// A block takes whole groups of rows that share a row of the gate, or (parts > 1)
// one part of one group.
template <typename T, int NT, int E, bool VEC>
__global__ __launch_bounds__(join_threads(NT)) void residual_norm_backward_rows(JoinParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int BT = join_threads(NT), ROWS = BT / NT;
    __shared__ float red[NT > 64 ? 4 * BT / 64 : 1];
    __shared__ float sums[ROWS > 1 ? BT * 8 : 1];
    int turn = 0;
    const int t = threadIdx.x % NT, slot = threadIdx.x / NT, cols = p.cols;
    float s_post[E], s_post_b[E], s_pre[E], s_pre_b[E], s_gate[E];
#pragma unroll
    for (int e = 0; e < E; ++e) s_post[e] = s_post_b[e] = s_pre[e] = s_pre_b[e] = 0.0f;
    const int64_t g0 = p.parts > 1 ? blockIdx.x / p.parts : p.groups * (int64_t)blockIdx.x / gridDim.x;
    const int64_t g1 = p.parts > 1 ? g0 + 1 : p.groups * (int64_t)(blockIdx.x + 1) / gridDim.x;
    const int part = p.parts > 1 ? blockIdx.x % p.parts : 0;
    for (int64_t g = g0; g < g1; ++g) {
#pragma unroll
        for (int e = 0; e < E; ++e) s_gate[e] = 0.0f;
        const int64_t first = g * p.span + p.span * part / p.parts, end = g * p.span + p.span * (part + 1) / p.parts;
        for (int64_t r0 = first; r0 < end; r0 += ROWS) {
            const int64_t r = r0 + slot;
            const bool live = r < end;
            const int64_t at = live ? r : end - 1;
            float f[E], h[E], m[E], d[E], fp[E];
            const tokens_f32x4 st = *(const tokens_f32x4 *)(p.stats + 4 * at);
            load_row<T, NT, E, VEC>((const raw_t *)p.branch + at * p.branch_stride, cols, t, f);
            load_row<T, NT, E, VEC>((const raw_t *)p.x + at * p.x_stride, cols, t, h);
            load_gate<T, NT, E, VEC>(p, p.gate ? at / p.group : 0, t, m);
            if (p.d_h) {
                load_row<T, NT, E, VEC>((const raw_t *)p.d_h + at * p.dh_stride, cols, t, d);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = 0.0f;
            }
            // f: normalised branch; fp: what the gate multiplies
            if (p.post) {
                float w[E], b[E];
                load_params<T, NT, E, VEC>(p.post, p.param_f32, cols, t, w);
                load_params<T, NT, E, VEC>(p.post_bias, p.param_f32, cols, t, b);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    f[e] = column<NT, VEC>(t, e) < cols ? (f[e] - st[0]) * st[1] : 0.0f;
                    fp[e] = fmaf(f[e], w[e], b[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) fp[e] = f[e];
            }
            if (p.pre) {
                float y[E], w[E], a = 0.0f, c = 0.0f;
                load_row<T, NT, E, VEC>((const raw_t *)p.d_y + at * p.dy_stride, cols, t, y);
                load_params<T, NT, E, VEC>(p.pre, p.param_f32, cols, t, w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float z = fmaf(p.alpha, h[e], m[e] * fp[e]);
                    h[e] = column<NT, VEC>(t, e) < cols ? (z - st[2]) * st[3] : 0.0f;
                    if (live) {
                        s_pre[e] = fmaf(y[e], h[e], s_pre[e]);
                        s_pre_b[e] += y[e];
                    }
                    y[e] *= w[e];
                    a += y[e];
                    c = fmaf(y[e], h[e], c);
                }
                join_totals<NT>(a, c, red, turn);
                a = p.layer ? a / (float)cols : 0.0f;
                c /= (float)cols;
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] += st[3] * (y[e] - a - h[e] * c);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = p.alpha * d[e];
            if (live) store_row<T, NT, E, VEC>((raw_t *)p.dx + r * p.dx_stride, cols, t, h);
            if (p.dgate) {
#pragma unroll
                for (int e = 0; e < E; ++e) h[e] = d[e] * fp[e];
                if (p.by_token) {
                    if (live && p.gate_f32)
                        store_row<F32, NT, E, VEC>((uint32_t *)p.dgate + r * cols, cols, t, h);
                    else if (live)
                        store_row<T, NT, E, VEC>((raw_t *)p.dgate + r * cols, cols, t, h);
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < E; ++e) s_gate[e] += h[e];
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= m[e];
            if (p.post) {
                float w[E], a = 0.0f, c = 0.0f;
                load_params<T, NT, E, VEC>(p.post, p.param_f32, cols, t, w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (live) {
                        s_post[e] = fmaf(d[e], f[e], s_post[e]);
                        s_post_b[e] += d[e];
                    }
                    d[e] = column<NT, VEC>(t, e) < cols ? d[e] * w[e] : 0.0f;
                    a += d[e];
                    c = fmaf(d[e], f[e], c);
                }
                join_totals<NT>(a, c, red, turn);
                a = p.layer ? a / (float)cols : 0.0f;
                c /= (float)cols;
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = st[1] * (d[e] - a - f[e] * c);
            }
            if (live) store_row<T, NT, E, VEC>((raw_t *)p.dbranch + r * p.dbranch_stride, cols, t, d);
        }
        if (p.dgate && !p.by_token) {
            if (p.parts > 1) {
                float *const out = p.partial + ((int64_t)blockIdx.x * p.vectors + p.vectors - 1) * cols;
                slot_sums<NT, E, VEC>(s_gate, sums, t, slot, cols, [&](int c, float s) { out[c] = s; });
            } else {
                slot_sums<NT, E, VEC>(s_gate, sums, t, slot, cols, [&](int c, float s) {
                    if (p.gate_f32) ((float *)p.dgate)[g * cols + c] = s;
                    else ((raw_t *)p.dgate)[g * cols + c] = to_bits<T>(s);
                });
            }
        }
    }
    float *out = p.partial + (int64_t)blockIdx.x * p.vectors * cols;
    const auto put = [&](const float *v, const void *wanted) {
        if (!wanted) return;
        slot_sums<NT, E, VEC>(v, sums, t, slot, cols, [&](int c, float s) { out[c] = s; });
        out += cols;
    };
    put(s_post, p.dpost);
    put(s_post_b, p.dpost_bias);
    put(s_pre, p.dpre);
    put(s_pre_b, p.dpre_bias);
}

// Sums of the parts: 64 columns a block, sixteen waves with a range of the parts
// each, added in order.  The first `rows_of_params` rows of blocks are the
// parameters' vectors over all parts, the others the gate's rows over theirs.
template <typename T>
__global__ __launch_bounds__(1024) void residual_norm_sums(JoinParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = (int)blockIdx.x * 64 + lane;
    const int wide = (p.cols + 63) / 64;
    (void)wide;
    void *const outs[4] = {p.dpost, p.dpost_bias, p.dpre, p.dpre_bias};
    int which = 0, left = (int)blockIdx.y;
    for (; which < 4; ++which) {
        if (!outs[which]) continue;
        if (left == 0) break;
        --left;
    }
    const bool gate = which == 4;                    // then `left` is the gate's row
    const int vector = gate ? p.vectors - 1 : (int)blockIdx.y;
    const int n = gate ? p.parts : p.blocks;
    const int64_t step = (int64_t)p.vectors * p.cols;
    float s = 0.0f;
    if (c < p.cols) {
        const float *v = p.partial + (gate ? (int64_t)left * p.parts * step : 0) + (int64_t)vector * p.cols + c;
        const int i0 = n * wave / 16, i1 = n * (wave + 1) / 16;
        int i = i0;
        for (; i + 8 <= i1; i += 8) {
            float a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = v[(i + j) * step];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += a[j];
        }
        for (; i < i1; ++i) s += v[i * step];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave || c >= p.cols) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    if (gate) {
        const int64_t at = (int64_t)left * p.cols + c;
        if (p.gate_f32) ((float *)p.dgate)[at] = s;
        else ((raw_t *)p.dgate)[at] = to_bits<T>(s);
    } else if (p.param_f32) {
        ((float *)outs[which])[c] = s;
    } else {
        ((raw_t *)outs[which])[c] = to_bits<T>(s);
    }
}

// --------------------------------------------------------------- launches

// Threads of a row: eight elements each up to 8192 columns.
int row_threads(int64_t cols) {
    if (cols <= 64) return 8;
    if (cols <= 256) return 32;
    if (cols <= 512) return 64;
    if (cols <= 1024) return 128;
    if (cols <= 2048) return 256;
    return cols <= 4096 ? 512 : 1024;
}

int block_rows(int64_t cols) { return join_threads(row_threads(cols)) / row_threads(cols); }

constexpr int kForwardBlocks = 1024, kBackwardBlocks = 512;

template <typename T, int NT, int E>
void rows_form(const JoinParams &p, bool backward, hipStream_t stream) {
    constexpr int BT = join_threads(NT);
    if (backward) {
        if (p.vec) hipLaunchKernelGGL((residual_norm_backward_rows<T, NT, E, true>), dim3(p.blocks), dim3(BT), 0, stream, p);
        else hipLaunchKernelGGL((residual_norm_backward_rows<T, NT, E, false>), dim3(p.blocks), dim3(BT), 0, stream, p);
        return;
    }
    const int64_t blocks = (p.rows + BT / NT - 1) / (BT / NT);
    const dim3 grid((unsigned)(blocks < kForwardBlocks ? blocks : kForwardBlocks));
    if (p.vec) hipLaunchKernelGGL((residual_norm_rows<T, NT, E, true>), grid, dim3(BT), 0, stream, p);
    else hipLaunchKernelGGL((residual_norm_rows<T, NT, E, false>), grid, dim3(BT), 0, stream, p);
}

template <typename T>
int rows_launch(const JoinParams &p, bool backward, hipStream_t stream) {
    switch (row_threads(p.cols)) {
        case 8: rows_form<T, 8, 8>(p, backward, stream); break;
        case 32: rows_form<T, 32, 8>(p, backward, stream); break;
        case 64: rows_form<T, 64, 8>(p, backward, stream); break;
        case 128: rows_form<T, 128, 8>(p, backward, stream); break;
        case 256: rows_form<T, 256, 8>(p, backward, stream); break;
        case 512: rows_form<T, 512, 8>(p, backward, stream); break;
        default:
            if (p.cols <= 8192) rows_form<T, 1024, 8>(p, backward, stream);
            else rows_form<T, 1024, 16>(p, backward, stream);
    }
    return (int)hipGetLastError();
}

template <typename T>
int backward(const JoinParams &p, hipStream_t stream) {
    if (p.rows > 0)
        if (const int e = rows_launch<T>(p, true, stream)) return e;
    const int sums = (p.dpost != nullptr) + (p.dpost_bias != nullptr) + (p.dpre != nullptr) + (p.dpre_bias != nullptr) +
                     (p.parts > 1 && p.dgate && !p.by_token ? (int)p.groups : 0);
    if (sums == 0) return 0;
    const dim3 grid((unsigned)((p.cols + 63) / 64), (unsigned)sums);
    hipLaunchKernelGGL(residual_norm_sums<T>, grid, dim3(1024), 0, stream, p);
    return (int)hipGetLastError();
}

}  // namespace

// Groups of rows, their parts and the blocks of a backward call.  A group's rows
// are cut into parts where there are fewer groups than blocks that run at once;
// without sums for the gate all rows are one group.
JoinPlan plan_residual_norm(int64_t rows, int64_t cols, int64_t gate_rows) {
    JoinPlan s = {};
    s.by_token = gate_rows == rows;
    s.groups = gate_rows == 0 || s.by_token ? 1 : gate_rows;
    if (rows == 0) s.groups = 0;
    s.span = s.groups ? rows / s.groups : 0;
    s.parts = 1;
    if (s.groups >= kBackwardBlocks) {
        s.blocks = kBackwardBlocks;
    } else if (s.groups > 0) {
        const int64_t slots = (s.span + block_rows(cols) - 1) / block_rows(cols), most = kBackwardBlocks / s.groups;
        s.parts = (int)(slots < most ? slots : most);
        if (s.parts < 1) s.parts = 1;
        s.blocks = (int)(s.groups * s.parts);
    }
    return s;
}

int launch_residual_norm(const JoinParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return rows_launch<F32>(p, false, stream);
    if (dtype == 1) return rows_launch<F16>(p, false, stream);
    return rows_launch<BF16>(p, false, stream);
}

int launch_residual_norm_backward(const JoinParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return backward<F32>(p, stream);
    if (dtype == 1) return backward<F16>(p, stream);
    return backward<BF16>(p, stream);
}

}  // namespace gs
