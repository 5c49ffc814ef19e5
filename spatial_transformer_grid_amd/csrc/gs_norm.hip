// gs_norm.hip -- layer normalisation, forward and backward.
//
// Forward: mean, then the sum of (x - mean)^2 (two passes over the row, so
// that a large mean does not cancel).  The mean is a division: times a rounded
// 1 / cols a constant row of 1e4 in 41 columns keeps a deviation of 1e-3, which
// epsilon = 1e-5 makes y = 0.3 (400000 x 40 bf16: 14.8 us, with a product 14.3;
// wider rows the same).  Backward, with xh = (x - mean) inv_std
// and g = dy scale: dx = inv_std (g - mean(g) - xh mean(g xh)); dscale and
// dbias are sums over rows, made in parts (one per block, its rows in order)
// and added up by a second kernel, so that the order is fixed.
//
// Both are bound by memory, so each row is read once and stays in registers
// between its passes: NT threads hold E elements each (eight lanes up to 64
// columns, 32 up to 256, a wave up to 2048, a block of 256 threads up to 8192,
// one of 1024 up to 32768), and what belongs to a column (scale, bias, the sums
// of dscale and dbias) stays there from row to row.  Wider rows take the loops
// over memory at the end.
// Measured at 16384 x 2048 bf16 with fp32 parameters: forward 23 us (5.8 TB/s),
// backward 39 us (5.2 TB/s), the parts' sums 4.6 us; with a block a row and the
// row read again for each pass it was 68, 61 + 75 and 21 us.  40000 x 40 bf16:
// 3.8 and 11 us, a wave a row 12.5 and 17 us.  4000 x 8000 bf16: 23 and 51 us,
// with 1024 threads of eight elements 29 and 63 us.
#include "gs_rows.hpp"

namespace gs {

namespace {

constexpr int block_threads(int nt) { return nt < 256 ? 256 : nt; }

template <typename T, int NT, int E, bool VEC>
__global__ __launch_bounds__(block_threads(NT)) void layer_norm_rows(NormParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int ROWS = block_threads(NT) / NT;    // rows of a block at a time
    __shared__ float red[NT > 64 ? 2 * NT / 64 : 1];
    const int t = threadIdx.x % NT, cols = p.cols;
    const float inv_n = 1.0f / (float)cols;
    float w[E], b[E];
    load_params<T, NT, E, VEC>(p.scale, p.param_f32, cols, t, w);
    load_params<T, NT, E, VEC>(p.bias, p.param_f32, cols, t, b);
    for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT; r < p.rows; r += (int64_t)gridDim.x * ROWS) {
        float x[E];
        load_row<T, NT, E, VEC>((const raw_t *)p.X + r * p.x_stride, cols, t, x);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += x[e];
        const float mean = row_total<NT>(s, red) / (float)cols;
        s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] -= mean;
            if (column<NT, VEC>(t, e) < cols) s = fmaf(x[e], x[e], s);
        }
        const float inv = 1.0f / sqrtf(row_total<NT>(s, red) * inv_n + p.epsilon);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(x[e] * inv, w[e], b[e]);
        store_row<T, NT, E, VEC>((raw_t *)p.Y + r * p.y_stride, cols, t, x);
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.inv_std) p.inv_std[r] = inv;
        }
    }
}

// Block `part` takes the rows of one part: dx of each, and their sums of dy xh
// and dy, which the groups of threads add up in order at the end.
template <typename T, int NT, int E, bool VEC>
__global__ __launch_bounds__(block_threads(NT)) void layer_norm_backward_rows(NormParams p) {
    typedef typename T::raw_t raw_t;
    constexpr int ROWS = block_threads(NT) / NT;
    __shared__ float red[NT > 64 ? 2 * NT / 64 : 1];
    __shared__ float sums[ROWS > 1 ? ROWS * NT * 8 : 1];
    const int t = threadIdx.x % NT, group = threadIdx.x / NT, cols = p.cols;
    const float inv_n = 1.0f / (float)cols;
    float w[E], ds[E], db[E];
    load_params<T, NT, E, VEC>(p.scale, p.param_f32, cols, t, w);
#pragma unroll
    for (int e = 0; e < E; ++e) ds[e] = db[e] = 0.0f;
    const int64_t r0 = p.rows * (int64_t)blockIdx.x / gridDim.x, r1 = p.rows * (int64_t)(blockIdx.x + 1) / gridDim.x;
    for (int64_t r = r0 + group; r < r1; r += ROWS) {
        float x[E], g[E];
        load_row<T, NT, E, VEC>((const raw_t *)p.X + r * p.x_stride, cols, t, x);
        load_row<T, NT, E, VEC>((const raw_t *)p.dY + r * p.dy_stride, cols, t, g);
        const float mean = p.mean[r], inv = p.inv_std[r];
        float a = 0.0f, c = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            // (past the row's end x is 0, and mean inv_std may be infinite)
            x[e] = column<NT, VEC>(t, e) < cols ? (x[e] - mean) * inv : 0.0f;
            ds[e] = fmaf(g[e], x[e], ds[e]);
            db[e] += g[e];
            g[e] *= w[e];                            // 0 past the row's end, with w
            a += g[e];
            c = fmaf(g[e], x[e], c);
        }
        row_totals<NT>(a, c, red);
        a *= inv_n;
        c *= inv_n;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = inv * (g[e] - a - x[e] * c);
        store_row<T, NT, E, VEC>((raw_t *)p.dX + r * p.dx_stride, cols, t, x);
    }
    if (!p.dscale) return;
    float *out = p.partial + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float *v = which ? db : ds;
        if constexpr (ROWS > 1) {
            // eight elements of every thread at a time
#pragma unroll
            for (int e = 0; e < E; e += 8) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < 8; ++j) sums[(group * 8 + j) * NT + t] = v[e + j];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float s = v[e + j];
#pragma unroll
                        for (int i = 1; i < ROWS; ++i) s += sums[(i * 8 + j) * NT + t];
                        const int c = column<NT, VEC>(t, e + j);
                        if (c < cols) out[which * (int64_t)cols + c] = s;
                    }
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = column<NT, VEC>(t, e);
                if (c < cols) out[which * (int64_t)cols + c] = v[e];
            }
        }
    }
}

// dscale and dbias from the parts: 64 of the 2 cols columns a block, sixteen
// waves with a range of the parts each, added in order.
template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_param_sums(NormParams p) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t both = 2 * (int64_t)p.cols, c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < both) {
        const int i0 = p.parts * wave / 16, i1 = p.parts * (wave + 1) / 16;
        const float *v = p.partial + c;
        int i = i0;
        for (; i + 8 <= i1; i += 8) {
            float a[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] = v[(i + j) * both];
#pragma unroll
            for (int j = 0; j < 8; ++j) s += a[j];
        }
        for (; i < i1; ++i) s += v[i * both];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave || c >= both) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    void *const out = c < p.cols ? p.dscale : p.dbias;
    const int64_t at = c < p.cols ? c : c - p.cols;
    if (p.param_f32) ((float *)out)[at] = s;
    else ((typename T::raw_t *)out)[at] = to_bits<T>(s);
}

// ------------------------------------------- rows past 32768 columns

template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_wide(NormParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ float red[32];
    const int t = threadIdx.x;
    const float inv_n = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const raw_t *x = (const raw_t *)p.X + r * p.x_stride;
        raw_t *y = (raw_t *)p.Y + r * p.y_stride;
        float s = 0.0f;
        for (int c = t; c < p.cols; c += 1024) s += T::from_raw(x[c]);
        const float mean = row_total<1024>(s, red) / (float)p.cols;
        s = 0.0f;
        for (int c = t; c < p.cols; c += 1024) {
            const float d = T::from_raw(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float inv = 1.0f / sqrtf(row_total<1024>(s, red) * inv_n + p.epsilon);
        for (int c = t; c < p.cols; c += 1024) {
            const float xh = (T::from_raw(x[c]) - mean) * inv;
            const float b = p.bias ? param<T>(p.bias, c, p.param_f32) : 0.0f;
            y[c] = to_bits<T>(fmaf(xh, param<T>(p.scale, c, p.param_f32), b));
        }
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.inv_std) p.inv_std[r] = inv;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(1024) void layer_norm_dx_wide(NormParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ float red[32];
    const int t = threadIdx.x;
    const float inv_n = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const raw_t *x = (const raw_t *)p.X + r * p.x_stride;
        const raw_t *dy = (const raw_t *)p.dY + r * p.dy_stride;
        raw_t *dx = (raw_t *)p.dX + r * p.dx_stride;
        const float mean = p.mean[r], inv = p.inv_std[r];
        float a = 0.0f, b = 0.0f;
        for (int c = t; c < p.cols; c += 1024) {
            const float g = T::from_raw(dy[c]) * param<T>(p.scale, c, p.param_f32);
            a += g;
            b = fmaf(g, (T::from_raw(x[c]) - mean) * inv, b);
        }
        row_totals<1024>(a, b, red);
        a *= inv_n;
        b *= inv_n;
        for (int c = t; c < p.cols; c += 1024) {
            const float g = T::from_raw(dy[c]) * param<T>(p.scale, c, p.param_f32);
            const float xh = (T::from_raw(x[c]) - mean) * inv;
            dx[c] = to_bits<T>(inv * (g - a - xh * b));
        }
    }
}

// Sums of one part's rows: block (c, part) owns 256 columns.
template <typename T>
__global__ __launch_bounds__(256) void layer_norm_params_wide(NormParams p) {
    typedef typename T::raw_t raw_t;
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    const int part = blockIdx.y;
    const int64_t r0 = p.rows * part / p.parts, r1 = p.rows * (part + 1) / p.parts;
    float ds = 0.0f, db = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float dy = T::from_raw(((const raw_t *)p.dY)[r * p.dy_stride + c]);
        const float x = T::from_raw(((const raw_t *)p.X)[r * p.x_stride + c]);
        ds = fmaf(dy, (x - p.mean[r]) * p.inv_std[r], ds);
        db += dy;
    }
    p.partial[((int64_t)part * 2) * p.cols + c] = ds;
    p.partial[((int64_t)part * 2 + 1) * p.cols + c] = db;
}

// --------------------------------------------------------------- launches

constexpr int kWidest = 32768;       // columns of a row that stays in registers

// Rows of a block at a time, and blocks that run at once (registers allow two to
// eight a compute unit).
int block_rows(int64_t cols) { return cols <= 64 ? 32 : cols <= 256 ? 8 : cols <= 2048 ? 4 : 1; }
int forward_blocks(int64_t cols) { return cols <= 512 ? 2048 : cols <= 1024 ? 1536 : 1024; }
int backward_blocks(int64_t cols) { return cols <= 512 ? 1536 : cols <= 1024 ? 768 : 512; }

template <typename T, int NT, int E>
void rows_form(const NormParams &p, bool backward, hipStream_t stream) {
    constexpr int B = block_threads(NT);
    if (backward) {
        const dim3 grid((unsigned)p.parts);
        if (p.vec) hipLaunchKernelGGL((layer_norm_backward_rows<T, NT, E, true>), grid, dim3(B), 0, stream, p);
        else hipLaunchKernelGGL((layer_norm_backward_rows<T, NT, E, false>), grid, dim3(B), 0, stream, p);
        return;
    }
    const int64_t blocks = (p.rows + B / NT - 1) / (B / NT), most = forward_blocks(p.cols);
    const dim3 grid((unsigned)(blocks < most ? blocks : most));
    if (p.vec) hipLaunchKernelGGL((layer_norm_rows<T, NT, E, true>), grid, dim3(B), 0, stream, p);
    else hipLaunchKernelGGL((layer_norm_rows<T, NT, E, false>), grid, dim3(B), 0, stream, p);
}

template <typename T>
int rows_launch(const NormParams &p, bool backward, hipStream_t stream) {
    if (p.cols <= 64) rows_form<T, 8, 8>(p, backward, stream);
    else if (p.cols <= 256) rows_form<T, 32, 8>(p, backward, stream);
    else if (p.cols <= 512) rows_form<T, 64, 8>(p, backward, stream);
    else if (p.cols <= 1024) rows_form<T, 64, 16>(p, backward, stream);
    else if (p.cols <= 2048) rows_form<T, 64, 32>(p, backward, stream);
    else if (p.cols <= 4096) rows_form<T, 256, 16>(p, backward, stream);
    else if (p.cols <= 8192) rows_form<T, 256, 32>(p, backward, stream);
    else if (p.cols <= 16384) rows_form<T, 1024, 16>(p, backward, stream);
    else rows_form<T, 1024, 32>(p, backward, stream);
    return (int)hipGetLastError();
}

template <typename T>
int forward(const NormParams &p, hipStream_t stream) {
    if (p.cols <= kWidest) return rows_launch<T>(p, false, stream);
    hipLaunchKernelGGL(layer_norm_wide<T>, dim3((unsigned)(p.rows < 1024 ? p.rows : 1024)), dim3(1024), 0, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int backward(const NormParams &p, hipStream_t stream) {
    if (p.rows > 0 && p.cols <= kWidest) {
        if (const int e = rows_launch<T>(p, true, stream)) return e;
    } else if (p.rows > 0) {
        const dim3 grid((unsigned)(p.rows < 1024 ? p.rows : 1024));
        hipLaunchKernelGGL(layer_norm_dx_wide<T>, grid, dim3(1024), 0, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
        if (p.dscale) {
            const dim3 parts((unsigned)((p.cols + 255) / 256), (unsigned)p.parts);
            hipLaunchKernelGGL(layer_norm_params_wide<T>, parts, dim3(256), 0, stream, p);
            if (const int e = (int)hipGetLastError()) return e;
        }
    }
    if (!p.dscale) return 0;
    const dim3 grid((unsigned)((2 * (int64_t)p.cols + 63) / 64));
    hipLaunchKernelGGL(layer_norm_param_sums<T>, grid, dim3(1024), 0, stream, p);
    return (int)hipGetLastError();
}

}  // namespace

// As many parts as run at once, fewer where their sums would pass 32 MiB.
int layer_norm_parts(int64_t rows, int64_t cols) {
    if (rows == 0) return 0;
    int64_t n = (rows + block_rows(cols) - 1) / block_rows(cols);
    const int64_t most = (int64_t(1) << 22) / cols;
    if (n > backward_blocks(cols)) n = backward_blocks(cols);
    if (n > most) n = most < 1 ? 1 : most;
    return (int)n;
}

int launch_layer_norm(const NormParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return forward<F32>(p, stream);
    if (dtype == 1) return forward<F16>(p, stream);
    return forward<BF16>(p, stream);
}

int launch_layer_norm_backward(const NormParams &p, int dtype, hipStream_t stream) {
    if (dtype == 0) return backward<F32>(p, stream);
    if (dtype == 1) return backward<F16>(p, stream);
    return backward<BF16>(p, stream);
}

}  // namespace gs
