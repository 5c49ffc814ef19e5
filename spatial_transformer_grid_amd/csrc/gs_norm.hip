// gs_norm.hip -- layer normalisation, forward and backward.
//
// Forward: mean, then the sum of (x - mean)^2 (two passes over the row, so
// that a large mean does not cancel).  Backward, with xh = (x - mean) inv_std
// and g = dy scale: dx = inv_std (g - mean(g) - xh mean(g xh)); dscale and
// dbias are sums over rows, made in parts (one per block, its rows in order)
// and added up by a second kernel, so that the order is fixed.
#include "gs_tokens.hpp"

namespace gs {

namespace {

__device__ __forceinline__ float wave_total(float v) {
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

// Sum over the 256 threads of a block; `red` holds 4 floats.
__device__ __forceinline__ float block_total(float v, float *red) {
    v = wave_total(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <typename T>
__device__ __forceinline__ float param(const void *v, int64_t i, int f32) {
    if (f32) return ((const float *)v)[i];
    return T::from_raw(((const typename T::raw_t *)v)[i]);
}

// One block per row, the row read three times (from the cache after the first).
template <typename T>
__global__ __launch_bounds__(256) void layer_norm_rows(NormParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ float red[4];
    const int t = threadIdx.x;
    const float inv_n = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const raw_t *x = (const raw_t *)p.X + r * p.x_stride;
        raw_t *y = (raw_t *)p.Y + r * p.y_stride;
        float s = 0.0f;
        for (int c = t; c < p.cols; c += 256) s += T::from_raw(x[c]);
        const float mean = block_total(s, red) * inv_n;
        s = 0.0f;
        for (int c = t; c < p.cols; c += 256) {
            const float d = T::from_raw(x[c]) - mean;
            s = fmaf(d, d, s);
        }
        const float inv = 1.0f / sqrtf(block_total(s, red) * inv_n + p.epsilon);
        for (int c = t; c < p.cols; c += 256) {
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
__global__ __launch_bounds__(256) void layer_norm_dx_rows(NormParams p) {
    typedef typename T::raw_t raw_t;
    __shared__ float red[4];
    const int t = threadIdx.x;
    const float inv_n = 1.0f / (float)p.cols;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const raw_t *x = (const raw_t *)p.X + r * p.x_stride;
        const raw_t *dy = (const raw_t *)p.dY + r * p.dy_stride;
        raw_t *dx = (raw_t *)p.dX + r * p.dx_stride;
        const float mean = p.mean[r], inv = p.inv_std[r];
        float a = 0.0f, b = 0.0f;
        for (int c = t; c < p.cols; c += 256) {
            const float g = T::from_raw(dy[c]) * param<T>(p.scale, c, p.param_f32);
            a += g;
            b = fmaf(g, (T::from_raw(x[c]) - mean) * inv, b);
        }
        a = block_total(a, red) * inv_n;
        b = block_total(b, red) * inv_n;
        for (int c = t; c < p.cols; c += 256) {
            const float g = T::from_raw(dy[c]) * param<T>(p.scale, c, p.param_f32);
            const float xh = (T::from_raw(x[c]) - mean) * inv;
            dx[c] = to_bits<T>(inv * (g - a - xh * b));
        }
    }
}

// Partial sums of dscale and dbias: block (c, part) owns 256 columns and the
// rows of one part.
template <typename T>
__global__ __launch_bounds__(256) void layer_norm_dparam_parts(NormParams p) {
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

template <typename T>
__global__ __launch_bounds__(256) void layer_norm_dparam_sum(NormParams p) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float s[2] = {0.0f, 0.0f};
    for (int part = 0; part < p.parts; ++part)
        for (int i = 0; i < 2; ++i) s[i] += p.partial[((int64_t)part * 2 + i) * p.cols + c];
    void *const out[2] = {p.dscale, p.dbias};
    for (int i = 0; i < 2; ++i) {
        if (p.param_f32) ((float *)out[i])[c] = s[i];
        else ((typename T::raw_t *)out[i])[c] = to_bits<T>(s[i]);
    }
}

template <typename T>
int forward(const NormParams &p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.rows < 65536 ? p.rows : 65536));
    hipLaunchKernelGGL(layer_norm_rows<T>, grid, dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

template <typename T>
int backward(const NormParams &p, hipStream_t stream) {
    const unsigned cb = (unsigned)((p.cols + 255) / 256);
    if (p.rows > 0) {
        const dim3 grid((unsigned)(p.rows < 65536 ? p.rows : 65536));
        hipLaunchKernelGGL(layer_norm_dx_rows<T>, grid, dim3(256), 0, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    if (!p.dscale) return 0;
    if (p.parts > 0) {
        hipLaunchKernelGGL(layer_norm_dparam_parts<T>, dim3(cb, (unsigned)p.parts), dim3(256), 0, stream, p);
        if (const int e = (int)hipGetLastError()) return e;
    }
    hipLaunchKernelGGL(layer_norm_dparam_sum<T>, dim3(cb), dim3(256), 0, stream, p);
    return (int)hipGetLastError();
}

}  // namespace

int layer_norm_parts(int64_t rows, int64_t cols) {
    (void)cols;
    return (int)(rows < 64 ? rows : 64);
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
