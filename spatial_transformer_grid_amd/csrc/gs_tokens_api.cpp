// gs_tokens_api.cpp -- C ABI of the token operators (gsample_tokens.h):
// argument validation and kernel dispatch.  As in gs_api.cpp every check runs
// before any launch, and nothing is allocated or kept.
#include "gsample_tokens.h"
#include "gs_tokens.hpp"

#include <math.h>
#include <stdint.h>

namespace {

constexpr int64_t kInt32Max = 0x7fffffff;
// Blocks of a launch: of 256 threads, whose number has to stay below 2^32, in
// whole eighths (one an XCD).  Beside the table's sums there are at most 8192
// blocks that add up parts (of 256 blocks of 128 rows of 128 columns, dK and dV).
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 8;
constexpr int64_t kMaxTableSums = kMaxBlocks - 8192;
constexpr int64_t kMaxPosition = int64_t(1) << 29;  // positions and their differences fit 32 bits
constexpr int64_t kMaxHeads = int64_t(1) << 20;
constexpr uintptr_t kWsAlign = 256;

bool data_dtype(int d) { return d == GS_F32 || d == GS_F16 || d == GS_BF16; }
int dtype_bytes(int d) { return d == GS_F32 ? 4 : 2; }
int64_t round_ws(int64_t b) { return (b + 255) / 256 * 256; }
int hip_status(int rc) { return rc == 0 ? GS_OK : GS_ERR_HIP; }

// A row stride that keeps 16-byte rows aligned, and a pointer that is.
bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }

// Threshold of the 16-bit numbers; false when the ratio is out of range.
bool drop_threshold(float ratio, uint32_t *threshold, float *keep_scale) {
    if (!(ratio >= 0.0f && ratio < 1.0f)) return false;
    const double t = floor((double)ratio * 65536.0 + 0.5);
    if (t > 65535.0) return false;
    *threshold = (uint32_t)t;
    *keep_scale = (float)(65536.0 / (65536.0 - t));
    return true;
}

int norm_extents(int dtype, int param_dtype, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return GS_ERR_SHAPE;
    if (!data_dtype(dtype) || (param_dtype != dtype && param_dtype != GS_F32)) return GS_ERR_DTYPE;
    if (rows > 0 && cols == 0) return GS_ERR_SHAPE;
    if (cols > (int64_t(1) << 24) || rows > kInt32Max) return GS_ERR_TOO_LARGE;
    return GS_OK;
}

// First distances of the buckets of one side, and the last of them.  Bucket
// e + j begins at the smallest d with (d/e)^(n-e) >= (max_distance/e)^j,
// compared through logarithms in double.  Equal sides are off by roundings, less
// than 2e-12 (at most 256 log 1024, from logarithms good to 1e-16 of
// themselves); sides that differ do so by 5.03e-11 at least (435^11 10^9 against
// 1006^9 10^11, the closest of all borders up to 1024, the next past 1e-9).
int bucket_starts(int num_buckets, int max_distance, int bidirectional, uint16_t *starts, int *side) {
    if (bidirectional != 0 && bidirectional != 1) return GS_ERR_ATTR;
    if (num_buckets < 2 || num_buckets > gs::kMaxBuckets) return GS_ERR_ATTR;
    if (bidirectional && (num_buckets < 4 || num_buckets % 2)) return GS_ERR_ATTR;
    const int n = bidirectional ? num_buckets / 2 : num_buckets, e = n / 2;
    if (max_distance <= e) return GS_ERR_ATTR;
    *side = n;
    for (int i = 0; i < e; ++i) starts[i] = (uint16_t)i;
    const double whole = log((double)max_distance / e);
    int d = e;
    for (int j = 0; j < n - e; ++j) {
        const double need = whole * j;
        while (d <= gs::kMaxBorder && log((double)d / e) * (n - e) < need - 1e-11) ++d;
        if (d > gs::kMaxBorder) return GS_ERR_TOO_LARGE;
        starts[e + j] = (uint16_t)d;
    }
    return GS_OK;
}

bool strides_ok(const int64_t *s) {
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0) return false;
    return true;
}

bool strides_vec(const int64_t *s, int epc) {
    for (int i = 0; i < 3; ++i)
        if (s[i] % epc) return false;
    return true;
}

// Whether rows of an output of these extents lie apart: along an axis of more
// than one element by at least a row.
bool rows_apart(const int64_t *s, int64_t batch, int64_t heads, int64_t len, int64_t dim) {
    const int64_t n[3] = {batch, heads, len};
    if (batch * heads * len == 0) return true;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] < dim) return false;
    return true;
}

// Validation shared by the forward and backward calls; fills all of p but
// the pointers.
int attention_setup(const gs_attention_desc *d, bool backward, gs::AttnParams &p) {
    if (!d) return GS_ERR_NULL;
    if (!data_dtype(d->dtype)) return GS_ERR_DTYPE;
    if (d->num_buckets != 0 && d->table_dtype != d->dtype && d->table_dtype != GS_F32) return GS_ERR_DTYPE;
    if (d->batch < 0 || d->q_heads < 0 || d->kv_heads < 0 || d->q_len < 0 || d->kv_len < 0) return GS_ERR_SHAPE;
    if (d->head_dim < 1) return GS_ERR_SHAPE;
    if (d->kv_heads == 0 ? d->q_heads != 0 : d->q_heads % d->kv_heads != 0) return GS_ERR_SHAPE;
    if (!strides_ok(d->q_stride) || !strides_ok(d->k_stride) || !strides_ok(d->v_stride) || !strides_ok(d->o_stride))
        return GS_ERR_SHAPE;
    if (backward && (!strides_ok(d->do_stride) || !strides_ok(d->dq_stride) || !strides_ok(d->dk_stride) ||
                     !strides_ok(d->dv_stride)))
        return GS_ERR_SHAPE;
    if (!isfinite(d->scale)) return GS_ERR_ATTR;
    if ((d->causal != 0 && d->causal != 1) || (d->q_from_end != 0 && d->q_from_end != 1)) return GS_ERR_ATTR;
    p = gs::AttnParams{};
    if (!drop_threshold(d->ratio, &p.threshold, &p.keep_scale)) return GS_ERR_ATTR;
    if (d->num_buckets != 0) {
        const int rc = bucket_starts(d->num_buckets, d->max_distance, d->bidirectional, p.starts, &p.side);
        if (rc != GS_OK) return rc;
        p.buckets = d->num_buckets;
        p.bidirectional = d->bidirectional;
        p.border = p.starts[p.side - 1];
        p.lut = gs::lut_entries(p.border, p.bidirectional);
        p.table_f32 = d->table_dtype == GS_F32;
    }
    if (d->head_dim > 128 || d->q_len > kMaxPosition || d->kv_len > kMaxPosition || d->q_position > kMaxPosition ||
        d->q_position < -kMaxPosition || d->batch > kInt32Max || d->q_heads > kMaxHeads || d->kv_heads > kMaxHeads)
        return GS_ERR_TOO_LARGE;
    const int64_t tiles = (d->q_len + 31) / 32, ktiles = (d->kv_len + 31) / 32;
    const int64_t pairs = d->batch * d->q_heads, kv_pairs = d->batch * d->kv_heads;
    if (pairs > kMaxBlocks || pairs * tiles > kMaxBlocks || kv_pairs > kMaxBlocks || kv_pairs * ktiles > kMaxBlocks)
        return GS_ERR_TOO_LARGE;
    const int64_t B = d->batch, D = d->head_dim;
    if (backward ? !rows_apart(d->dq_stride, B, d->q_heads, d->q_len, D) ||
                       !rows_apart(d->dk_stride, B, d->kv_heads, d->kv_len, D) ||
                       !rows_apart(d->dv_stride, B, d->kv_heads, d->kv_len, D)
                 : !rows_apart(d->o_stride, B, d->q_heads, d->q_len, D))
        return GS_ERR_SHAPE;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = d->q_stride[i];
        p.ks[i] = d->k_stride[i];
        p.vs[i] = d->v_stride[i];
        p.os[i] = d->o_stride[i];
        p.dos[i] = d->do_stride[i];
        p.dqs[i] = d->dq_stride[i];
        p.dks[i] = d->dk_stride[i];
        p.dvs[i] = d->dv_stride[i];
    }
    p.B = (int)d->batch;
    p.H = (int)d->q_heads;
    p.Hkv = (int)d->kv_heads;
    p.G = d->kv_heads ? (int)(d->q_heads / d->kv_heads) : 0;
    p.Lq = (int)d->q_len;
    p.Lk = (int)d->kv_len;
    p.D = (int)d->head_dim;
    p.causal = d->causal;
    p.from_end = d->q_from_end;
    p.first = (int)d->q_position;
    p.scale = d->scale;
    p.scale2 = (float)((double)d->scale * 1.4426950408889634074);
    p.seed_lo = (uint32_t)d->seed;
    p.seed_hi = (uint32_t)(d->seed >> 32);
    p.call = d->call;
    p.fold = p.keep_scale < gs::kMaxFold ? p.keep_scale : gs::kMaxFold;
    p.fold_log2 = (float)log2((double)p.fold);
    p.rest = p.keep_scale / p.fold;
    p.units = (int)pairs;
    p.tiles = (int)tiles;
    const int epc = 16 / dtype_bytes(d->dtype);
    p.vec = p.D % epc == 0 && strides_vec(p.qs, epc) && strides_vec(p.ks, epc) && strides_vec(p.vs, epc) &&
            strides_vec(p.os, epc);
    if (backward)
        p.vec = p.vec && strides_vec(p.dos, epc) && strides_vec(p.dqs, epc) && strides_vec(p.dks, epc) &&
                strides_vec(p.dvs, epc);
    return GS_OK;
}

// Rows of a tile that an asynchronous load reaches from its first by a 32-bit
// byte offset.
bool stride_async(int64_t s) { return s <= (int64_t(1) << 22); }

// Workspace of a backward call: four numbers a query, in whole tiles of 64, and with
// a table its shift; the key tiles' sums for the table; the parts' sums of dK and
// dV.  Each 256-byte aligned.
struct BackwardSpace {
    int64_t part, split, bytes;
};

BackwardSpace backward_space(const gs::AttnParams &p, int dtype) {
    const gs::AttnPlan kv = gs::plan_backward_kv(p, dtype);
    BackwardSpace s;
    s.part = round_ws((int64_t)p.B * p.H * ((p.Lq + 63) / 64) * 64 * (p.buckets ? 20 : 16));
    s.split = s.part + round_ws((int64_t)p.B * p.H * kv.tiles * kv.splits * p.buckets * 4);
    s.bytes = s.split + round_ws(kv.split_floats * 4);
    return s;
}

}  // namespace

extern "C" {

int gs_layer_norm(const void *X, int dtype, int64_t rows, int64_t cols, int64_t x_stride, const void *scale,
                  const void *bias, int param_dtype, float epsilon, void *Y, int64_t y_stride, float *mean,
                  float *inv_std, void *stream) {
    const int rc = norm_extents(dtype, param_dtype, rows, cols);
    if (rc != GS_OK) return rc;
    if (x_stride < 0 || (rows > 1 && y_stride < cols)) return GS_ERR_SHAPE;
    if (!(epsilon >= 0.0f) || !isfinite(epsilon)) return GS_ERR_ATTR;
    if (rows == 0) return GS_OK;
    if (!X || !scale || !Y) return GS_ERR_NULL;
    gs::NormParams p = {};
    p.X = X;
    p.scale = scale;
    p.bias = bias;
    p.Y = Y;
    p.mean = mean;
    p.inv_std = inv_std;
    p.rows = rows;
    p.cols = (int)cols;
    p.x_stride = x_stride;
    p.y_stride = y_stride;
    p.epsilon = epsilon;
    p.param_f32 = param_dtype == GS_F32;
    const int epc = 16 / dtype_bytes(dtype);
    p.vec = cols % 8 == 0 && x_stride % epc == 0 && y_stride % epc == 0 && aligned16(X) && aligned16(Y) &&
            aligned16(scale) && aligned16(bias);
    return hip_status(gs::launch_layer_norm(p, dtype, (hipStream_t)stream));
}

int gs_layer_norm_backward_workspace_size(int64_t rows, int64_t cols, int64_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    const int rc = norm_extents(GS_F32, GS_F32, rows, cols);
    if (rc != GS_OK) return rc;
    *bytes = round_ws((int64_t)gs::layer_norm_parts(rows, cols) * 2 * cols * 4);
    return GS_OK;
}

int gs_layer_norm_backward(const void *dY, const void *X, int dtype, int64_t rows, int64_t cols, int64_t dy_stride,
                           int64_t x_stride, const void *scale, int param_dtype, const float *mean,
                           const float *inv_std, void *dX, int64_t dx_stride, void *dscale, void *dbias,
                           void *workspace, int64_t workspace_bytes, void *stream) {
    const int rc = norm_extents(dtype, param_dtype, rows, cols);
    if (rc != GS_OK) return rc;
    if (dy_stride < 0 || x_stride < 0 || (rows > 1 && dx_stride < cols)) return GS_ERR_SHAPE;
    if (workspace_bytes < 0) return GS_ERR_ATTR;
    if (cols == 0) return GS_OK;
    if ((dscale == nullptr) != (dbias == nullptr)) return GS_ERR_NULL;
    if (rows > 0 && (!dY || !X || !scale || !mean || !inv_std || !dX)) return GS_ERR_NULL;
    if (rows == 0 && !dscale) return GS_OK;
    gs::NormParams p = {};
    p.parts = gs::layer_norm_parts(rows, cols);
    const int64_t need = (int64_t)p.parts * 2 * cols * 4;
    if (dscale && need > 0) {
        if (!workspace) return GS_ERR_NULL;
        if (workspace_bytes < need || (uintptr_t)workspace % kWsAlign) return GS_ERR_ATTR;
    }
    p.X = X;
    p.dY = dY;
    p.scale = scale;
    p.dX = dX;
    p.mean = const_cast<float *>(mean);
    p.inv_std = const_cast<float *>(inv_std);
    p.rows = rows;
    p.cols = (int)cols;
    p.x_stride = x_stride;
    p.dy_stride = dy_stride;
    p.dx_stride = dx_stride;
    p.param_f32 = param_dtype == GS_F32;
    p.dscale = dscale;
    p.dbias = dbias;
    p.partial = (float *)workspace;
    const int epc = 16 / dtype_bytes(dtype);
    p.vec = cols % 8 == 0 && x_stride % epc == 0 && dy_stride % epc == 0 && dx_stride % epc == 0 && aligned16(X) &&
            aligned16(dY) && aligned16(dX) && aligned16(scale);
    return hip_status(gs::launch_layer_norm_backward(p, dtype, (hipStream_t)stream));
}

int gs_dropout(const void *X, int dtype, int64_t count, const void *residual, float ratio, uint64_t seed,
               uint32_t call, void *Y, void *stream) {
    if (count < 0) return GS_ERR_SHAPE;
    if (!data_dtype(dtype)) return GS_ERR_DTYPE;
    gs::DropoutParams p = {};
    if (!drop_threshold(ratio, &p.threshold, &p.keep_scale)) return GS_ERR_ATTR;
    if (count > (int64_t(1) << 40)) return GS_ERR_TOO_LARGE;
    if (count == 0) return GS_OK;
    if (!X || !Y) return GS_ERR_NULL;
    p.X = X;
    p.residual = residual;
    p.Y = Y;
    p.count = count;
    p.seed_lo = (uint32_t)seed;
    p.seed_hi = (uint32_t)(seed >> 32);
    p.call = call;
    p.vec = aligned16(X) && aligned16(residual) && aligned16(Y);
    return hip_status(gs::launch_dropout(p, dtype, (hipStream_t)stream));
}

int gs_relative_bucket(int64_t r, int num_buckets, int max_distance, int bidirectional, int *bucket) {
    if (!bucket) return GS_ERR_NULL;
    uint16_t starts[gs::kMaxBuckets];
    int side = 0;
    const int rc = bucket_starts(num_buckets, max_distance, bidirectional, starts, &side);
    if (rc != GS_OK) return rc;
    const uint64_t away = r < 0 ? 0 - (uint64_t)r : (bidirectional ? (uint64_t)r : 0);
    int n = side - 1;
    while (n > 0 && starts[n] > away) --n;
    *bucket = n + (bidirectional && r > 0 ? side : 0);
    return GS_OK;
}

int gs_attention_workspace_size(const gs_attention_desc *desc, int64_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    gs::AttnParams p;
    const int rc = attention_setup(desc, false, p);
    if (rc != GS_OK) return rc;
    *bytes = p.units * (int64_t)p.tiles == 0 ? 0 : round_ws(gs::plan_forward(p, desc->dtype, true).split_floats * 4);
    return GS_OK;
}

int gs_attention(const gs_attention_desc *desc, const void *Q, const void *K, const void *V, const int32_t *lengths,
                 const void *table, void *O, float *lse, void *workspace, int64_t workspace_bytes, void *stream) {
    gs::AttnParams p;
    const int rc = attention_setup(desc, false, p);
    if (rc != GS_OK) return rc;
    if (workspace_bytes < 0 || (workspace && (uintptr_t)workspace % kWsAlign)) return GS_ERR_ATTR;
    if (p.units == 0 || p.tiles == 0) return GS_OK;
    if (!Q || !O || (p.Lk > 0 && (!K || !V)) || (p.buckets && !table)) return GS_ERR_NULL;
    p.q = Q;
    p.k = K;
    p.v = V;
    p.lengths = lengths;
    p.table = table;
    p.o = O;
    p.lse = lse;
    p.vec = p.vec && aligned16(Q) && aligned16(K) && aligned16(V) && aligned16(O);
    p.async = p.vec && stride_async(p.ks[2]) && stride_async(p.vs[2]);
    const int64_t need = gs::plan_forward(p, desc->dtype, true).split_floats * 4;
    if (workspace && workspace_bytes >= need) p.split = (float *)workspace;
    return hip_status(gs::launch_attention(p, desc->dtype, (hipStream_t)stream));
}

int gs_attention_backward_workspace_size(const gs_attention_desc *desc, int64_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    gs::AttnParams p;
    const int rc = attention_setup(desc, true, p);
    if (rc != GS_OK) return rc;
    *bytes = backward_space(p, desc->dtype).bytes;
    return GS_OK;
}

int gs_attention_backward(const gs_attention_desc *desc, const void *dO, const void *Q, const void *K, const void *V,
                          const void *O, const float *lse, const int32_t *lengths, const void *table, void *dQ,
                          void *dK, void *dV, void *dtable, void *workspace, int64_t workspace_bytes, void *stream) {
    gs::AttnParams p;
    const int rc = attention_setup(desc, true, p);
    if (rc != GS_OK) return rc;
    if (workspace_bytes < 0) return GS_ERR_ATTR;
    if (dtable && p.buckets * (int64_t)p.H > kMaxTableSums) return GS_ERR_TOO_LARGE;
    const bool queries = p.units > 0 && p.tiles > 0, keys = (int64_t)p.B * p.Hkv * p.Lk > 0;
    if (queries && (!dO || !Q || !O || !lse || !dQ)) return GS_ERR_NULL;
    if (keys && (!K || !V || !dK || !dV)) return GS_ERR_NULL;
    if (p.buckets && queries && !table) return GS_ERR_NULL;
    const BackwardSpace space = backward_space(p, desc->dtype);
    const int64_t need = space.bytes;
    if (need > 0) {
        if (!workspace) return GS_ERR_NULL;
        if (workspace_bytes < need || (uintptr_t)workspace % kWsAlign) return GS_ERR_ATTR;
    }
    p.d_o = dO;
    p.q = Q;
    p.k = K;
    p.v = V;
    p.o_in = O;
    p.lse = const_cast<float *>(lse);
    p.lengths = lengths;
    p.table = table;
    p.dq = dQ;
    p.dk = dK;
    p.dv = dV;
    p.dtable = p.buckets ? dtable : nullptr;
    p.rows = (float *)workspace;
    p.part = p.dtable && workspace ? (float *)((char *)workspace + space.part) : nullptr;
    p.split = (float *)((char *)workspace + space.split);
    p.vec = p.vec && aligned16(Q) && aligned16(K) && aligned16(V) && aligned16(O) && aligned16(dO) && aligned16(dQ) &&
            aligned16(dK) && aligned16(dV);
    p.async = p.vec && stride_async(p.ks[2]) && stride_async(p.vs[2]) && stride_async(p.qs[2]) &&
              stride_async(p.dos[2]);
    return hip_status(gs::launch_attention_backward(p, desc->dtype, (hipStream_t)stream));
}

}  // extern "C"
