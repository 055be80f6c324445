// abi.cpp -- the extern "C" entry points declared in include/loom.h.
//
// Every entry point validates its arguments on the host (sizes, then
// pointers, then alignment), evaluates its kernel's launch configuration
// through the same table embeddings use, and enqueues the kernel on the
// caller's stream.  Nothing is launched when there is nothing to compute or
// when a check fails.
#include <stdint.h>

#include "internal.hpp"

namespace {

bool misaligned(const void *p, uintptr_t a) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Runs a kernel launcher and maps its result.  The thread's last HIP error
// is cleared first, so LOOM_ERR_DEVICE reports this launch only, not an
// error some earlier, unrelated HIP call left behind.
template <typename Launch>
int launch(Launch &&f) {
    (void)hipGetLastError();
    return f() == hipSuccess ? LOOM_OK : LOOM_ERR_DEVICE;
}

constexpr int64_t kMaxRows = 0x7FFFFFFF;        // row / segment counts index a 1-D grid
constexpr int64_t kMaxTileRows = int64_t(1) << 26;
constexpr int64_t kMaxTotalRows = int64_t(1) << 40;
constexpr int64_t kMaxSegmentCols = int64_t(1) << 20;
constexpr int64_t kMaxCopy = (int64_t(1) << 32) - 256;  // one work-item per element, below 2^32 work-items
constexpr int64_t kMaxOutputs = int64_t(0x7FFFFFFF) * 255;

}  // namespace

extern "C" const char *loom_status_string(int status) {
    switch (status) {
        case LOOM_OK: return "ok";
        case LOOM_ERR_NULL: return "a required pointer is NULL";
        case LOOM_ERR_RANGE: return "a size or count is outside its documented range";
        case LOOM_ERR_ALIGN: return "a pointer or stride is not aligned as documented";
        case LOOM_ERR_SHAPE: return "inconsistent shape";
        case LOOM_ERR_UNKNOWN_EXPORT: return "no kernel exports this name";
        case LOOM_ERR_TOKEN: return "invalid launch-config token or workload arity";
        case LOOM_ERR_DEVICE: return "the HIP runtime refused the launch";
        default: return "unknown status";
    }
}

extern "C" int loom_version(void) { return 100; }

extern "C" int loom_copy_f32(const float *in, float *out, int64_t n, void *stream) {
    if (n < 0 || n > kMaxCopy) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[1] = {n};
    if (int st = loom::evaluate_launch(loom::kCopyF32, w, &cfg)) return st;
    if (n == 0) return LOOM_OK;
    if (!in || !out) return LOOM_ERR_NULL;
    if (misaligned(in, 4) || misaligned(out, 4)) return LOOM_ERR_ALIGN;
    return launch([&] { return loom::launch_copy_f32(cfg, in, out, n, (hipStream_t)stream); });
}

extern "C" int loom_row_sum_tiles(const float *values, int64_t rows_alloc, int64_t count, const float *initial,
                                  float *sums, int32_t *final_row, int32_t *tail_count, void *stream) {
    if (rows_alloc < 0 || rows_alloc > kMaxTileRows || count < 0 || count > rows_alloc) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[1] = {count};
    if (int st = loom::evaluate_launch(loom::kRowSumTiles, w, &cfg)) return st;
    if (!sums || !final_row || !tail_count || (!values && rows_alloc > 0)) return LOOM_ERR_NULL;
    if (misaligned(values, 4) || misaligned(initial, 4) || misaligned(sums, 4) || misaligned(final_row, 4) ||
        misaligned(tail_count, 4))
        return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_row_sum_tiles(cfg, values, (int)count, initial, sums, final_row, tail_count,
                                          (hipStream_t)stream);
    });
}

extern "C" int loom_row_sums(const float *x, int64_t rows, int64_t cols, int64_t row_stride, float *out,
                             void *stream) {
    if (rows < 0 || rows > kMaxRows || cols < 0 || cols > kMaxRows) return LOOM_ERR_RANGE;
    if (row_stride < cols) return LOOM_ERR_SHAPE;
    if (rows > 0 && row_stride > (INT64_MAX / 4) / rows) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[2] = {rows, cols};
    if (int st = loom::evaluate_launch(loom::kRowSums, w, &cfg)) return st;
    if (rows == 0) return LOOM_OK;
    if (!out || (!x && cols > 0)) return LOOM_ERR_NULL;
    if (misaligned(x, 4) || misaligned(out, 4)) return LOOM_ERR_ALIGN;
    return launch(
        [&] { return loom::launch_row_sums(cfg, x, (int)rows, (int)cols, row_stride, out, (hipStream_t)stream); });
}

namespace {

// The checks of both segment-sum entry points, in the documented order; on
// LOOM_OK with *nothing false, cfg holds the launch geometry.
int segment_sums_checks(const float *x, int64_t total_rows, const int64_t *offsets, int64_t segments, int64_t cols,
                        const float *out, const int32_t *tail_counts, loom_launch_config *cfg, bool *nothing) {
    *nothing = true;
    if (segments < 0 || segments > kMaxRows - 1 || cols < 0 || cols > kMaxSegmentCols || total_rows < 0 ||
        total_rows > kMaxTotalRows)
        return LOOM_ERR_RANGE;
    const int64_t w[3] = {segments, cols, total_rows};
    if (int st = loom::evaluate_launch(loom::kSegmentSums, w, cfg)) return st;
    if (segments == 0) return LOOM_OK;
    if (!offsets || (!out && cols > 0) || (!x && total_rows > 0 && cols > 0)) return LOOM_ERR_NULL;
    if (misaligned(offsets, 8) || misaligned(x, 4) || misaligned(out, 4) || misaligned(tail_counts, 4))
        return LOOM_ERR_ALIGN;
    *nothing = false;
    return LOOM_OK;
}

}  // namespace

extern "C" int loom_segment_sums(const float *x, int64_t total_rows, const int64_t *offsets, int64_t segments,
                                 int64_t cols, float *out, int32_t *tail_counts, void *stream) {
    loom_launch_config cfg;
    bool nothing;
    if (int st = segment_sums_checks(x, total_rows, offsets, segments, cols, out, tail_counts, &cfg, &nothing))
        return st;
    if (nothing) return LOOM_OK;
    const int64_t workspace_bytes = loom::segment_sums_workspace_bytes(segments, cols, total_rows);
    if (workspace_bytes == 0)
        return launch([&] {
            return loom::launch_segment_sums(cfg, x, total_rows, offsets, segments, (int)cols, out, tail_counts,
                                             nullptr, (hipStream_t)stream);
        });
    // a split launch's partials or a longest-first launch's order index live
    // in stream-ordered memory, taken and given back on the caller's stream
    return launch([&] {
        void *workspace = nullptr;
        hipError_t e = hipMallocAsync(&workspace, (size_t)workspace_bytes, (hipStream_t)stream);
        if (e != hipSuccess) return e;
        e = loom::launch_segment_sums(cfg, x, total_rows, offsets, segments, (int)cols, out, tail_counts, workspace,
                                      (hipStream_t)stream);
        const hipError_t f = hipFreeAsync(workspace, (hipStream_t)stream);
        return e != hipSuccess ? e : f;
    });
}

extern "C" int loom_segment_sums_noalloc(const float *x, int64_t total_rows, const int64_t *offsets,
                                         int64_t segments, int64_t cols, float *out, int32_t *tail_counts,
                                         void *stream) {
    loom_launch_config cfg;
    bool nothing;
    if (int st = segment_sums_checks(x, total_rows, offsets, segments, cols, out, tail_counts, &cfg, &nothing))
        return st;
    if (nothing) return LOOM_OK;
    const int64_t workspace_bytes = loom::segment_sums_workspace_bytes(segments, cols, total_rows);
    if (workspace_bytes > loom::kSegmentSplitMaxBytes) return LOOM_ERR_RANGE;  // beyond the static array
    return launch([&] {
        void *workspace = nullptr;
        if (workspace_bytes > 0) {
            const hipError_t e = loom::segment_scratch(&workspace);
            if (e != hipSuccess) return e;
        }
        return loom::launch_segment_sums(cfg, x, total_rows, offsets, segments, (int)cols, out, tail_counts,
                                         workspace, (hipStream_t)stream);
    });
}

extern "C" int loom_i8_dequant_dot(const int32_t *w, const float *w_scale, const int32_t *x, const float *x_scale,
                                   int64_t rows, int64_t k, int64_t batch, float *out, int32_t *acc, void *stream) {
    if (k < 0 || k > loom::kMaxK || batch < 1 || batch > loom::kMaxBatch || rows < 0 || rows > kMaxRows)
        return LOOM_ERR_RANGE;
    if (k % 4 != 0) return LOOM_ERR_SHAPE;
    loom_launch_config cfg;
    const int64_t wl[3] = {rows, k, batch};
    if (int st = loom::evaluate_launch(loom::kI8DequantDot, wl, &cfg)) return st;
    if (rows == 0) return LOOM_OK;
    if (!w_scale || !out || (k > 0 && (!w || !x))) return LOOM_ERR_NULL;
    if (misaligned(w, 4) || misaligned(x, 4) || misaligned(w_scale, 4) || misaligned(x_scale, 4) ||
        misaligned(out, 4) || misaligned(acc, 4))
        return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_i8_dequant_dot(cfg, w, w_scale, x, x_scale, (int)rows, (int)(k / 4), (int)batch, out,
                                           acc, (hipStream_t)stream);
    });
}

extern "C" int loom_packed_dot(const int32_t *fields, const uint16_t *scales, const float *rhs, int64_t streams,
                               const float *initial, int64_t records, int64_t count, int64_t outputs, float *out,
                               void *stream) {
    if (records < 0 || count < 0 || count > records || count > kMaxRows || outputs < 0 || outputs > kMaxOutputs ||
        streams < 1 || streams > kMaxRows)
        return LOOM_ERR_RANGE;
    if (records > 0 && outputs > INT64_MAX / 4 / records) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[3] = {outputs, count, streams};
    if (int st = loom::evaluate_launch(loom::kPackedDot, w, &cfg)) return st;
    if (outputs == 0) return LOOM_OK;
    if (!out || (count > 0 && (!fields || !scales || !rhs))) return LOOM_ERR_NULL;
    if (misaligned(fields, 4) || misaligned(scales, 2) || misaligned(rhs, 16) || misaligned(initial, 4) ||
        misaligned(out, 4))
        return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_packed_dot(cfg, fields, scales, rhs, (int)streams, initial, (int)count, outputs, out,
                                       (hipStream_t)stream);
    });
}

extern "C" int loom_sum_guarded_rows(const float *values, int64_t rows_alloc, int64_t count, int64_t columns,
                                     int64_t active_lanes, float *sums, void *stream) {
    if (rows_alloc < 0 || rows_alloc > kMaxTileRows || count < 0 || count > rows_alloc || columns < 0 ||
        columns > 4 || active_lanes < 0 || active_lanes > 32)
        return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[1] = {count};
    if (int st = loom::evaluate_launch(loom::kSumGuardedRows, w, &cfg)) return st;
    if (!sums || (!values && rows_alloc > 0)) return LOOM_ERR_NULL;
    if (misaligned(values, 16) || misaligned(sums, 4)) return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_sum_guarded_rows(cfg, values, (int)count, (int)columns, (int)active_lanes, sums,
                                             (hipStream_t)stream);
    });
}

extern "C" int loom_routed_combine(const int32_t *ids, const float *weights, const float *payload, int64_t num_rows,
                                   int64_t tokens, int64_t routes, int64_t hidden, float *out, void *stream) {
    if (tokens < 0 || tokens > kMaxRows || routes < 0 || routes > (int64_t(1) << 20) || hidden < 0 ||
        hidden > (int64_t(1) << 20) || num_rows < 0 || num_rows > kMaxRows)
        return LOOM_ERR_RANGE;
    if (hidden % 4 != 0) return LOOM_ERR_SHAPE;
    loom_launch_config cfg;
    const int64_t w[3] = {tokens, routes, hidden};
    if (int st = loom::evaluate_launch(loom::kRoutedCombine, w, &cfg)) return st;
    if (tokens == 0 || hidden == 0) return LOOM_OK;
    if (!out || (routes > 0 && (!ids || !weights)) || (num_rows > 0 && !payload)) return LOOM_ERR_NULL;
    if (misaligned(ids, 4) || misaligned(weights, 4) || misaligned(payload, 16) || misaligned(out, 16))
        return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_routed_combine(cfg, ids, weights, payload, num_rows, tokens, (int)routes, (int)hidden,
                                           out, (hipStream_t)stream);
    });
}

namespace {

constexpr int64_t element_size(int type) { return type == LOOM_F32 ? 4 : 2; }
bool known_type(int type) { return type == LOOM_F32 || type == LOOM_F16 || type == LOOM_BF16; }
bool known_act(int act) { return act >= LOOM_SILU && act <= LOOM_RELU; }

// The size checks shared by the int8 product, the gated projection and its
// gradients: `stride` is the row stride of the [tokens][rows] matrix.
int product_sizes(loom::ExportId id, int64_t rows, int64_t k, int64_t tokens, int type, int64_t stride,
                  loom_launch_config *cfg) {
    if (k < 0 || k > loom::kMaxK || rows < 0 || rows > kMaxRows || tokens < 0 || tokens > kMaxRows ||
        !known_type(type))
        return LOOM_ERR_RANGE;
    if (k % 4 != 0 || stride < rows) return LOOM_ERR_SHAPE;
    if (tokens > 0 && stride > (INT64_MAX / 4) / tokens) return LOOM_ERR_RANGE;
    const int64_t w[3] = {rows, k, tokens};
    return loom::evaluate_launch(id, w, cfg);
}

}  // namespace

extern "C" int loom_quantize_rows(const void *x, int type, int64_t rows, int64_t cols, int64_t row_stride, int32_t *q,
                                  float *scale, void *stream) {
    if (rows < 0 || rows > kMaxRows || cols < 0 || cols > kMaxRows || !known_type(type)) return LOOM_ERR_RANGE;
    if (cols % 4 != 0 || row_stride < cols) return LOOM_ERR_SHAPE;
    if (rows > 0 && row_stride > (INT64_MAX / 4) / rows) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    const int64_t w[2] = {rows, cols};
    if (int st = loom::evaluate_launch(loom::kQuantizeRows, w, &cfg)) return st;
    if (rows == 0) return LOOM_OK;
    if (!scale || (cols > 0 && (!x || !q))) return LOOM_ERR_NULL;
    if (misaligned(x, element_size(type)) || misaligned(q, 4) || misaligned(scale, 4)) return LOOM_ERR_ALIGN;
    return launch([&] {
        return loom::launch_quantize_rows(cfg, x, type, (int)rows, cols, row_stride, q, scale, (hipStream_t)stream);
    });
}

extern "C" int loom_i8_matmul(const int32_t *w, const float *w_scale, const int32_t *x, const float *x_scale,
                              const float *bias, int64_t rows, int64_t k, int64_t tokens, void *out, int type,
                              int64_t out_stride, void *stream) {
    loom_launch_config cfg;
    if (int st = product_sizes(loom::kI8Matmul, rows, k, tokens, type, out_stride, &cfg)) return st;
    if (rows == 0 || tokens == 0) return LOOM_OK;
    if (!w_scale || !out || (k > 0 && (!w || !x))) return LOOM_ERR_NULL;
    if (misaligned(w, 4) || misaligned(x, 4) || misaligned(w_scale, 4) || misaligned(x_scale, 4) ||
        misaligned(bias, 4) || misaligned(out, element_size(type)))
        return LOOM_ERR_ALIGN;
    const loom::I8Product p = {w,         w_scale,     nullptr,        nullptr, x,   x_scale,   bias,
                               (int)rows, (int)tokens, (int)(k / 4),   0,       out, out_stride};
    return launch([&] { return loom::launch_i8_matmul(cfg, p, type, (hipStream_t)stream); });
}

extern "C" int loom_i8_gated_projection(const int32_t *w_gate, const float *gate_scale, const int32_t *w_up,
                                        const float *up_scale, const int32_t *x, const float *x_scale, int64_t rows,
                                        int64_t k, int64_t tokens, int act, void *out, int type, int64_t out_stride,
                                        void *stream) {
    if (!known_act(act)) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    if (int st = product_sizes(loom::kI8GatedProjection, rows, k, tokens, type, out_stride, &cfg)) return st;
    if (rows == 0 || tokens == 0) return LOOM_OK;
    if (!gate_scale || !up_scale || !out || (k > 0 && (!w_gate || !w_up || !x))) return LOOM_ERR_NULL;
    if (misaligned(w_gate, 4) || misaligned(w_up, 4) || misaligned(x, 4) || misaligned(gate_scale, 4) ||
        misaligned(up_scale, 4) || misaligned(x_scale, 4) || misaligned(out, element_size(type)))
        return LOOM_ERR_ALIGN;
    const loom::I8Product p = {w_gate,    gate_scale,  w_up,         up_scale, x,   x_scale,   nullptr,
                               (int)rows, (int)tokens, (int)(k / 4), act,      out, out_stride};
    return launch([&] { return loom::launch_i8_gated_projection(cfg, p, type, (hipStream_t)stream); });
}

extern "C" int loom_i8_gated_projection_backward_workspace(int64_t rows, int64_t k, int64_t tokens, int type,
                                                           int64_t *bytes) {
    if (!bytes) return LOOM_ERR_NULL;
    loom_launch_config cfg;
    if (int st = product_sizes(loom::kI8GatedBackward, rows, k, tokens, type, rows, &cfg)) return st;
    *bytes = loom::gated_backward_workspace_bytes(rows, k, tokens, type);
    return LOOM_OK;
}

extern "C" int loom_i8_gated_projection_backward(const int32_t *w_gate, const float *gate_scale, const int32_t *w_up,
                                                 const float *up_scale, const int32_t *x, const float *x_scale,
                                                 int64_t rows, int64_t k, int64_t tokens, int act, const void *d_out,
                                                 int type, int64_t d_stride, void *d_x, float *d_gate_scale,
                                                 float *d_up_scale, void *workspace, int64_t workspace_bytes,
                                                 void *stream) {
    if (!known_act(act)) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    if (int st = product_sizes(loom::kI8GatedBackward, rows, k, tokens, type, d_stride, &cfg)) return st;
    if (workspace_bytes < loom::gated_backward_workspace_bytes(rows, k, tokens, type)) return LOOM_ERR_RANGE;
    if ((!d_x || tokens == 0 || k == 0) && ((!d_gate_scale && !d_up_scale) || rows == 0)) return LOOM_OK;
    if (rows > 0 && tokens > 0 &&
        (!gate_scale || !up_scale || !d_out || !workspace || (k > 0 && (!w_gate || !w_up || !x))))
        return LOOM_ERR_NULL;
    if (misaligned(w_gate, 4) || misaligned(w_up, 4) || misaligned(x, 4) || misaligned(gate_scale, 4) ||
        misaligned(up_scale, 4) || misaligned(x_scale, 4) || misaligned(d_out, element_size(type)) ||
        misaligned(d_x, element_size(type)) || misaligned(d_gate_scale, 4) || misaligned(d_up_scale, 4) ||
        misaligned(workspace, 16))
        return LOOM_ERR_ALIGN;
    const loom::I8Product p = {w_gate,    gate_scale,  w_up,         up_scale, x,       x_scale, nullptr,
                               (int)rows, (int)tokens, (int)(k / 4), act,      nullptr, 0};
    const auto run = type == LOOM_F32   ? loom::launch_i8_gated_backward_f32
                     : type == LOOM_F16 ? loom::launch_i8_gated_backward_f16
                                        : loom::launch_i8_gated_backward_bf16;
    return launch([&] {
        return run(cfg, p, d_out, d_stride, d_x, d_gate_scale, d_up_scale, workspace, (hipStream_t)stream);
    });
}

namespace {

bool known_score(int score) { return score == LOOM_SOFTMAX || score == LOOM_SIGMOID; }

// The size checks shared by the router and its gradient.
int route_sizes(loom::ExportId id, int64_t tokens, int64_t experts, int64_t groups, int64_t top_k, int type, int score,
                int64_t stride, loom_launch_config *cfg) {
    if (tokens < 0 || tokens > kMaxRows || !known_type(type) || !known_score(score)) return LOOM_ERR_RANGE;
    if (experts < 1 || experts > loom::kRouteMaxExperts || groups < 1 || groups > loom::kRouteMaxGroups || top_k < 1 ||
        top_k > loom::kRouteMaxTopK)
        return LOOM_ERR_RANGE;
    if (stride < experts || top_k > experts) return LOOM_ERR_SHAPE;
    if (tokens > 0 && stride > (INT64_MAX / 4) / tokens) return LOOM_ERR_RANGE;
    const int64_t w[4] = {tokens, experts, groups, top_k};
    return loom::evaluate_launch(id, w, cfg);
}

}  // namespace

extern "C" int loom_route_experts(const void *logits, int type, int64_t tokens, int64_t experts, int64_t row_stride,
                                  int score, const float *bias, int64_t groups, int64_t top_groups, int64_t group_top,
                                  int64_t top_k, int renormalize, float scale, int32_t *ids, float *weights,
                                  void *stream) {
    if (group_top < 1 || group_top > 2) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    if (int st = route_sizes(loom::kRouteExperts, tokens, experts, groups, top_k, type, score, row_stride, &cfg)) return st;
    if (top_groups < 1 || top_groups > groups) return LOOM_ERR_RANGE;
    if (experts % groups != 0 || top_k > top_groups * (experts / groups)) return LOOM_ERR_SHAPE;
    if (tokens == 0) return LOOM_OK;
    if (!logits || !ids || !weights) return LOOM_ERR_NULL;
    if (misaligned(logits, element_size(type)) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4))
        return LOOM_ERR_ALIGN;
    loom::RouteArgs a = {};
    a.logits = logits, a.bias = bias, a.tokens = tokens, a.stride = row_stride;
    a.type = type, a.score = score, a.experts = (int)experts, a.groups = (int)groups, a.top_groups = (int)top_groups;
    a.group_top = (int)group_top, a.top_k = (int)top_k, a.renormalize = renormalize != 0, a.scale = scale;
    a.ids = ids, a.weights = weights;
    return launch([&] { return loom::launch_route_experts(cfg, a, (hipStream_t)stream); });
}

extern "C" int loom_route_experts_backward(const void *logits, int type, int64_t tokens, int64_t experts,
                                           int64_t row_stride, int score, int64_t top_k, int renormalize, float scale,
                                           const int32_t *ids, const float *d_weights, void *d_logits, int64_t d_stride,
                                           void *stream) {
    loom_launch_config cfg;
    if (int st = route_sizes(loom::kRouteExpertsBackward, tokens, experts, 1, top_k, type, score, row_stride, &cfg))
        return st;
    if (d_stride < experts) return LOOM_ERR_SHAPE;
    if (tokens > 0 && d_stride > (INT64_MAX / 4) / tokens) return LOOM_ERR_RANGE;
    if (tokens == 0) return LOOM_OK;
    if (!logits || !ids || !d_weights || !d_logits) return LOOM_ERR_NULL;
    if (misaligned(logits, element_size(type)) || misaligned(ids, 4) || misaligned(d_weights, 4) ||
        misaligned(d_logits, element_size(type)))
        return LOOM_ERR_ALIGN;
    loom::RouteArgs a = {};
    a.logits = logits, a.tokens = tokens, a.stride = row_stride, a.type = type, a.score = score;
    a.experts = (int)experts, a.groups = 1, a.top_groups = 1, a.group_top = 1, a.top_k = (int)top_k;
    a.renormalize = renormalize != 0, a.scale = scale, a.ids = const_cast<int32_t *>(ids);
    a.d_weights = d_weights, a.d_logits = d_logits, a.d_stride = d_stride;
    return launch([&] { return loom::launch_route_experts_backward(cfg, a, (hipStream_t)stream); });
}

namespace {

int group_sizes(int64_t tokens, int64_t routes, int64_t experts, loom_launch_config *cfg) {
    if (tokens < 0 || tokens > kMaxRows || routes < 0 || routes > (int64_t(1) << 20) || tokens * routes > kMaxRows ||
        experts < 1 || experts > loom::kGroupMaxExperts)
        return LOOM_ERR_RANGE;
    const int64_t w[2] = {tokens * routes, experts};
    return loom::evaluate_launch(loom::kGroupRoutes, w, cfg);
}

}  // namespace

extern "C" int loom_group_routes_workspace(int64_t tokens, int64_t routes, int64_t experts, int64_t *bytes) {
    if (!bytes) return LOOM_ERR_NULL;
    loom_launch_config cfg;
    if (int st = group_sizes(tokens, routes, experts, &cfg)) return st;
    *bytes = loom::group_workspace_bytes(tokens * routes, experts);
    return LOOM_OK;
}

extern "C" int loom_group_routes(const int32_t *ids, int64_t tokens, int64_t routes, int64_t experts, int32_t *slots,
                                 int32_t *rows, int32_t *offsets, void *workspace, int64_t workspace_bytes,
                                 void *stream) {
    loom_launch_config cfg;
    if (int st = group_sizes(tokens, routes, experts, &cfg)) return st;
    const int64_t pairs = tokens * routes, need = loom::group_workspace_bytes(pairs, experts);
    if (workspace_bytes < need) return LOOM_ERR_RANGE;
    if (!offsets || (pairs > 0 && (!ids || !slots || !rows)) || (need > 0 && !workspace)) return LOOM_ERR_NULL;
    if (misaligned(ids, 4) || misaligned(slots, 4) || misaligned(rows, 4) || misaligned(offsets, 4) ||
        misaligned(workspace, 4))
        return LOOM_ERR_ALIGN;
    const loom::GroupArgs a = {ids,   pairs, routes > 0 ? routes : 1, loom::group_part(pairs), (int)experts, slots,
                               rows, offsets, (int32_t *)workspace};
    return launch([&] { return loom::launch_group_routes(cfg, a, (hipStream_t)stream); });
}

namespace {

// The size checks of the 4-bit products; experts 0 for the dense one.
int i4_sizes(loom::ExportId id, int64_t rows, int64_t k, int64_t tokens, int64_t group, int64_t experts,
             int scale_type, int type, int64_t stride, loom_launch_config *cfg) {
    if (k < 0 || k > loom::kI4MaxK || rows < 0 || rows > kMaxRows || tokens < 0 || tokens > kMaxRows ||
        !known_type(type) || !known_type(scale_type) || group < 32 || group > (int64_t(1) << 17))
        return LOOM_ERR_RANGE;
    if (id != loom::kI4Matmul && (experts < 1 || experts > loom::kI4MaxExperts)) return LOOM_ERR_RANGE;
    if (k % 32 != 0 || (group & (group - 1)) != 0 || stride < rows) return LOOM_ERR_SHAPE;
    if (tokens > 0 && stride > (INT64_MAX / 4) / tokens) return LOOM_ERR_RANGE;
    const int64_t w[5] = {rows, k, tokens, group, experts};
    return loom::evaluate_launch(id, w, cfg);
}

void i4_fill(loom::I4Product &p, int64_t rows, int64_t k, int64_t tokens, int64_t group, int64_t experts) {
    p.rows = (int)rows, p.tokens = (int)tokens, p.chunks = (int)(k / 32);
    p.groups = (int)loom::ceil_of(k, group), p.chunk_shift = __builtin_ctzll((uint64_t)group) - 5;
    p.experts = (int)experts;
}

}  // namespace

extern "C" int loom_i4_matmul(const int32_t *w, const void *w_scale, int scale_type, int64_t group, const int32_t *x,
                              const float *x_scale, const float *bias, int64_t rows, int64_t k, int64_t tokens,
                              void *out, int type, int64_t out_stride, void *stream) {
    loom_launch_config cfg;
    if (int st = i4_sizes(loom::kI4Matmul, rows, k, tokens, group, 0, scale_type, type, out_stride, &cfg)) return st;
    if (rows == 0 || tokens == 0) return LOOM_OK;
    if (!out || (k > 0 && (!w || !w_scale || !x))) return LOOM_ERR_NULL;
    if (misaligned(w, 16) || misaligned(x, 16) || misaligned(w_scale, element_size(scale_type)) ||
        misaligned(x_scale, 4) || misaligned(bias, 4) || misaligned(out, element_size(type)))
        return LOOM_ERR_ALIGN;
    loom::I4Product p = {};
    i4_fill(p, rows, k, tokens, group, 1);
    p.w = w, p.w_scale = w_scale, p.x = x, p.x_scale = x_scale, p.bias = bias, p.x_rows = tokens;
    p.out = out, p.out_stride = out_stride;
    return launch([&] { return loom::launch_i4_product(cfg, p, loom::kI4Dense, scale_type, type, (hipStream_t)stream); });
}

extern "C" int loom_i4_expert_matmul(const int32_t *w, const void *w_scale, int scale_type, int64_t group,
                                     const int32_t *x, const float *x_scale, int64_t x_rows, const int32_t *index,
                                     const int32_t *offsets, const float *bias, int64_t experts, int64_t rows,
                                     int64_t k, int64_t pairs, void *out, int type, int64_t out_stride, void *stream) {
    loom_launch_config cfg;
    if (int st = i4_sizes(loom::kI4ExpertMatmul, rows, k, pairs, group, experts, scale_type, type, out_stride, &cfg))
        return st;
    if (x_rows < 0 || x_rows > kMaxRows) return LOOM_ERR_RANGE;
    if (pairs > 0 && x_rows < (index ? 1 : pairs)) return LOOM_ERR_SHAPE;
    if (rows == 0 || pairs == 0) return LOOM_OK;
    if (!offsets || !out || (k > 0 && (!w || !w_scale || !x))) return LOOM_ERR_NULL;
    if (misaligned(w, 16) || misaligned(x, 16) || misaligned(w_scale, element_size(scale_type)) ||
        misaligned(x_scale, 4) || misaligned(index, 4) || misaligned(offsets, 4) || misaligned(bias, 4) ||
        misaligned(out, element_size(type)))
        return LOOM_ERR_ALIGN;
    loom::I4Product p = {};
    i4_fill(p, rows, k, pairs, group, experts);
    p.w = w, p.w_scale = w_scale, p.x = x, p.x_scale = x_scale, p.bias = bias, p.index = index, p.offsets = offsets;
    p.x_rows = x_rows, p.out = out, p.out_stride = out_stride;
    return launch([&] { return loom::launch_i4_product(cfg, p, loom::kI4Routed, scale_type, type, (hipStream_t)stream); });
}

extern "C" int loom_i4_expert_gated_projection(const int32_t *w_gate, const void *gate_scale, const int32_t *w_up,
                                               const void *up_scale, int scale_type, int64_t group, const int32_t *x,
                                               const float *x_scale, int64_t x_rows, const int32_t *index,
                                               const int32_t *offsets, int64_t experts, int64_t rows, int64_t k,
                                               int64_t pairs, int act, void *out, int type, int64_t out_stride,
                                               void *stream) {
    if (!known_act(act)) return LOOM_ERR_RANGE;
    loom_launch_config cfg;
    if (int st = i4_sizes(loom::kI4ExpertGatedProjection, rows, k, pairs, group, experts, scale_type, type, out_stride,
                          &cfg))
        return st;
    if (x_rows < 0 || x_rows > kMaxRows) return LOOM_ERR_RANGE;
    if (pairs > 0 && x_rows < (index ? 1 : pairs)) return LOOM_ERR_SHAPE;
    if (rows == 0 || pairs == 0) return LOOM_OK;
    if (!offsets || !out || (k > 0 && (!w_gate || !w_up || !gate_scale || !up_scale || !x))) return LOOM_ERR_NULL;
    if (misaligned(w_gate, 16) || misaligned(w_up, 16) || misaligned(x, 16) ||
        misaligned(gate_scale, element_size(scale_type)) || misaligned(up_scale, element_size(scale_type)) ||
        misaligned(x_scale, 4) || misaligned(index, 4) || misaligned(offsets, 4) || misaligned(out, element_size(type)))
        return LOOM_ERR_ALIGN;
    loom::I4Product p = {};
    i4_fill(p, rows, k, pairs, group, experts);
    p.w = w_gate, p.w_scale = gate_scale, p.w_up = w_up, p.up_scale = up_scale, p.x = x, p.x_scale = x_scale;
    p.index = index, p.offsets = offsets, p.act = act, p.x_rows = x_rows, p.out = out, p.out_stride = out_stride;
    return launch([&] { return loom::launch_i4_product(cfg, p, loom::kI4RoutedGated, scale_type, type, (hipStream_t)stream); });
}
