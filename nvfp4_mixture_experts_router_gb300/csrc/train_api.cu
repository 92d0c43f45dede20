// Entry points of the training operators (moe_nvfp4_train.h): argument
// validation and launches.
#include <math.h>

#include "host.h"
#include "layout.h"
#include "train_kernels.h"

using namespace moe;

namespace {

constexpr int64_t kMaxRows = 1ll << 27;
constexpr int kMaxTokens = 1 << 22;

bool tokens_ok(int T) { return T >= 0 && T <= kMaxTokens; }
bool width_ok(int H) { return H >= 1 && H <= 65536; }
bool dtype_ok(int d) { return d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F32; }
int elem_of(int d) { return d == MOE_DTYPE_F32 ? 4 : 2; }
bool routes_ok(int T, int K) { return tokens_ok(T) && K >= 1 && K <= 32 && (int64_t)T * K <= (1 << 26); }

// A range of device memory an argument covers: `bytes` from p on; of rows
// `stride` bytes apart (0: one run) only the first `width` bytes each.
struct Span {
    const void* p;
    size_t bytes;
    bool out;
    size_t stride = 0, width = 0;
};

// The rows of a [rows][width] buffer, `stride` elements apart.
Span rows_span(const void* p, int64_t rows, int64_t stride, int64_t width, int elem, bool out) {
    const size_t bytes = rows > 0 ? (size_t)((rows - 1) * stride + width) * elem : 0;
    return Span{p, bytes, out, (size_t)stride * elem, (size_t)width * elem};
}

// Do two spans share a byte?  Rows of one stride share none where their columns,
// taken modulo the stride, lie side by side; other ranges that cross count as
// shared.
bool shared(const Span& a, const Span& b) {
    if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return false;
    if (a.stride == 0 || a.stride != b.stride) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t after = y >= x ? (y - x) % a.stride : (a.stride - (x - y) % a.stride) % a.stride;   // b's column from a's
    return after < a.width || after + b.width > a.stride;
}

bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= (1ll << 40); }

// Every span with bytes has a pointer aligned to `align`, and no output
// overlaps another span.
bool spans_ok(const Span* s, int n, const uintptr_t* align) {
    for (int i = 0; i < n; ++i)
        if (s[i].bytes && (!s[i].p || !aligned(s[i].p, align[i]))) return false;
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j)
            if (i != j && s[i].out && s[i].bytes && s[j].bytes && shared(s[i], s[j])) return false;
    return true;
}

// The launch context of one call.  Every kernel waits for its predecessor
// before it touches memory, so all may start early.
moe_status begin(void* stream, LaunchCtx* c, int* sms, int* device = nullptr) {
    const moe_status st = device_state(sms, device);
    if (st != MOE_OK) return st;
    c->stream = static_cast<cudaStream_t>(stream);
    c->pdl = true;
    return MOE_OK;
}

bool row_args_ok(int T, int H, int K, int64_t rows, int dtype, int64_t stride) {
    return routes_ok(T, K) && width_ok(H) && dtype_ok(dtype) && rows >= 0 && rows <= kMaxRows && stride_ok(stride, H);
}

// The row that MOE_DEBUG_NORM_SKIP_COPY in a layer norm's dtype leaves out, or
// -1; takes the flag out of the dtype.
int skipped_row(int T, int* dtype) {
    if (*dtype < 0 || !(*dtype & MOE_DEBUG_NORM_SKIP_COPY)) return -1;
    *dtype &= ~MOE_DEBUG_NORM_SKIP_COPY;
    return T / 2;
}

}  // namespace

extern "C" {

size_t moe_nvfp4_sort_workspace_bytes(int T, int E, int K) {
    if (!routes_ok(T, K) || E < 1 || E > 1024) return 0;
    return sort_workspace_bytes(T, E, K);
}

moe_status moe_nvfp4_sort_routes(int T, int E, int K, const int32_t* topk_ids, int32_t* count, int32_t* offsets,
                                 int32_t* row_of_route, int32_t* route_of_row, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    const size_t need = moe_nvfp4_sort_workspace_bytes(T, E, K);
    if (need == 0) return MOE_ERR_INVALID_ARG;
    const size_t rb = (size_t)T * K * 4;
    const Span s[] = {{topk_ids, rb, false},     {count, (size_t)E * 4, true}, {offsets, (size_t)(E + 1) * 4, true},
                      {row_of_route, rb, true},  {route_of_row, rb, true},     {workspace, need, true}};
    const uintptr_t al[] = {4, 4, 4, 4, 4, 256};
    if (!spans_ok(s, 6, al)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_sort_routes(c, T, E, K, topk_ids, count, offsets, row_of_route, route_of_row,
                                          static_cast<int*>(workspace)));
}

moe_status moe_nvfp4_dispatch(int T, int H, int K, int64_t rows, int dtype, const void* x, int64_t x_stride,
                              const int32_t* row_of_route, const int32_t* rows_used, void* x_rows, void* stream) {
    if (!row_args_ok(T, H, K, rows, dtype, x_stride)) return MOE_ERR_INVALID_ARG;
    const int el = elem_of(dtype);
    const Span s[] = {rows_span(x, T, x_stride, H, el, false),
                      {row_of_route, (size_t)T * K * 4, false},
                      {rows_used, rows_used ? 4u : 0u, false},
                      {x_rows, (size_t)rows * H * el, true}};
    const uintptr_t al[] = {(uintptr_t)el, 4, 4, (uintptr_t)el};
    if (!spans_ok(s, 4, al)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_dispatch(c, T, H, K, rows, el, x, x_stride, row_of_route, rows_used, x_rows));
}

// combine, and dispatch_backward as its form without weights
static moe_status gather_sum(int T, int H, int K, int64_t rows, int dtype, const void* in, const int32_t* row_of_route,
                             bool weighted, const float* w, void* out, int64_t out_stride, void* stream) {
    if (!row_args_ok(T, H, K, rows, dtype, out_stride)) return MOE_ERR_INVALID_ARG;
    const int el = elem_of(dtype);
    const Span s[] = {{in, (size_t)rows * H * el, false},
                      {row_of_route, (size_t)T * K * 4, false},
                      {w, weighted ? (size_t)T * K * 4 : 0, false},
                      rows_span(out, T, out_stride, H, el, true)};
    const uintptr_t al[] = {(uintptr_t)el, 4, 4, (uintptr_t)el};
    if (!spans_ok(s, 4, al)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_combine(c, T, H, K, rows, el, in, row_of_route, weighted ? w : nullptr, out, out_stride));
}

moe_status moe_nvfp4_dispatch_backward(int T, int H, int K, int64_t rows, int dtype, const void* dx_rows,
                                       const int32_t* row_of_route, void* dx, int64_t dx_stride, void* stream) {
    return gather_sum(T, H, K, rows, dtype, dx_rows, row_of_route, false, nullptr, dx, dx_stride, stream);
}

moe_status moe_nvfp4_combine(int T, int H, int K, int64_t rows, int dtype, const void* o_rows,
                             const int32_t* row_of_route, const float* topk_w, void* y, int64_t y_stride,
                             void* stream) {
    return gather_sum(T, H, K, rows, dtype, o_rows, row_of_route, true, topk_w, y, y_stride, stream);
}

moe_status moe_nvfp4_combine_backward(int T, int H, int K, int64_t rows, int dtype, const void* dy, int64_t dy_stride,
                                      const void* o_rows, const int32_t* row_of_route, const float* topk_w,
                                      const int32_t* rows_used, void* do_rows, float* dw, void* stream) {
    if (!row_args_ok(T, H, K, rows, dtype, dy_stride)) return MOE_ERR_INVALID_ARG;
    const int el = elem_of(dtype);
    const size_t rb = (size_t)T * K * 4;
    const Span s[] = {rows_span(dy, T, dy_stride, H, el, false),
                      {o_rows, (size_t)rows * H * el, false},
                      {row_of_route, rb, false},
                      {topk_w, rb, false},
                      {rows_used, rows_used ? 4u : 0u, false},
                      {do_rows, (size_t)rows * H * el, true},
                      {dw, rb, true}};
    const uintptr_t al[] = {(uintptr_t)el, (uintptr_t)el, 4, 4, 4, (uintptr_t)el, 4};
    if (!spans_ok(s, 7, al)) return MOE_ERR_INVALID_ARG;
    if (T == 0 && rows == 0) return MOE_OK;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_combine_backward(c, T, H, K, rows, el, dy, dy_stride, o_rows, row_of_route, topk_w,
                                               rows_used, do_rows, dw));
}

static moe_status expert_product(int product, int64_t rows, int N, int K, int E, const void* a, const void* b,
                                 const int32_t* count, const int32_t* offsets, void* out, uint32_t* status,
                                 void* stream) {
    if (rows < 0 || rows > kMaxRows || E < 1 || E > 1024) return MOE_ERR_INVALID_ARG;
    if (N < 8 || N % 8 != 0 || N > 65536 || K < 8 || K % 8 != 0 || K > 65536) return MOE_ERR_INVALID_ARG;
    if ((int64_t)E * N >= (1ll << 31) || (int64_t)E * K >= (1ll << 31)) return MOE_ERR_INVALID_ARG;
    const size_t xb = (size_t)rows * K * 2, yb = (size_t)rows * N * 2, wb = (size_t)E * N * K * 2;
    const bool fwd = product == kExpertForward, wg = product == kExpertWgrad;
    const Span s[] = {{a, fwd ? xb : yb, false},
                      {b, wg ? xb : wb, false},
                      {count, (size_t)E * 4, false},
                      {offsets, (size_t)E * 4, false},
                      {status, status ? 4u : 0u, true},
                      {out, fwd ? yb : wg ? wb : xb, true}};
    const uintptr_t al[] = {16, 16, 4, 4, 4, 16};
    if (!spans_ok(s, 6, al)) return MOE_ERR_INVALID_ARG;
    if (rows == 0 && !wg && !status) return MOE_OK;
    LaunchCtx c;
    int sms = 0, device = 0;
    const moe_status st = begin(stream, &c, &sms, &device);
    if (st != MOE_OK) return st;
    const ExpertArgs args{rows, N, K, E, a, b, out, count, offsets, status};
    return cuda_status(launch_expert_linear(c, product, device, args));
}

moe_status moe_nvfp4_expert_linear(int64_t rows, int N, int K, int E, const void* x_rows, const void* w,
                                   const int32_t* count, const int32_t* offsets, void* y_rows, uint32_t* status,
                                   void* stream) {
    return expert_product(kExpertForward, rows, N, K, E, x_rows, w, count, offsets, y_rows, status, stream);
}

moe_status moe_nvfp4_expert_linear_dgrad(int64_t rows, int N, int K, int E, const void* dy_rows, const void* w,
                                         const int32_t* count, const int32_t* offsets, void* dx_rows, uint32_t* status,
                                         void* stream) {
    return expert_product(kExpertDgrad, rows, N, K, E, dy_rows, w, count, offsets, dx_rows, status, stream);
}

moe_status moe_nvfp4_expert_linear_wgrad(int64_t rows, int N, int K, int E, const void* dy_rows, const void* x_rows,
                                         const int32_t* count, const int32_t* offsets, void* dw, uint32_t* status,
                                         void* stream) {
    return expert_product(kExpertWgrad, rows, N, K, E, dy_rows, x_rows, count, offsets, dw, status, stream);
}

moe_status moe_nvfp4_layer_norm(int T, int H, int dtype, const void* x, int64_t x_stride, const float* gamma,
                                const float* beta, float eps, void* y, int64_t y_stride, float* mean, float* rstd,
                                void* stream) {
    const int skip_row = skipped_row(T, &dtype);
    if (!tokens_ok(T) || !width_ok(H) || !dtype_ok(dtype) || !stride_ok(x_stride, H) || !stride_ok(y_stride, H))
        return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || isinf(eps) || (mean == nullptr) != (rstd == nullptr)) return MOE_ERR_INVALID_ARG;
    const int el = elem_of(dtype);
    const bool in_place = y == x && y_stride == x_stride;
    const size_t sb = mean ? (size_t)T * 4 : 0;
    const Span s[] = {rows_span(x, in_place ? 0 : T, x_stride, H, el, false),
                      {gamma, (size_t)H * 4, false},
                      {beta, beta ? (size_t)H * 4 : 0, false},
                      rows_span(y, T, y_stride, H, el, true),
                      {mean, sb, true},
                      {rstd, sb, true}};
    const uintptr_t al[] = {(uintptr_t)el, 4, 4, (uintptr_t)el, 4, 4};
    if (!spans_ok(s, 6, al)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_layer_norm(c, T, H, el, x, x_stride, gamma, beta, eps, y, y_stride, mean, rstd,
                                         skip_row));
}

size_t moe_nvfp4_layer_norm_workspace_bytes(int T, int H) {
    if (!tokens_ok(T) || !width_ok(H)) return 0;
    return layer_norm_workspace_bytes(T, H);
}

moe_status moe_nvfp4_layer_norm_backward(int T, int H, int dtype, const void* dy, int64_t dy_stride, const void* x,
                                         int64_t x_stride, const float* gamma, const float* mean, const float* rstd,
                                         void* dx, int64_t dx_stride, float* dgamma, float* dbeta, void* workspace,
                                         size_t workspace_bytes, void* stream) {
    const int skip_row = skipped_row(T, &dtype);
    if (!tokens_ok(T) || !width_ok(H) || !dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
    if (!stride_ok(dy_stride, H) || !stride_ok(x_stride, H) || !stride_ok(dx_stride, H)) return MOE_ERR_INVALID_ARG;
    const int el = elem_of(dtype);
    const size_t need = layer_norm_workspace_bytes(T, H);
    const bool over_dy = dx == dy && dx_stride == dy_stride, over_x = dx == x && dx_stride == x_stride;
    const Span s[] = {rows_span(dy, over_dy ? 0 : T, dy_stride, H, el, false),
                      rows_span(x, over_x ? 0 : T, x_stride, H, el, false),
                      {gamma, (size_t)H * 4, false},
                      {mean, (size_t)T * 4, false},
                      {rstd, (size_t)T * 4, false},
                      rows_span(dx, T, dx_stride, H, el, true),
                      {dgamma, (size_t)H * 4, true},
                      {dbeta, dbeta ? (size_t)H * 4 : 0, true},
                      {workspace, need, true}};
    const uintptr_t al[] = {(uintptr_t)el, (uintptr_t)el, 4, 4, 4, (uintptr_t)el, 4, 4, 256};
    if (!spans_ok(s, 9, al)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_layer_norm_backward(c, T, H, el, dy, dy_stride, x, x_stride, gamma, mean, rstd, dx,
                                                  dx_stride, dgamma, dbeta, static_cast<float*>(workspace), skip_row));
}

size_t moe_nvfp4_grad_norm_workspace_bytes(int n) {
    if (n < 0 || n > 65536) return 0;
    return grad_norm_workspace_bytes(n);
}

static bool grad_list_ok(int n, const void* const* grads, const int64_t* numels, const int32_t* dtypes) {
    if (n < 0 || n > 65536) return false;
    if (n > 0 && (!grads || !numels || !dtypes)) return false;
    for (int i = 0; i < n; ++i) {
        if (!dtype_ok(dtypes[i]) || numels[i] < 0 || numels[i] >= (1ll << 40)) return false;
        if (numels[i] > 0 && (!grads[i] || !aligned(grads[i], elem_of(dtypes[i])))) return false;
    }
    return true;
}

moe_status moe_nvfp4_grad_norm(int n, const void* const* grads, const int64_t* numels, const int32_t* dtypes,
                               float* norm, void* workspace, size_t workspace_bytes, void* stream) {
    if (!grad_list_ok(n, grads, numels, dtypes) || !norm || !aligned(norm, 4)) return MOE_ERR_INVALID_ARG;
    const size_t need = grad_norm_workspace_bytes(n);
    if (!workspace || !aligned(workspace, 256) || overlaps(norm, 4, workspace, need)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_grad_norm(c, n, grads, numels, dtypes, norm, static_cast<float*>(workspace)));
}

moe_status moe_nvfp4_grad_clip(int n, const void* const* grads, void* const* out, const int64_t* numels,
                               const int32_t* dtypes, const float* norm, float max_norm, float eps, void* stream) {
    if (!grad_list_ok(n, grads, numels, dtypes) || !norm || !aligned(norm, 4)) return MOE_ERR_INVALID_ARG;
    if (!(max_norm >= 0.0f) || isinf(max_norm) || !(eps >= 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    if (n > 0 && !out) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (numels[i] > 0 && (!out[i] || !aligned(out[i], elem_of(dtypes[i])))) return MOE_ERR_INVALID_ARG;
    LaunchCtx c;
    int sms = 0;
    const moe_status st = begin(stream, &c, &sms);
    if (st != MOE_OK) return st;
    return cuda_status(launch_grad_clip(c, sms, n, grads, out, numels, dtypes, norm, max_norm, eps));
}

}  // extern "C"
